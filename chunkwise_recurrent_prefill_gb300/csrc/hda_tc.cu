// Linear attention with one decay per head on the tensor cores.
#include "hda_internal.h"

namespace gla {

bool hda_tc_supported(const HdaProblem &) { return false; }
size_t hda_tc_workspace_bytes(const HdaProblem &, int, int) { return 0; }
cudaError_t launch_hda_tc(const HdaProblem &, int, int, void *, unsigned int *, cudaStream_t) {
    return cudaErrorNotSupported;
}

}  // namespace gla

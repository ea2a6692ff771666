// Argument checks shared by the ABI layers of the operators (host code).
#pragma once

#include <stdint.h>

#include "gla.h"
#include "gla_internal.h"

namespace gla {
namespace api {

constexpr int64_t kMostElems = int64_t(1) << 62;

inline bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }
inline bool bad_int(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u); }
// Element alignment of a strided tensor's base (rows may start anywhere).
inline bool unaligned(const void *p, int io) {
    return p && (reinterpret_cast<uintptr_t>(p) & (io == GLA_IO_BF16 ? 1u : 3u));
}

// a * b of non-negative sizes; false past 2^62 (so byte counts still fit)
inline bool mul_ok(int64_t a, int64_t b, int64_t *r) {
    if (a < 0 || b < 0 || (a != 0 && b > kMostElems / 16 / a)) return false;
    *r = a * b;
    return true;
}

// A memory range an argument covers.
struct Range {
    const void *p;
    int64_t bytes;
};
inline bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (size_t)b.bytes && y < x + (size_t)a.bytes;
}
// GLA_ERR_ALIAS if an output overlaps an input or another output.
inline gla_status check_alias(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return GLA_ERR_ALIAS;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return GLA_ERR_ALIAS;
    }
    return GLA_OK;
}

// The caller's workspace if it will do, else the stream's own.
inline gla_status get_workspace(void *ws, size_t bytes, size_t need, cudaStream_t s, const Range *used,
                         int nu, void **out) {
    *out = nullptr;
    if (ws) {
        if (misaligned(ws) || bytes < need) return GLA_ERR_WORKSPACE;
        for (int i = 0; i < nu; ++i)
            if (overlap(Range{ws, (int64_t)need}, used[i])) return GLA_ERR_WORKSPACE;
        *out = ws;
        return GLA_OK;
    }
    if (need == 0) return GLA_OK;
    return (gla_status)gla::stream_workspace(s, need, out);
}

}  // namespace api
}  // namespace gla

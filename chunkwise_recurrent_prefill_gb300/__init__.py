"""GB300 (sm_103a) gated linear attention (GLA) prefill forward, the gated delta rule
forward (gdn_fwd), and linear attention with one decay per head (hda_*: prompts, gradients and
single tokens) with the group norm and the state pages that go with it.

The compute runs in ``_build/libgla.so`` (CUDA kernels behind the C ABI of
``include/gla.h``); ``gla.py`` only marshals torch tensors onto it.
"""
from .gla import (  # noqa: F401
    GLAError,
    gdn_fwd,
    gdn_workspace_size,
    gla_fwd,
    gla_fwd_noalloc,
    gla_fwd_varlen,
    gla_step,
    last_device_status,
    load_library,
    workspace_size,
)
from .hda import (  # noqa: F401
    hda_bwd,
    hda_fwd,
    hda_path_for,
    hda_step,
    hda_workspace_size,
)
from .norm import (  # noqa: F401
    group_norm_bwd,
    group_norm_fwd,
    group_norm_workspace_size,
)
from .pages import (  # noqa: F401
    pages_compact,
    pages_copy,
    pages_fork,
    pages_free,
    pages_workspace_size,
)
from .workloads import (  # noqa: F401
    BENCH_WORKLOAD,
    GDN_BENCH_WORKLOAD,
    GDN_WORKLOADS,
    WORKLOADS,
    Workload,
    make_gdn_inputs,
    make_inputs,
)

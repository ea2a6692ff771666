"""GB300 (sm_103a) gated linear attention (GLA) prefill forward, the gated delta rule
forward (gdn_fwd), and linear attention with one decay per head (hda_*: prompts, gradients and
single tokens) with the group norm and the state pages that go with it. Around the recurrences: a
short causal convolution (conv_*), the norm and rotation of queries and keys (qk_norm_*), and the
selective state space scan (ssm_*), for prompts, gradients and single tokens.

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
from .conv import (  # noqa: F401
    conv_bwd,
    conv_fwd,
    conv_step,
    conv_workspace_size,
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
from .qk_norm import (  # noqa: F401
    qk_norm_bwd,
    qk_norm_fwd,
    qk_norm_workspace_size,
)
from .ssm import (  # noqa: F401
    ssm_bwd,
    ssm_fwd,
    ssm_step,
    ssm_workspace_size,
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

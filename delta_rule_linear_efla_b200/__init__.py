"""B200-native Exact Flow Linear Attention (EFLA): forward, decode and backward passes.

The computation lives in libefla.so (hand-written CUDA for sm_100a behind the
C ABI in include/efla.h); `efla` is its Python binding and `inputs` the seeded
synthetic workloads.  Importing the package does not load the library; the
first call does, and raises if it is missing.
"""
from . import inputs  # noqa: F401
from .decay import (  # noqa: F401
    DecayFunction, decay_attention, decay_bwd, decay_chunk_fwd, decay_recurrent_step, decay_workspace_size,
)
from .efla import (  # noqa: F401
    ABI_SYMBOLS, EflaError, EflaFunction, alpha, bwd, chunk_fwd, chunk_fwd_path, efla_attention,
    kernel_launches, last_device_error, load_library, recurrent_step, state_affine, status_str,
    workspace_size,
)
from .norms import (  # noqa: F401
    GatedNormFunction, HeadNormFunction, gated_norm, gated_norm_bwd, gated_norm_fwd, head_norm, head_norm_bwd,
    head_norm_fwd,
)

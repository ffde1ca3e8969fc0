"""MI355X-native sLSTM (mix='diag') forward: Newton-parallel solve and sequential steps,
hand-written HIP for gfx950 behind a C ABI (include/slstm.h), with this thin ctypes binding; and
what stands beside it in a block: layer norm and linear attention with a decay for each head.
"""
from .layer_norm import layer_norm_backward, layer_norm_forward  # noqa: F401
from .linear_attention import (  # noqa: F401
    linear_attention_backward,
    linear_attention_forward,
    linear_attention_step,
)
from .slstm import (  # noqa: F401
    NewtonDivergenceError,
    NewtonStats,
    SlstmError,
    input_projection,
    load,
    newton_forward,
    newton_workspace_bytes,
    read_stats,
    residual_jacobian,
    scan_block4,
    sequential_forward,
    warm_start,
)

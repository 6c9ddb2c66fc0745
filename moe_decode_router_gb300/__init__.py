"""GB300 (sm_103a) Flint MoE sublayer: C-ABI CUDA library plus a thin binding.

The compute path is libflint_moe.so (csrc/, declared in include/flint_moe.h);
``flint_moe`` marshals torch tensors into its entry points.
"""

from .flint_moe import (  # noqa: F401
    ACT_GELU,
    ACT_NONE,
    ACT_SILU,
    W_NVFP4,
    W_BF16,
    FlintLayer,
    FlintMoeError,
    alloc_workspace,
    block_gemm,
    combine,
    decode_layer,
    decode_stack,
    device_error,
    gated_linear,
    gated_linear_backward,
    group_pairs,
    integer_gemm,
    integer_quantize_rows,
    linear,
    linear_backward,
    load_library,
    pack_layer,
    pack_weights,
    packed_bytes,
    prefill_layer,
    quantize_rows,
    release,
    route,
    workspace_bytes,
)

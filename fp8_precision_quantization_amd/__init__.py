"""libmxcast: bf16 -> MXFP8 casts, the 128x4 blocked e8m0 scale layout and
the row-wise and tensor-wise fp8 casts on AMD Instinct MI355X (gfx950), the training-step
operators around them (layer norm, MoE router, gated activation and weight gradient from 8-bit
activation checkpoints), and the MXFP4 cast with the products and the gated feed-forward block
that read it, as hand-written HIP kernels behind a C ABI (include/mxcast.h, include/mxtrain.h,
include/mxfp4.h).  This package is the thin Python binding over that ABI;
the library is loaded on first use and its absence is an error."""
from ._binding import (  # noqa: F401
    MX_BLOCK,
    MX_MAX_GROUPS,
    MxError,
    LIB_PATH,
    lib,
    mx_blocked_bytes,
    mx_blocked_grouped_bytes,
    mx_cast_dim0_dim1,
    mx_cast_dim0_dim1_blocked,
    mx_cast_dim0_dim1_grouped_blocked,
    mx_cast_dim0_dim1_mgrouped,
    mx_cast_dim1_3d,
    mx_cast_dim1_3d_blocked,
    mx_gemm_mxfp8,
    mx_grouped_gemm_mxfp8,
    mx_kgrouped_gemm_mxfp8,
    mx_quantize_fp8_rowwise,
    mx_quantize_fp8_tensorwise,
    mx_quantize_fp8_tensorwise_noalloc,
    mx_scales_to_blocked,
    mx_scales_to_blocked_grouped,
    mx_tensorwise_workspace_bytes,
    status_string,
)
from ._train import (  # noqa: F401
    MX_MAX_NORM_COLS,
    MX_MAX_TOPK,
    mx_gated_act,
    mx_gated_act_backward,
    mx_layernorm,
    mx_layernorm_backward,
    mx_layernorm_backward_workspace_bytes,
    mx_layernorm_checkpoint,
    mx_router_balance,
    mx_router_balance_backward,
    mx_router_workspace_bytes,
    mx_wgrad_checkpoint,
    mx_wgrad_checkpoint_workspace_bytes,
)
from ._fp4 import (  # noqa: F401
    MX_MAX_DECODE_ROWS,
    mx_cast_mxfp4,
    mx_dequantize_mxfp4,
    mx_gated_ffn,
    mx_gated_ffn_backward,
    mx_gated_ffn_decode,
    mx_gemm_mxfp4,
    mx_grouped_gemm_mxfp4,
    mx_linear_decode,
)

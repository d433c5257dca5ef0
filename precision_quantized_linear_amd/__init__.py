"""MI355X (gfx950) quantized linear: fp8r and nvfp4 (BFL schemes) with an optional
SVDQuant low-rank branch and smoothing, its INT4 variant, the 8-bit integer linear
(one linear, or one for each expert of a mixture), the block-scaled fp8 linear and the gated
feed-forward block on it, with their backward passes, and the weight-only 4-bit (awq_w4a16)
linear, with GELU and fused-QKV epilogues, the fused GELU MLP, the GELU MLP of experts, and the
norm and rotation of queries and keys.
The HIP library libqpl.so does the work; this package is its thin Python binding."""
from ._binding import (EXPORTS, KERNELS, LIB_PATH, QPL_ACT_GELU_TANH, QPL_ACT_NONE, QPL_ACT_SILU, QPL_FP8B,  # noqa: F401
                       QPL_FP8R, QPL_INT4, QPL_INT8, QPL_NVFP4, Epilogue, Fp8bWeight, Heads, Nvfp4Layer, QPLError,
                       Rope, RopeScaling, amax_bf16, dequant_weight,
                       expert_combine, expert_plan, expert_plan_workspace_bytes, load, nvfp4_global_scale, qk_norm_rope,
                       qk_norm_rope_backward, qk_norm_rope_backward_workspace_bytes, qlinear_awq_w4a16, qlinear_fp8b,
                       qlinear_fp8r, qlinear_fp8r_noalloc, qlinear_gated_fp8b, qlinear_gated_fp8b_backward,
                       qlinear_gated_fp8b_backward_workspace_bytes, qlinear_gated_fp8b_workspace_bytes,
                       qlinear_grouped_int8, qlinear_grouped_int8_workspace_bytes, qlinear_int4,
                       qlinear_int8, qlinear_mlp_nvfp4, qlinear_mlp_nvfp4_workspace_bytes, qlinear_moe_int8,
                       qlinear_moe_int8_workspace_bytes, qlinear_nvfp4, qlinear_weight_grad, qlinear_workspace_bytes,
                       quant_act_fp8_row, quant_act_fp8b, quant_act_int4, quant_act_int8, quant_act_nvfp4,
                       quant_weight_awq, quant_weight_fp8b, rope_frequencies, timing_collect, timing_enable,
                       timing_select, transpose_fp8b)

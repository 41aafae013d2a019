"""DeepSeekMoE layer forward on MI355X (gfx950): FP8 block-scaled experts,
sigmoid + bias group-limited routing, behind the C ABI of libmoe_fp8.so."""
from . import _lib  # noqa: F401
from ._lib import (ACT_GELU, ACT_SILU, QUANT_E4M3, QUANT_INT8, QUANT_NONE, SCORE_SIGMOID,  # noqa: F401
                   SCORE_SOFTMAX, MoEError, fp8_quant_1x128, fp8_quant_128x128,
                   fp8_quant_128x1_grouped, fp8_transpose_128x128, grouped_fp8_gemm,
                   grouped_fp8_gemm_dgrad,
                   grouped_fp8_gemm_swiglu, grouped_fp8_gemm_swiglu_keep, grouped_fp8_wgrad,
                   grouped_bf16_gemm, grouped_bf16_gemm_dgrad, grouped_bf16_gemm_dgrad_glu,
                   grouped_bf16_gemm_glu, grouped_bf16_wgrad,
                   grouped_int8_gemm, grouped_int8_gemm_swiglu, int8_quant_channels,
                   int8_quant_rows, moe_bias_update, moe_combine,
                   moe_combine_backward, moe_combine_norm, moe_combine_norm_backward,
                   moe_combine_norm_backward_workspace_bytes, moe_norm, moe_norm_backward,
                   moe_norm_backward_workspace_bytes, moe_gate, moe_gate_backward, moe_permute, moe_permute_noalloc,
                   moe_permute_workspace_bytes, moe_route,
                   moe_route_scores, moe_route_workspace_bytes, moe_router_backward,
                   moe_router_backward_dense, moe_router_backward_dense_workspace_bytes,
                   moe_router_dcentroids, moe_router_logits, moe_router_logits_backward,
                   moe_seq_balance, moe_seq_balance_workspace_bytes,
                   swiglu_backward, swiglu_backward_grouped, wgrad_chunks)
from .layer import (BackwardBuffers, Bf16BackwardBuffers, Bf16Buffers, Bf16MoELayer,  # noqa: F401
                    BlockBuffers, Buffers, Gate, Int8Buffers, Int8MoELayer, LayerShape, MoEBlock,
                    MoELayer)

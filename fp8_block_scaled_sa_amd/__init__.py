"""MI355X (gfx950) fine-grained block-scaled FP8 GEMM.

D = A . B^T with e4m3 operands, 1x128 LHS scales, 128x128 RHS scales, fp32
per-K-block promotion and a bf16 output, as a dense NT GEMM and as two MoE
grouped layouts (contiguous, masked), plus the 1x128 activation quantiser
that produces the GEMM's LHS and the MoE routing steps around the
contiguous layout, a serving step's mixture-of-experts half for a few tokens
(residual norm to codes, router top-k, the expert layer), and its attention half
over a paged cache of e4m3 codes (rotary positions and the cache's write, its
read, attention). The kernels live in libdg_fp8.so behind the C ABI of
include/dg_fp8.h; this package is its thin Python binding.
"""
from .ops import (DGError, dg_fp8_gemm_nt, dg_fp8_gemm_nt_fmt, dg_fp8_grouped_gemm_contiguous,  # noqa: F401
                  dg_fp8_gemm_nt_ws, dg_fp8_gemm_nt_workspace_bytes, dg_fp8_grouped_gemm_contiguous_ws,
                  dg_fp8_grouped_gemm_contiguous_workspace_bytes, workspace,
                  dg_fp8_grouped_gemm_contiguous_fmt, dg_fp8_grouped_gemm_contiguous_layout,
                  dg_fp8_grouped_gemm_contiguous_to_tokens,
                  dg_fp8_grouped_gemm_masked_fmt,
                  dg_fp8_grouped_gemm_masked, dg_fp8_quantize_1x128, dg_fp8_quantize_1x128_gather,
                  dg_moe_contiguous_max_rows, dg_moe_route_contiguous, dg_moe_unpermute,
                  dg_fp8_rmsnorm_quantize_1x128, dg_moe_gate_topk, dg_fp8_moe_layer,
                  dg_fp8_moe_layer_workspace_bytes, dg_rope_frequencies, dg_fp8_rope_cache_write, dg_fp8_cache_read,
                  dg_fp8_paged_attention, dg_fp8_paged_attention_workspace_bytes)

"""FP8 (e4m3) block-scaled GEMM (NT, and NN/TN/TT with K-major operands), with
M-grouped MoE forms, the K-grouped TN form and an FP8 x FP4 GEMM, for AMD
MI355X (gfx950), with the operators around them: the router, the experts' row
layouts, the quantising scatter and the weighted gather, and low-rank adapters
beside a dense projection.  The kernels live in libdg.so behind the C ABI of
include/dg.h; this package is its Python binding."""
from ._lib import (  # noqa: F401
    DGError,
    EXPORTED,
    LIB_PATH,
    dg_bind_stream_workspace,
    dg_check_grouped_layout,
    dg_choose_config,
    dg_fp8_fp4_gemm_nt,
    dg_fp8_gemm_nn,
    dg_fp8_gemm_nt,
    dg_fp8_gemm_nt_noalloc,
    dg_fp8_gemm_tn,
    dg_fp8_gemm_tt,
    dg_init,
    dg_k_grouped_fp8_gemm_tn_contiguous,
    dg_k_grouped_scatter_fp8,
    dg_lora_bf16_nt,
    dg_m_grouped_fp8_fp4_gemm_nt_contiguous,
    dg_m_grouped_fp8_fp4_gemm_nt_masked,
    dg_m_grouped_fp8_gemm_nt_contiguous,
    dg_m_grouped_fp8_gemm_nt_masked,
    dg_m_grouped_gather,
    dg_m_grouped_gather_weight_grad,
    dg_m_grouped_layout_contiguous,
    dg_m_grouped_layout_masked,
    dg_m_grouped_rows_bound,
    dg_m_grouped_scatter_fp8_contiguous,
    dg_m_grouped_scatter_fp8_masked,
    dg_route_topk,
    dg_route_topk_backward,
    dg_version,
    load,
)

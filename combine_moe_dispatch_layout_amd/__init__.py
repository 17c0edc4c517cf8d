"""MI355X-native MoE token dispatch-layout / dispatch / combine, the experts' products in between, and the
router, dense product and few-token layer around them.

The work happens in libmoe_ep.so (hand-written HIP for gfx950, C ABI in
include/moe_ep.h); this package is its thin Python binding.  PyTorch is used
only for device memory and streams.
"""
from ._binding import (  # noqa: F401
    EXPORTS, KERNEL_NAMES, LIB_PATH, Context, DispatchBuffers, Handle, Hook, MoeError,
    MOE_BUF_COMBINE_OUT, MOE_BUF_EXPERT_OUT, MOE_BUF_HANDLE_EXPERT_OFFSETS, MOE_BUF_HANDLE_POS,
    MOE_BUF_HANDLE_RANK_OFFSETS, MOE_BUF_HANDLE_RECV_COUNTS, MOE_BUF_HANDLE_RECV_SRC,
    MOE_BUF_HANDLE_SEND_SRC, MOE_BUF_LAYOUT_EXPERT_COUNTS, MOE_BUF_LAYOUT_RANK_COUNTS,
    MOE_BUF_LAYOUT_TOKEN_IN_RANK, MOE_BUF_RECV_ROWS, MOE_BUF_RECV_SCALES, MOE_BUF_SEND_ROWS,
    MOE_BUF_SEND_SCALES, MOE_BUF_WORKSPACE, MOE_ERR_BAD_TOPK, MOE_ERR_CAPACITY,
    MOE_ERR_DEVICE_BOUNDS, MOE_ERR_HANDLE, MOE_ERR_HIP, MOE_ERR_INVALID_ARG, MOE_ERR_NONFINITE,
    MOE_ERR_STALE_LAYOUT, MOE_ERR_UNSUPPORTED, ERR_FLAG_BAD_TOPK, ERR_FLAG_BOUNDS, ERR_FLAG_CAPACITY,
    ERR_FLAG_NONFINITE, ERR_FLAG_STALE, StaticConfig,
    MOE_GRAD_BF16, MOE_GRAD_F32, MOE_KERNEL_EXPERT_BWD_ROWS, MOE_KERNEL_EXPERT_BWD_WEIGHTS, MOE_KERNEL_EXPERT_GEMM,
    MOE_KERNEL_SWIGLU, MOE_KERNEL_SWIGLU_BWD, MOE_MAX_FEATURES, MOE_ROWS_PACKED, MOE_ROWS_RECV,
    MOE_KERNEL_COMBINE, MOE_KERNEL_COMBINE_BWD, MOE_KERNEL_DISPATCH, MOE_KERNEL_DISPATCH_BWD,
    MOE_KERNEL_LAYOUT, MOE_LAYOUT_CONTIGUOUS, MOE_LAYOUT_PADDED_LL, MOE_OK, MOE_QUANT_BF16,
    MOE_QUANT_FP8_E4M3, load_library, make_config, moe_combine, moe_combine_backward, moe_dispatch,
    moe_dispatch_backward, moe_dispatch_layout, moe_dispatch_noalloc, moe_expert_gemm, moe_expert_gemm_backward_rows,
    moe_expert_gemm_backward_weights, moe_expert_gemm_fp8, moe_poll_error, moe_size_hint, moe_swiglu,
    moe_swiglu_backward, moe_swiglu_fp8, prepare_combine, prepare_dispatch, status_str,
    MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_SWIGLU, MOE_KERNEL_LAYER,
    MOE_KERNEL_LINEAR, MOE_KERNEL_LINEAR_BWD, MOE_KERNEL_ROUTE, MOE_KERNEL_ROUTE_BWD, MOE_LAYER_MAX_ROWS, MOE_LOGIT_BF16,
    MOE_LOGIT_F32, MOE_MAX_GROUPS, MOE_OUT_BF16, MOE_OUT_F32, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, moe_layer, moe_layer_fp8,
    moe_linear, moe_linear_backward, moe_linear_backward_workspace, moe_linear_workspace, moe_route, moe_route_backward)

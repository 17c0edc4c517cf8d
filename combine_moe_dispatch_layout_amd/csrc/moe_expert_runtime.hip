// C entry points of the expert products and the gated activation: argument
// checks, the segments of the handle, launches.  Nothing here allocates or
// blocks.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_context.h"
#include "moe_ep.h"
#include "moe_expert.h"

using namespace moe;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool order_ok(int32_t o) { return o == MOE_ROWS_RECV || o == MOE_ROWS_PACKED; }

// The checks that every call shares: context, device, handle, orders.
moe_status check_call(const moe_ctx* ctx, const moe_handle* h, int32_t order_a, int32_t order_b) {
    if (ctx == nullptr || h == nullptr || !on_ctx_device(ctx)) return MOE_ERR_INVALID_ARG;
    if (h->tag != ctx->tag || h->num_tokens < 0 || h->num_tokens > ctx->cfg.max_tokens || h->expert_offsets == nullptr)
        return MOE_ERR_HANDLE;
    return order_ok(order_a) && order_ok(order_b) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

moe_status check_features(int32_t k, int32_t n, int32_t k_multiple) {
    if (k < 1 || n < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_FEATURES || n > MOE_MAX_FEATURES || k % k_multiple != 0 || n % 8 != 0) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// A padded row buffer is addressed through its windows; a packed one, and the
// contiguous layout, through the offsets alone.
bool padded(const moe_ctx* ctx, int32_t order) {
    return ctx->cfg.layout == MOE_LAYOUT_PADDED_LL && order == MOE_ROWS_RECV;
}

Segments segments(moe_ctx* ctx, const moe_handle* h) {
    const moe_config& c = ctx->cfg;
    Segments s;
    s.eoff = h->expert_offsets;
    s.E = c.num_experts;
    // what the handle's tokens can have, as the grids are sized for (at most the buffers' rows)
    s.max_rows = (int32_t)((int64_t)h->num_tokens * c.topk);
    // a low-latency window holds max_tokens rows; the dispatch places no more
    s.seg_cap = c.layout == MOE_LAYOUT_PADDED_LL ? c.max_tokens : INT32_MAX;
    s.cap = ctx->g.cap;
    s.first = (int64_t)c.src_rank * c.max_tokens;
    s.err = ctx->err();
    return s;
}

template <class F>
moe_status timed(moe_ctx* ctx, hipStream_t s, int id, F launch) {
    TimedLaunch tl(ctx, s, id);
    const hipError_t e = launch();
    tl.done();
    return e == hipSuccess ? MOE_OK : e == hipErrorInvalidConfiguration ? MOE_ERR_UNSUPPORTED : MOE_ERR_HIP;
}

moe_status run_gemm(moe_ctx* ctx, const void* rows, const float* row_scales, int32_t rows_order, const void* weights,
                    const float* weight_scales, int32_t K, int32_t N, const moe_handle* handle, void* out,
                    int32_t out_order, bool fp8, void* stream) {
    moe_status st = check_call(ctx, handle, rows_order, out_order);
    if (st != MOE_OK) return st;
    st = check_features(K, N, fp8 ? 128 : 8);
    if (st != MOE_OK) return st;
    if (handle->num_tokens == 0) return MOE_OK;
    if (rows == nullptr || weights == nullptr || out == nullptr || out == rows || out == weights)
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(rows) || !aligned16(weights) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
    if (fp8 && (row_scales == nullptr || weight_scales == nullptr || !aligned4(row_scales) || !aligned4(weight_scales)))
        return MOE_ERR_INVALID_ARG;
    ExpertGemmArgs a = {};
    a.seg = segments(ctx, handle);
    a.p = weights;
    a.q = rows;
    a.p_scales = weight_scales;
    a.q_scales = row_scales;
    a.out = out;
    a.K = K;
    a.N = N;
    a.q_padded = padded(ctx, rows_order);
    a.out_padded = padded(ctx, out_order);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t pairs = (int64_t)handle->num_tokens * ctx->cfg.topk;
    return timed(ctx, s, MOE_KERNEL_EXPERT_GEMM, [&] { return launch_expert_gemm(a, fp8, pairs, s); });
}

moe_status run_swiglu(moe_ctx* ctx, const void* gate_up, const void* grad_out, int32_t I, int32_t order,
                      const moe_handle* handle, void* out, float* scales, bool fp8, bool bwd, void* stream) {
    moe_status st = check_call(ctx, handle, order, order);
    if (st != MOE_OK) return st;
    if (I < 1) return MOE_ERR_INVALID_ARG;
    if (I > MOE_MAX_FEATURES / 2 || I % (fp8 ? 128 : 8) != 0) return MOE_ERR_UNSUPPORTED;
    if (handle->num_tokens == 0) return MOE_OK;
    if (gate_up == nullptr || out == nullptr || (!bwd && out == gate_up) || !aligned16(gate_up) || !aligned16(out))
        return MOE_ERR_INVALID_ARG;
    if (bwd && (grad_out == nullptr || out == grad_out || !aligned16(grad_out))) return MOE_ERR_INVALID_ARG;
    if (fp8 && (scales == nullptr || !aligned4(scales))) return MOE_ERR_INVALID_ARG;
    SwigluArgs a = {};
    a.seg = segments(ctx, handle);
    a.gate_up = static_cast<const uint16_t*>(gate_up);
    a.grad_out = static_cast<const uint16_t*>(grad_out);
    a.out = out;
    a.scales = scales;
    a.I = I;
    a.padded = padded(ctx, order);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t pairs = (int64_t)handle->num_tokens * ctx->cfg.topk;
    return timed(ctx, s, bwd ? MOE_KERNEL_SWIGLU_BWD : MOE_KERNEL_SWIGLU,
                 [&] { return bwd ? launch_swiglu_bwd(a, pairs, s) : launch_swiglu(a, fp8, pairs, s); });
}

}  // namespace

MOE_API moe_status moe_expert_gemm(moe_ctx* ctx, const void* rows, int32_t rows_order, const void* weights,
                                   int32_t in_features, int32_t out_features, const moe_handle* handle, void* out,
                                   int32_t out_order, void* stream) {
    return run_gemm(ctx, rows, nullptr, rows_order, weights, nullptr, in_features, out_features, handle, out, out_order,
                    false, stream);
}

MOE_API moe_status moe_expert_gemm_fp8(moe_ctx* ctx, const void* rows, const float* row_scales, int32_t rows_order,
                                       const void* weights, const float* weight_scales, int32_t in_features,
                                       int32_t out_features, const moe_handle* handle, void* out, int32_t out_order,
                                       void* stream) {
    return run_gemm(ctx, rows, row_scales, rows_order, weights, weight_scales, in_features, out_features, handle, out,
                    out_order, true, stream);
}

MOE_API moe_status moe_expert_gemm_backward_rows(moe_ctx* ctx, const void* grad_out, int32_t out_order,
                                                 const void* weights, int32_t in_features, int32_t out_features,
                                                 const moe_handle* handle, void* grad_rows, int32_t rows_order,
                                                 void* stream) {
    moe_status st = check_call(ctx, handle, rows_order, out_order);
    if (st != MOE_OK) return st;
    st = check_features(in_features, out_features, 8);
    if (st != MOE_OK) return st;
    if (handle->num_tokens == 0) return MOE_OK;
    if (grad_out == nullptr || weights == nullptr || grad_rows == nullptr || grad_rows == grad_out ||
        grad_rows == weights || !aligned16(grad_out) || !aligned16(weights) || !aligned16(grad_rows))
        return MOE_ERR_INVALID_ARG;
    ExpertGemmArgs a = {};
    a.seg = segments(ctx, handle);
    a.p = weights;
    a.q = grad_out;
    a.out = grad_rows;
    a.K = in_features;
    a.N = out_features;
    a.q_padded = padded(ctx, out_order);
    a.out_padded = padded(ctx, rows_order);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t pairs = (int64_t)handle->num_tokens * ctx->cfg.topk;
    return timed(ctx, s, MOE_KERNEL_EXPERT_BWD_ROWS, [&] { return launch_expert_gemm_bwd_rows(a, pairs, s); });
}

MOE_API moe_status moe_expert_gemm_backward_weights(moe_ctx* ctx, const void* grad_out, int32_t out_order,
                                                    const void* rows, int32_t rows_order, int32_t in_features,
                                                    int32_t out_features, const moe_handle* handle, void* grad_weights,
                                                    int32_t grad_type, int32_t accumulate, void* stream) {
    moe_status st = check_call(ctx, handle, rows_order, out_order);
    if (st != MOE_OK) return st;
    st = check_features(in_features, out_features, 8);
    if (st != MOE_OK) return st;
    if ((grad_type != MOE_GRAD_BF16 && grad_type != MOE_GRAD_F32) || (accumulate != 0 && accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    const bool any = handle->num_tokens > 0;
    if (grad_weights == nullptr || !aligned16(grad_weights) || (any && (grad_out == nullptr || rows == nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(grad_out) || !aligned16(rows) || grad_weights == grad_out || grad_weights == rows)
        return MOE_ERR_INVALID_ARG;
    if (!any && accumulate) return MOE_OK;
    ExpertGemmArgs a = {};
    a.seg = segments(ctx, handle);
    a.p = rows;
    a.q = grad_out;
    a.out = grad_weights;
    a.K = in_features;
    a.N = out_features;
    a.p_padded = padded(ctx, rows_order);
    a.q_padded = padded(ctx, out_order);
    a.out_f32 = grad_type == MOE_GRAD_F32;
    a.accumulate = accumulate;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return timed(ctx, s, MOE_KERNEL_EXPERT_BWD_WEIGHTS, [&] { return launch_expert_gemm_bwd_weights(a, s); });
}

MOE_API moe_status moe_swiglu(moe_ctx* ctx, const void* gate_up, int32_t features, int32_t order,
                              const moe_handle* handle, void* out, void* stream) {
    return run_swiglu(ctx, gate_up, nullptr, features, order, handle, out, nullptr, false, false, stream);
}

MOE_API moe_status moe_swiglu_fp8(moe_ctx* ctx, const void* gate_up, int32_t features, int32_t order,
                                  const moe_handle* handle, void* out, float* out_scales, void* stream) {
    return run_swiglu(ctx, gate_up, nullptr, features, order, handle, out, out_scales, true, false, stream);
}

MOE_API moe_status moe_swiglu_backward(moe_ctx* ctx, const void* grad_out, const void* gate_up, int32_t features,
                                       int32_t order, const moe_handle* handle, void* grad_gate_up, void* stream) {
    return run_swiglu(ctx, gate_up, grad_out, features, order, handle, grad_gate_up, nullptr, false, true, stream);
}

// C entry points of the router, the dense product and the layer of a few tokens:
// argument checks and launches.  Nothing here allocates or blocks.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "moe_context.h"
#include "moe_ep.h"
#include "moe_expert.h"
#include "moe_layer.h"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <class F>
moe_status timed(moe_ctx* ctx, hipStream_t s, int id, F launch) {
    TimedLaunch tl(ctx, s, id);
    const hipError_t e = launch();
    tl.done();
    return e == hipSuccess ? MOE_OK : e == hipErrorInvalidConfiguration ? MOE_ERR_UNSUPPORTED : MOE_ERR_HIP;
}

moe_status check_tokens(const moe_ctx* ctx, int32_t T) {
    if (ctx == nullptr || !on_ctx_device(ctx) || T < 0) return MOE_ERR_INVALID_ARG;
    return T > ctx->cfg.max_tokens ? MOE_ERR_CAPACITY : MOE_OK;
}

// ---------------------------------------------------------------- router
moe_status check_router(const moe_config& c, int32_t T, const moe_router* r, const void* logits, int32_t type, int64_t stride) {
    if (r == nullptr || (type != MOE_LOGIT_F32 && type != MOE_LOGIT_BF16) || stride < c.num_experts) return MOE_ERR_INVALID_ARG;
    if ((r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) || (r->normalize != 0 && r->normalize != 1) ||
        !std::isfinite(r->scale))
        return MOE_ERR_INVALID_ARG;
    if (r->groups < 1 || r->topk_groups < 1 || r->topk_groups > r->groups || (r->group_top != 1 && r->group_top != 2))
        return MOE_ERR_INVALID_ARG;
    if (T >= 1 << 26) return MOE_ERR_UNSUPPORTED;   // of 64 lanes each: a launch has fewer than 2^32
    if (r->groups > MOE_MAX_GROUPS || c.num_experts % r->groups != 0) return MOE_ERR_UNSUPPORTED;
    return aligned(logits, type == MOE_LOGIT_F32 ? 4 : 2) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// ---------------------------------------------------------------- dense product
bool act_ok(int32_t act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_SWIGLU; }
bool type_ok(int32_t t) { return t == MOE_OUT_BF16 || t == MOE_OUT_F32; }
int64_t columns(int32_t features, int32_t act) { return (act == MOE_ACT_SWIGLU ? 2 : 1) * (int64_t)features; }

moe_status check_linear(int32_t rows, int32_t K, int32_t F, int32_t act, int32_t type) {
    if (rows < 0 || K < 1 || F < 1 || !act_ok(act) || !type_ok(type)) return MOE_ERR_INVALID_ARG;
    if (K > MOE_MAX_FEATURES || columns(F, act) > MOE_MAX_FEATURES || K % 8 != 0 || F % 8 != 0) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// The backward's workspace: the gradient before the activation, unless grad_out is that already; then sums, of columns and
// after them of products in parts (one after the other, on one stream).
struct BackwardPlan {
    bool own_pre;
    size_t sums, total;
};
BackwardPlan plan_backward(int32_t rows, int32_t K, int32_t F, int32_t act, int32_t type, bool with_bias) {
    const int64_t M = columns(F, act);
    BackwardPlan p;
    p.own_pre = act != MOE_ACT_NONE || type == MOE_OUT_F32;
    p.sums = p.own_pre ? ((size_t)rows * M * 2 + 255) & ~(size_t)255 : 0;
    const int64_t bias = with_bias ? linear_sum_blocks(rows) * M * 4 : 0;
    p.total = p.sums + (size_t)std::max({bias, linear_bwd_workspace(rows, K, M), linear_bwd_workspace(M, K, rows)});
    return p;
}

// ---------------------------------------------------------------- a few tokens
moe_status run_layer(moe_ctx* ctx, const void* x, const int64_t* idx, const float* weights, int32_t T, const void* w1,
                     const float* s1, const void* w2, const float* s2, int32_t I, const void* residual, void* out,
                     void* workspace, bool fp8, void* stream) {
    const moe_status st = check_tokens(ctx, T);
    if (st != MOE_OK) return st;
    const moe_config& c = ctx->cfg;
    if (I < 1) return MOE_ERR_INVALID_ARG;
    const int multiple = fp8 ? 128 : 8;
    if (I > MOE_MAX_FEATURES / 2 || I % multiple != 0 || c.hidden % multiple != 0 || (int64_t)T * c.topk > MOE_LAYER_MAX_ROWS)
        return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    for (const void* p : {x, w1, w2, static_cast<const void*>(out), static_cast<const void*>(workspace)})
        if (p == nullptr || !aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (idx == nullptr || weights == nullptr || !aligned(idx, 8) || !aligned(weights, 4) || !aligned16(residual))
        return MOE_ERR_INVALID_ARG;
    if (fp8 && (s1 == nullptr || s2 == nullptr || !aligned(s1, 4) || !aligned(s2, 4))) return MOE_ERR_INVALID_ARG;
    for (const void* p : {x, w1, w2, static_cast<const void*>(idx), static_cast<const void*>(weights), static_cast<const void*>(workspace)})
        if (out == p) return MOE_ERR_INVALID_ARG;
    for (const void* p : {x, w1, w2, static_cast<const void*>(idx), static_cast<const void*>(weights), residual})
        if (workspace == p) return MOE_ERR_INVALID_ARG;
    LayerArgs a = {};
    a.x = x;
    a.idx = idx;
    a.w = weights;
    a.residual = residual;
    a.w1 = w1;
    a.w2 = w2;
    a.s1 = s1;
    a.s2 = s2;
    a.act = static_cast<uint16_t*>(workspace);
    a.out = out;
    a.err = ctx->err();
    a.T = T;
    a.k = c.topk;
    a.E = c.num_experts;
    a.H = c.hidden;
    a.I = I;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return timed(ctx, s, MOE_KERNEL_LAYER, [&] { return launch_layer(a, fp8, s); });
}

}  // namespace

MOE_API moe_status moe_route(moe_ctx* ctx, const void* logits, int32_t logit_type, int64_t logits_stride, int32_t num_tokens,
                             const moe_router* router, const float* bias, int64_t* topk_idx, float* topk_weights,
                             void* stream) {
    moe_status st = check_tokens(ctx, num_tokens);
    if (st != MOE_OK) return st;
    const moe_config& c = ctx->cfg;
    st = check_router(c, num_tokens, router, logits, logit_type, logits_stride);
    if (st != MOE_OK) return st;
    if (num_tokens == 0) return MOE_OK;
    if (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr || !aligned(bias, 4) || !aligned(topk_idx, 8) ||
        !aligned(topk_weights, 4) || topk_idx == logits || topk_weights == logits || topk_weights == bias ||
        static_cast<const void*>(topk_idx) == bias || static_cast<const void*>(topk_idx) == topk_weights)
        return MOE_ERR_INVALID_ARG;
    RouteArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.idx = topk_idx;
    a.weights = topk_weights;
    a.err = ctx->err();
    a.stride = logits_stride;
    a.T = num_tokens;
    a.E = c.num_experts;
    a.k = c.topk;
    a.groups = router->groups;
    a.keep = router->topk_groups;
    a.top = router->group_top;
    const uint64_t size = (uint64_t)(c.num_experts / router->groups);
    a.group_magic = size > 1 ? (uint32_t)(((1ull << 32) + size - 1) / size) : 0;
    a.group_lanes = 32;
    while (a.group_lanes * router->groups > 64) a.group_lanes /= 2;
    a.sigmoid = router->score == MOE_SCORE_SIGMOID;
    a.normalize = router->normalize;
    a.scale = router->scale;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return timed(ctx, s, MOE_KERNEL_ROUTE, [&] { return launch_route(a, logit_type == MOE_LOGIT_BF16, s); });
}

MOE_API moe_status moe_route_backward(moe_ctx* ctx, const float* grad_weights, const void* logits, int32_t logit_type,
                                      int64_t logits_stride, const int64_t* topk_idx, int32_t num_tokens,
                                      const moe_router* router, float* grad_logits, void* stream) {
    moe_status st = check_tokens(ctx, num_tokens);
    if (st != MOE_OK) return st;
    const moe_config& c = ctx->cfg;
    st = check_router(c, num_tokens, router, logits, logit_type, logits_stride);
    if (st != MOE_OK) return st;
    if (num_tokens == 0) return MOE_OK;
    if (grad_weights == nullptr || logits == nullptr || topk_idx == nullptr || grad_logits == nullptr || grad_logits == logits ||
        grad_logits == grad_weights || static_cast<const void*>(grad_logits) == topk_idx || !aligned(grad_weights, 4) || !aligned(topk_idx, 8) || !aligned(grad_logits, 4))
        return MOE_ERR_INVALID_ARG;
    RouteBwdArgs a = {};
    a.grad = grad_weights;
    a.logits = logits;
    a.idx = topk_idx;
    a.grad_logits = grad_logits;
    a.err = ctx->err();
    a.stride = logits_stride;
    a.T = num_tokens;
    a.E = c.num_experts;
    a.k = c.topk;
    a.sigmoid = router->score == MOE_SCORE_SIGMOID;
    a.normalize = router->normalize;
    a.scale = router->scale;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return timed(ctx, s, MOE_KERNEL_ROUTE_BWD, [&] { return launch_route_bwd(a, logit_type == MOE_LOGIT_BF16, s); });
}

MOE_API moe_status moe_linear(moe_ctx* ctx, const void* x, int32_t num_rows, const void* weights, int32_t in_features,
                              int32_t features, const void* bias, int32_t act, const void* residual, void* out,
                              int32_t out_type, void* pre, void* workspace, void* stream) {
    if (ctx == nullptr || !on_ctx_device(ctx)) return MOE_ERR_INVALID_ARG;
    const moe_status st = check_linear(num_rows, in_features, features, act, out_type);
    if (st != MOE_OK) return st;
    if (!linear_fits(num_rows, columns(features, act))) return MOE_ERR_UNSUPPORTED;
    if (num_rows == 0) return MOE_OK;
    for (const void* p : {x, weights, static_cast<const void*>(out)})
        if (p == nullptr || !aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(bias) || !aligned16(residual) || !aligned16(pre) || !aligned16(workspace)) return MOE_ERR_INVALID_ARG;
    if (workspace == nullptr && linear_workspace(num_rows, in_features, features, act == MOE_ACT_SWIGLU) > 0) return MOE_ERR_INVALID_ARG;
    if (workspace != nullptr)
        for (const void* p : {x, weights, bias, residual, static_cast<const void*>(out), static_cast<const void*>(pre)})
            if (workspace == p) return MOE_ERR_INVALID_ARG;
    if (out == x || out == weights || out == bias || (out == residual && out_type != MOE_OUT_BF16)) return MOE_ERR_INVALID_ARG;
    if (pre != nullptr && (pre == x || pre == weights || pre == bias || pre == residual || pre == out)) return MOE_ERR_INVALID_ARG;
    LinearArgs a = {};
    a.x = x;
    a.w = weights;
    a.bias = static_cast<const uint16_t*>(bias);
    a.residual = static_cast<const uint16_t*>(residual);
    a.out = out;
    a.pre = static_cast<uint16_t*>(pre);
    a.partial = static_cast<float*>(workspace);
    a.T = num_rows;
    a.K = in_features;
    a.F = features;
    a.act = act;
    a.out_f32 = out_type == MOE_OUT_F32;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return timed(ctx, s, MOE_KERNEL_LINEAR, [&] { return launch_linear(a, s); });
}

MOE_API moe_status moe_linear_workspace(int32_t num_rows, int32_t in_features, int32_t features, int32_t act, size_t* bytes) {
    if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
    const moe_status st = check_linear(num_rows, in_features, features, act, MOE_OUT_BF16);
    if (st != MOE_OK) return st;
    if (!linear_fits(num_rows, columns(features, act))) return MOE_ERR_UNSUPPORTED;
    *bytes = (size_t)linear_workspace(num_rows, in_features, features, act == MOE_ACT_SWIGLU);
    return MOE_OK;
}

MOE_API moe_status moe_linear_backward_workspace(int32_t num_rows, int32_t in_features, int32_t features, int32_t act,
                                                 int32_t out_type, int32_t with_bias, size_t* bytes) {
    if (bytes == nullptr || (with_bias != 0 && with_bias != 1)) return MOE_ERR_INVALID_ARG;
    const moe_status st = check_linear(num_rows, in_features, features, act, out_type);
    if (st != MOE_OK) return st;
    if (!linear_bwd_fits(num_rows, features)) return MOE_ERR_UNSUPPORTED;
    *bytes = plan_backward(num_rows, in_features, features, act, out_type, with_bias != 0).total;
    return MOE_OK;
}

MOE_API moe_status moe_linear_backward(moe_ctx* ctx, const void* grad_out, int32_t out_type, int32_t num_rows, const void* x,
                                       const void* weights, int32_t in_features, int32_t features, int32_t act,
                                       const void* pre, void* grad_x, void* grad_weights, int32_t grad_type,
                                       int32_t accumulate, float* grad_bias, void* workspace, void* stream) {
    if (ctx == nullptr || !on_ctx_device(ctx)) return MOE_ERR_INVALID_ARG;
    const moe_status st = check_linear(num_rows, in_features, features, act, out_type);
    if (st != MOE_OK) return st;
    if (!linear_bwd_fits(num_rows, features)) return MOE_ERR_UNSUPPORTED;
    if ((grad_type != MOE_GRAD_BF16 && grad_type != MOE_GRAD_F32) || (accumulate != 0 && accumulate != 1)) return MOE_ERR_INVALID_ARG;
    const BackwardPlan plan = plan_backward(num_rows, in_features, features, act, out_type, grad_bias != nullptr);
    const bool any = num_rows > 0;
    for (const void* p : {grad_out, x, weights, pre, static_cast<const void*>(grad_x), static_cast<const void*>(grad_weights),
                          static_cast<const void*>(grad_bias), static_cast<const void*>(workspace)})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (any && (grad_out == nullptr || (act != MOE_ACT_NONE && pre == nullptr) || (grad_x != nullptr && weights == nullptr) ||
                (grad_weights != nullptr && x == nullptr) || (plan.total != 0 && workspace == nullptr)))
        return MOE_ERR_INVALID_ARG;
    const void* results[] = {grad_x, grad_weights, grad_bias, workspace};
    for (int i = 0; i < 4; ++i) {
        if (results[i] == nullptr) continue;
        for (const void* p : {grad_out, x, weights, pre})
            if (results[i] == p) return MOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (results[i] == results[j]) return MOE_ERR_INVALID_ARG;
    }
    if (!any && accumulate) return MOE_OK;
    const int32_t M = (int32_t)columns(features, act);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    LinearGradArgs g = {};
    g.grad = grad_out;
    g.pre = static_cast<const uint16_t*>(pre);
    // (the bias alone does not need it)
    if (plan.own_pre && (grad_x != nullptr || grad_weights != nullptr)) g.grad_pre = static_cast<uint16_t*>(workspace);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.sums);
    if (linear_sum_blocks(num_rows) > 0) g.partial = sums;
    g.grad_bias = grad_bias;
    g.T = num_rows;
    g.F = features;
    g.act = act;
    g.grad_f32 = out_type == MOE_OUT_F32;
    g.accumulate = accumulate;
    const void* d = plan.own_pre ? static_cast<const void*>(g.grad_pre) : grad_out;
    ExpertGemmArgs e = {};   // of one matrix that every row belongs to
    e.seg.E = 1;
    e.seg.max_rows = num_rows;
    e.seg.seg_cap = INT32_MAX;
    e.seg.err = ctx->err();
    e.q = d;
    e.K = in_features;
    e.N = M;
    // grad_x [rows, K] over M, or grad_weights [M, K] over the rows
    auto product = [&](const void* p, void* out, int32_t R, int32_t X, bool weights) {
        if (linear_bwd_here(R, in_features))
            return launch_linear_bwd(LinearBwdArgs{p, d, out, sums, R, in_features, X, weights && grad_type == MOE_GRAD_F32, weights && accumulate},
                                     weights, s);
        e.p = p;
        e.out = out;
        if (!weights) return launch_expert_gemm_bwd_rows(e, num_rows, s);
        e.out_f32 = grad_type == MOE_GRAD_F32;
        e.accumulate = accumulate;
        return launch_expert_gemm_bwd_weights(e, s);
    };
    return timed(ctx, s, MOE_KERNEL_LINEAR_BWD, [&] {
        hipError_t st = hipSuccess;
        if (g.grad_pre != nullptr || grad_bias != nullptr) st = launch_linear_grad(g, s);
        if (st == hipSuccess && grad_x != nullptr && any) st = product(weights, grad_x, num_rows, M, false);
        if (st == hipSuccess && grad_weights != nullptr) st = product(x, grad_weights, M, num_rows, true);
        return st;
    });
}

MOE_API moe_status moe_layer(moe_ctx* ctx, const void* x, const int64_t* topk_idx, const float* topk_weights, int32_t num_tokens,
                             const void* w1, const void* w2, int32_t features, const void* residual, void* out,
                             void* workspace, void* stream) {
    return run_layer(ctx, x, topk_idx, topk_weights, num_tokens, w1, nullptr, w2, nullptr, features, residual, out, workspace,
                     false, stream);
}

MOE_API moe_status moe_layer_fp8(moe_ctx* ctx, const void* x, const int64_t* topk_idx, const float* topk_weights,
                                 int32_t num_tokens, const void* w1, const float* w1_scales, const void* w2,
                                 const float* w2_scales, int32_t features, const void* residual, void* out, void* workspace,
                                 void* stream) {
    return run_layer(ctx, x, topk_idx, topk_weights, num_tokens, w1, w1_scales, w2, w2_scales, features, residual, out,
                     workspace, true, stream);
}

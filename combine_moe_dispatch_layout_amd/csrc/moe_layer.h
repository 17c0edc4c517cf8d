// Internal declarations of the router, the dense product and the layer of a few
// tokens, shared by their kernels (moe_route_kernels.hip, moe_linear_kernels.hip,
// moe_layer_kernels.hip) and their host entry points (moe_layer_runtime.hip).  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct RouteArgs {
    const void* logits;        // [T, stride], E columns of them
    const float* bias;         // [E], nullable
    int64_t* idx;              // [T, k]
    float* weights;            // [T, k]
    uint32_t* err;
    int64_t stride;
    int32_t T, E, k;
    int32_t groups, keep, top; // groups of E / groups experts, how many stay, scores that make a group's
    uint32_t group_magic;      // ceil(2^32 / (E / groups)), 0 for groups of one expert
    int32_t group_lanes;       // the largest power of two of lanes that each group can have, at most 32
    int32_t sigmoid, normalize;
    float scale;
};

struct RouteBwdArgs {
    const float* grad;         // [T, k]
    const void* logits;        // [T, stride]
    const int64_t* idx;        // [T, k]
    float* grad_logits;        // [T, E]
    uint32_t* err;
    int64_t stride;
    int32_t T, E, k;
    int32_t sigmoid, normalize;
    float scale;
};

struct LayerArgs {
    const void* x;             // bf16 [T, H]
    const int64_t* idx;        // [T, k]
    const float* w;            // [T, k]
    const void* residual;      // bf16 [T, H], nullable
    const void *w1, *w2;       // [E, 2I, H] and [E, H, I], bf16 or E4M3 codes
    const float *s1, *s2;      // E4M3: a scale for each 128 x 128 block
    uint16_t* act;             // workspace, bf16 [T * k, I]
    void* out;                 // bf16 [T, H]
    uint32_t* err;
    int32_t T, k, E, H, I;
    int32_t split;             // of the second product's contraction
};

struct LinearArgs {
    const void* x;             // bf16 [T, K]
    const void* w;             // bf16 [M, K]; M = F, or 2F for a gated activation
    const uint16_t* bias;      // bf16 [M], nullable
    const uint16_t* residual;  // bf16 [T, F], nullable
    void* out;                 // [T, F]
    uint16_t* pre;             // bf16 [T, M], nullable
    float* partial;            // workspace: [split, T, M] sums
    int32_t T, K, F;
    int32_t act, out_f32;
};

// The products of the backward pass: D[r][c] = sum over x of P(c, x) Q(r, x), c along the rows of the output.
struct LinearBwdArgs {
    const void* p;             // weights [X, C] (grad_x), x [X, C] (grad_weights)
    const void* q;             // grad [R, X] (grad_x), grad [X, R] (grad_weights)
    void* out;                 // [R, C]
    float* partial;            // workspace: [split, R, C] sums
    int32_t R, C, X;
    int32_t out_f32, accumulate;
};

struct LinearGradArgs {
    const void* grad;          // [T, F]
    const uint16_t* pre;       // bf16 [T, M]; not read without an activation
    uint16_t* grad_pre;        // bf16 [T, M], nullable
    float* partial;            // [linear_sum_blocks(), M] sums of columns, where grad_bias is wanted; NULL for none
    float* grad_bias;          // [M], nullable
    int32_t T, F;
    int32_t act, grad_f32, accumulate;
};

hipError_t launch_layer(const LayerArgs& a, bool fp8, hipStream_t s);
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);
// Whether one launch has enough workgroups.
bool linear_fits(int64_t T, int64_t M);
bool linear_bwd_fits(int64_t T, int64_t F);
int64_t linear_workspace(int64_t T, int64_t K, int64_t F, bool gated);   // bytes
// The backward's products where linear_bwd_here() says so; the others are the expert products' gradients.
bool linear_bwd_here(int64_t R, int64_t C);
hipError_t launch_linear_bwd(const LinearBwdArgs& a, bool weights, hipStream_t s);
int64_t linear_bwd_workspace(int64_t R, int64_t C, int64_t X);           // bytes
// The gradient before the activation, and the bias's from linear_sum_blocks() rows of partial sums.
int64_t linear_sum_blocks(int64_t T);   // 0 where one workgroup has all rows
hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t s);
hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t s);
hipError_t launch_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t s);

}  // namespace moe

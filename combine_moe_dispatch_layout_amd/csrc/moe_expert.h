// Internal declarations of the expert products and the gated activation,
// shared by the kernels (moe_expert_kernels.hip, moe_swiglu_kernels.hip) and
// their host entry points (moe_expert_runtime.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Where an expert's rows stand.  Expert e has eoff[e+1] - eoff[e] rows, at most
// seg_cap of them placed; they start at row eoff[e] of a packed buffer and at
// row e * cap + first of a padded one.
struct Segments {
    const int32_t* eoff;   // [E+1], the handle's expert offsets
    int32_t E;
    int32_t max_rows;      // eoff[E] may not exceed it
    int32_t seg_cap;
    int64_t cap, first;    // padded layout
    uint32_t* err;

    // Offsets of an expert's rows, [lo, hi): they ascend, inside the packed rows.
    __device__ __forceinline__ bool ascending(int lo, int hi) const { return lo >= 0 && hi >= lo && hi <= max_rows; }
};

// One product D[j][i] = sum_c P(i, c) Q(j, c) for each expert; i runs along the
// contiguous dimension of the output.
struct ExpertGemmArgs {
    Segments seg;
    const void* p;            // forward and backward_rows: weights [E, N, K]; backward_weights: rows
    const void* q;            // rows / grad_out rows; backward_weights: grad_out rows
    const float* p_scales;    // fp8: [E, ceil(N/128), K/128]
    const float* q_scales;    // fp8: [rows, K/128]
    void* out;
    int32_t K, N;             // the matrices are [N, K]
    int32_t p_padded, q_padded, out_padded;   // row buffers in the padded receive layout
    int32_t out_f32, accumulate;              // backward_weights
};

struct SwigluArgs {
    Segments seg;
    const uint16_t* gate_up;   // bf16 [rows, 2I]
    const uint16_t* grad_out;  // bf16 [rows, I] (backward)
    void* out;                 // bf16 or E4M3 [rows, I]; backward: bf16 [rows, 2I]
    float* scales;             // fp8: [rows, I/128]
    int32_t I;
    int32_t padded;
};

// pairs: tokens times slots, as many rows as the segments can have (host, from the token count).
hipError_t launch_expert_gemm(const ExpertGemmArgs& a, bool fp8, int64_t pairs, hipStream_t s);
hipError_t launch_expert_gemm_bwd_rows(const ExpertGemmArgs& a, int64_t pairs, hipStream_t s);
hipError_t launch_expert_gemm_bwd_weights(const ExpertGemmArgs& a, hipStream_t s);
hipError_t launch_swiglu(const SwigluArgs& a, bool fp8, int64_t pairs, hipStream_t s);
hipError_t launch_swiglu_bwd(const SwigluArgs& a, int64_t pairs, hipStream_t s);

}  // namespace moe

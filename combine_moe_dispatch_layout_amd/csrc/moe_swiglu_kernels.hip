// The gated activation between the experts' products, and its gradient:
//   act = silu(gate) * up,  silu(g) = g s,  s = 1 / (1 + e^-g)
//   d gate = d act * up * s (1 + g (1 - s)),  d up = d act * g s
// over the valid rows of a row buffer, as bf16 or as E4M3 codes with one scale
// for each 128 channels (the FP8 dispatch's row format, so that the fp8 product
// reads them).  Everything is computed in binary32 and rounded once.
//
// Bound by memory: each input is read once and each output written once, 16
// bytes a lane; one wavefront handles 512 channels, of one row or of several.
// 32,768 rows of 2048 channels take 71 us (5.7 TB/s, where a large copy does 4.8),
// the gradient of 49,152 rows 176 us (5.7 TB/s); 1,024 packed rows as E4M3 take 5 us,
// a launch's latency.
#include "moe_expert.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kSlice = 512;   // channels of a work item: 64 lanes x 8

__device__ __forceinline__ void unpack(const u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {   // round to nearest even
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16);
}

__device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    return u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// Buffer row of packed row r, or -1 if it was not placed.  Where windows bound
// the segments, the expert is the last one whose offset is at most r, found
// with one load per lane over every per-th offset and one over the run in
// between.
__device__ __forceinline__ int64_t row_of(const Segments& s, int r, bool padded) {
    if (s.seg_cap == INT32_MAX) return r;
    const int lane = threadIdx.x & 63;
    const int per = (s.E + 63) / 64;
    const uint64_t at_most = __ballot(lane * per < s.E && s.eoff[min(lane * per, s.E)] <= r);
    const int run = (at_most ? 63 - __clzll((long long)at_most) : 0) * per;
    const int e = run + lane;
    const int off = lane < per && e < s.E ? s.eoff[e] : INT32_MAX;
    const uint64_t in_run = __ballot(off <= r);
    const int l = in_run ? 63 - __clzll((long long)in_run) : 0;
    const int within = r - __builtin_amdgcn_readlane(off, l);
    if (within < 0 || within >= s.seg_cap) return -1;
    return padded ? (int64_t)(run + l) * s.cap + s.first + within : r;
}

// Rows of all segments; none if the offsets cannot be right.
__device__ __forceinline__ int total_rows(const Segments& s) {
    const int n = s.eoff[s.E];
    return n >= 0 && n <= s.max_rows ? n : 0;
}

// Reports offsets that do not ascend.  One workgroup of the launch does it for all: every row is computed alike, so
// nobody else needs more than the total.
__device__ __forceinline__ void check_offsets(const Segments& s) {
    bool right = true;
    for (int e = threadIdx.x; e < s.E; e += kThreads) right &= s.ascending(s.eoff[e], s.eoff[e + 1]);
    if (!right) atomicOr(s.err, kErrBounds);
}

enum Mode { kBf16, kFp8, kBackward };

// FLAT: a wavefront takes 64 consecutive runs of eight channels, also of several rows (every row is where its
// number says).  Otherwise 512 channels of one row, which is looked up once for the wavefront.
template <int MODE, bool FLAT>
__global__ __launch_bounds__(kThreads) void k_swiglu(SwigluArgs a) {
    const int workers = gridDim.x - 1;
    if ((int)blockIdx.x == workers) return check_offsets(a.seg);
    const int lane = threadIdx.x & 63;
    const int slices = (a.I + kSlice - 1) / kSlice, runs = a.I / 8;
    const int rows = total_rows(a.seg);
    const int64_t items = FLAT ? ((int64_t)rows * runs + 63) / 64 : (int64_t)rows * slices;
    const int64_t step = (int64_t)workers * (kThreads / 64);
    for (int64_t it = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         it < items; it += step) {
        int64_t row;
        int c;
        if constexpr (FLAT) {
            const int64_t r = it * 64 / runs;
            const uint32_t run = (uint32_t)(it * 64 - r * runs) + lane, next = run / (uint32_t)runs;
            row = r + next;
            c = (int)(run - next * runs) * 8;
            if (row >= rows) continue;
        } else {
            const int r = (int)(it / slices);
            row = row_of(a.seg, r, a.padded);
            if (row < 0) continue;
            c = (int)(it - (int64_t)r * slices) * kSlice + lane * 8;
            if (c >= a.I) continue;
        }
        const uint16_t* in = a.gate_up + row * 2 * a.I + c;
        float g[8], u[8], v[8];
        unpack(*reinterpret_cast<const u32x4*>(in), g);
        unpack(*reinterpret_cast<const u32x4*>(in + a.I), u);
        if constexpr (MODE == kBackward) {
            float d[8], w[8];
            unpack(*reinterpret_cast<const u32x4*>(a.grad_out + row * a.I + c), d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid(g[i]);
                v[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
                w[i] = d[i] * (g[i] * s);
            }
            uint16_t* out = static_cast<uint16_t*>(a.out) + row * 2 * a.I + c;
            *reinterpret_cast<u32x4*>(out) = pack(v);
            *reinterpret_cast<u32x4*>(out + a.I) = pack(w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = g[i] * sigmoid(g[i]) * u[i];
            if constexpr (MODE == kBf16) {
                *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + row * a.I + c) = pack(v);
            } else {
                // the 16 lanes of a 128-channel block share its maximum; blocks are whole: I is a multiple of 128
                float m = 0.0f;
                bool finite = true;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m = fmaxf(m, fabsf(v[i]));
                    finite &= fabsf(v[i]) < __builtin_inff();
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
                if (!finite) atomicOr(a.seg.err, kErrNonFinite);
                const float ap = fmaxf(m, 1e-4f), sc = 448.0f / ap;
                int lo = 0, hi = 0;
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * sc, v[1] * sc, lo, false);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * sc, v[3] * sc, lo, true);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * sc, v[5] * sc, hi, false);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * sc, v[7] * sc, hi, true);
                *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.out) + row * a.I + c) =
                    u32x2{(uint32_t)lo, (uint32_t)hi};
                if ((lane & 15) == 0) a.scales[row * (a.I / 128) + c / 128] = ap / 448.0f;
            }
        }
    }
}

template <int MODE>
hipError_t launch(const SwigluArgs& a, int64_t pairs, hipStream_t s) {
    // Contiguous rows, us, flat and not: 49,152 x 256 forward 16 and 23, backward 22 and 31; 32,768 x 744 27 and 30, 40
    // and 46; whole slices, 32,768 x 2048 forward 82 and 77, fp8 84 and 79, backward 123 and 125.
    const bool flat = a.seg.seg_cap == INT32_MAX && (MODE == kBackward || a.I % kSlice != 0);
    const int64_t items = flat ? (pairs * (a.I / 8) + 63) / 64 : pairs * ((a.I + kSlice - 1) / kSlice);
    const int64_t blocks = (items + kThreads / 64 - 1) / (kThreads / 64);
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20) + 1);   // the last one checks the offsets
    if (flat) k_swiglu<MODE, true><<<grid, dim3(kThreads), 0, s>>>(a);
    else k_swiglu<MODE, false><<<grid, dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, bool fp8, int64_t pairs, hipStream_t s) {
    return fp8 ? launch<kFp8>(a, pairs, s) : launch<kBf16>(a, pairs, s);
}

hipError_t launch_swiglu_bwd(const SwigluArgs& a, int64_t pairs, hipStream_t s) { return launch<kBackward>(a, pairs, s); }

}  // namespace moe

// The dense product with its epilogue, out = act(x W^T + bias) + residual, and
// what its backward pass needs beside two products: the gradient before the activation
// and the sums of its columns.
//
// Products are exact and added in binary32; the epilogue works on those sums in binary32 and
// rounds once.  A gated activation takes a gate's column and its up column in the same tile.
#include "moe_ep.h"
#include "moe_internal.h"
#include "moe_layer.h"
#include "moe_tiles.h"

namespace moe {
namespace {

__device__ __forceinline__ void unpack8(const u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
    const u32x2 lo = bf16_pack(f32x4{f[0], f[1], f[2], f[3]}), hi = bf16_pack(f32x4{f[4], f[5], f[6], f[7]});
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }
constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f, kTanhCubic = 0.044715f;   // gelu_tanh: sqrt(2 / pi), and the cube's factor

// (1 + tanh r(v)) / 2 is the sigmoid of 2 r(v)
__device__ __forceinline__ float tanh_gate(float v) { return sigmoid(2.0f * kTanhScale * (v + kTanhCubic * v * v * v)); }

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case MOE_ACT_RELU: return v < 0.0f ? 0.0f : v;   // NaN stays
        case MOE_ACT_SILU: return v * sigmoid(v);
        case MOE_ACT_GELU: return 0.5f * v * erfcf(-v * kSqrtHalf);   // 1 + erf without cancellation
        case MOE_ACT_GELU_TANH: return v * tanh_gate(v);
        default: return v;
    }
}
// its derivative
__device__ __forceinline__ float slope(int act, float v) {
    switch (act) {
        case MOE_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
        case MOE_ACT_SILU: {
            const float s = sigmoid(v);
            return s * (1.0f + v * (1.0f - s));
        }
        case MOE_ACT_GELU: return 0.5f * erfcf(-v * kSqrtHalf) + v * expf(-0.5f * v * v) * kInvSqrt2Pi;
        case MOE_ACT_GELU_TANH: {
            const float s = tanh_gate(v), bend = s * (1.0f - s);   // 0 where the square below may be infinite
            return bend == 0.0f ? s : s + v * bend * (2.0f * kTanhScale) * (1.0f + 3.0f * kTanhCubic * v * v);
        }
        default: return 1.0f;
    }
}

// ---------------------------------------------------------------- epilogue
// Eight neighbouring columns of one row, from the sums (gated: the gate's, and the up's) to memory.
template <bool GATED>
__device__ __forceinline__ void finish(const LinearArgs& a, int row, int col, float (&v)[8], float (&u)[8]) {
    if (a.bias != nullptr) {
        float b[8];
        unpack8(*reinterpret_cast<const u32x4*>(a.bias + col), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
        if constexpr (GATED) {
            unpack8(*reinterpret_cast<const u32x4*>(a.bias + a.F + col), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] += b[i];
        }
    }
    if (a.pre != nullptr) {
        uint16_t* pre = a.pre + (int64_t)row * (GATED ? 2 * a.F : a.F) + col;
        *reinterpret_cast<u32x4*>(pre) = pack8(v);
        if constexpr (GATED) *reinterpret_cast<u32x4*>(pre + a.F) = pack8(u);
    }
    if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate(a.act, v[i]);
    }
    const int64_t at = (int64_t)row * a.F + col;
    if (a.residual != nullptr) {
        float r[8];
        unpack8(*reinterpret_cast<const u32x4*>(a.residual + at), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    if (a.out_f32) {
        f32x4* out = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at);
        out[0] = f32x4{v[0], v[1], v[2], v[3]};
        out[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + at) = pack8(v);
    }
}

// ---------------------------------------------------------------- operands in registers
// PS x QS subtiles (gated: half of the PS are gates) for a workgroup whose NW wavefronts share out the contraction: every
// operand byte of the tile is read once, and nothing is waited for but a wavefront's own loads.  Their sums meet in LDS
// and are added in the order of the wavefronts.
template <int PS, int QS, bool GATED, int NW, int AHEAD>
__global__ __launch_bounds__(64 * NW) void k_linear_split(LinearArgs a) {
    constexpr int NP = GATED ? 2 : 1, kCols = PS / NP * 16, kRows = QS * 16;
    __shared__ f32x4 part[NW][PS][QS][64];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, t = lane & 15;
    const int ni = (a.F + kCols - 1) / kCols, nj = (a.T + kRows - 1) / kRows;
    const int tile = xcd_tile4((int)blockIdx.x);
    if (tile >= ni * nj) return;
    int ti, tj;
    band_order(tile, nj, ni, &tj, &ti);
    const int i0 = ti * kCols, j0 = tj * kRows, rows = min(kRows, a.T - j0);
    Direct<false, PS, QS, NP> d;
    d.ld = a.K * 2;
#pragma unroll
    for (int h = 0; h < NP; ++h)
        d.rp[h] = descriptor(static_cast<const char*>(a.w) + (int64_t)(h * a.F + i0) * d.ld, min(kCols, a.F - i0) * d.ld);
    d.rq = descriptor(static_cast<const char*>(a.x) + (int64_t)j0 * d.ld, rows * d.ld);
#pragma unroll
    for (int q = 0; q < QS; ++q) d.row[q] = (uint32_t)((q * 16 + t) * d.ld);   // past the last row: past the descriptor
    f32x4 acc[PS][QS];
    d.template run<AHEAD>(acc, w, NW, (d.ld + kStepBytes - 1) / kStepBytes, lane);
#pragma unroll
    for (int p = 0; p < PS; ++p)
#pragma unroll
        for (int q = 0; q < QS; ++q) part[w][p][q][lane] = acc[p][q];
    __syncthreads();
    for (int item = threadIdx.x; item < kRows * kCols / 8; item += 64 * NW) {
        const int r = item / (kCols / 8), c = item % (kCols / 8);
        if (r >= rows || i0 + 8 * c >= a.F) continue;
        float v[NP][8];
#pragma unroll
        for (int h = 0; h < NP; ++h) {
            const f32x4* from = &part[0][h * (PS / NP) + c / 2][r / 16][(c & 1) * 32 + (r & 15)];
            f32x4 lo = from[0], hi = from[16];
#pragma unroll
            for (int k = 1; k < NW; ++k) {
                lo += from[k * PS * QS * 64];
                hi += from[k * PS * QS * 64 + 16];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[h][i] = lo[i];
                v[h][i + 4] = hi[i];
            }
        }
        finish<GATED>(a, j0 + r, i0 + 8 * c, v[0], v[NP - 1]);
    }
}

// ---------------------------------------------------------------- large tiles
constexpr int kWaves = 8;
constexpr int kTileBytes = kTileP * kStepBytes;

// LoadKC of a tile whose subtiles of 16 matrix rows are a gate's and an up's in turn, each from a panel of its own.
struct LoadGated {
    static constexpr int kInstr = 4;   // of 256 rows and 8 wavefronts: two load gates, two ups
    const char* base[2];
    int bytes, kbytes;
    uint32_t voff[2], chunk;
    int lds;
    __device__ __forceinline__ void init(const void* gate, const void* up, int ld, int valid, int w, int lane) {
        base[0] = static_cast<const char*>(gate);
        base[1] = static_cast<const char*>(up);
        bytes = valid * ld;
        kbytes = ld;
        chunk = ((lane & 7) ^ (lane >> 3)) * 16;
        lds = w * kInstr * 1024;
#pragma unroll
        for (int i = 0; i < 2; ++i) voff[i] = (uint32_t)((w * 16 + i * 8 + (lane >> 3)) * ld) + chunk;
    }
    struct Step {
        __amdgpu_buffer_rsrc_t rsrc[2];
        int left;
    };
    __device__ __forceinline__ Step step_of(int step) const {
        const int at = step * kStepBytes, n = at < kbytes ? bytes - at : 0;
        return Step{{descriptor(base[0] + at, n), descriptor(base[1] + at, n)}, kbytes - at};
    }
    __device__ __forceinline__ void issue(char* stage, const Step& st, int i) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rsrc[i >> 1], LDS_PTR(void, stage + (lds + i * 1024)), 16,
                                                 (int)chunk < st.left ? voff[i & 1] : kOob, 0, 0, 0);
    }
};

template <int BQ, int WP, int STAGES, bool GATED>
__device__ __forceinline__ void wide_tile(const LinearArgs& a, int i0, int j0, int rows, const Stage (&st)[STAGES], char* scratch,
                                          int w, int lane) {
    using B = TileBody<kWaves, BQ, WP, STAGES, false, false, false>;
    static_assert(B::PS % 4 == 0, "");
    const int ld = a.K * 2;
    typename B::LQ lq;
    lq.init(static_cast<const char*>(a.x) + (int64_t)j0 * ld, ld, rows, ld, w, lane);
    LoadScales none;   // bf16 has none
    const Steps steps = {(ld + kStepBytes - 1) / kStepBytes, 0};
    f32x4 acc[B::PS][B::QS];
    if constexpr (GATED) {
        const char* gate = static_cast<const char*>(a.w) + (int64_t)i0 * ld;
        LoadGated lp;
        lp.init(gate, gate + (int64_t)a.F * ld, ld, min(kTileP / 2, a.F - i0), w, lane);
        B::begin(st, lp, lq, none, steps);
        B::run(st, lp, lq, none, steps, acc, w, lane);
    } else {
        typename B::LP lp;
        lp.init(static_cast<const char*>(a.w) + (int64_t)i0 * ld, ld, min(kTileP, a.F - i0), ld, w, lane);
        B::begin(st, lp, lq, none, steps);
        B::run(st, lp, lq, none, steps, acc, w, lane);
    }
    lds_barrier();   // the epilogue's LDS was a stage
    // A wavefront's 16 rows of 64 columns at a time go through LDS, so that a lane has eight neighbouring columns of one
    // row.  A row's 16-byte chunk c sits at c ^ row.
    const int wp = w % WP, wq = w / WP, g = lane >> 4, t = lane & 15;
    char* mine = scratch + w * 4096;
    auto chunk = [&](int r, int c) { return *reinterpret_cast<const f32x4*>(mine + r * 256 + ((c ^ r) << 4)); };
#pragma unroll
    for (int q = 0; q < B::QS; ++q) {
#pragma unroll
        for (int p0 = 0; p0 < B::PS; p0 += 4) {
#pragma unroll
            for (int p = 0; p < 4; ++p) *reinterpret_cast<f32x4*>(mine + t * 256 + (((4 * p + g) ^ t) << 4)) = acc[p0 + p][q];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
            for (int k = 0; k < (GATED ? 1 : 2); ++k) {
                const int r = GATED ? lane >> 2 : k * 8 + (lane >> 3), c = GATED ? lane & 3 : lane & 7;
                const int at = GATED ? (c >> 1) * 8 + (c & 1) * 2 : 2 * c;
                const int row = wq * B::QS * 16 + q * 16 + r;
                const int col = i0 + (wp * B::PS + p0) * (GATED ? 8 : 16) + 8 * c;
                const f32x4 lo = chunk(r, at), hi = chunk(r, at + 1);
                float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, u[8];
                if constexpr (GATED) {
                    const f32x4 ul = chunk(r, at + 4), uh = chunk(r, at + 5);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u[i] = ul[i];
                        u[i + 4] = uh[i];
                    }
                }
                if (row < rows && col < a.F) finish<GATED>(a, j0 + row, col, v, u);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        }
    }
}

// 256 rows x 256 columns (gated: 128 of each).
template <bool GATED>
__global__ __launch_bounds__(64 * kWaves, kWaves / 4) void k_linear(LinearArgs a) {
    constexpr int kCols = GATED ? kTileP / 2 : kTileP, kQ = 128 * kStepBytes;
    __shared__ __align__(1024) char lds[3 * (kTileBytes + kQ)];
    static_assert(sizeof(lds) >= 4 * kTileBytes, "");
    const Stage two[2] = {{lds, lds + 2 * kTileBytes}, {lds + kTileBytes, lds + 3 * kTileBytes}};
    char* q = lds + 3 * kTileBytes;
    const Stage three[3] = {{lds, q}, {lds + kTileBytes, q + kQ}, {lds + 2 * kTileBytes, q + 2 * kQ}};
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int ni = (a.F + kCols - 1) / kCols, nj = (a.T + 255) / 256;
    const int64_t tile = xcd_tile((int)blockIdx.x);
    if (tile >= (int64_t)ni * nj) return;
    int ti, tj;
    band_order((int)tile, nj, ni, &tj, &ti);
    const int i0 = ti * kCols, j0 = tj * 256, rows = min(256, a.T - j0);
    if (rows > 128) wide_tile<256, 2, 2, GATED>(a, i0, j0, rows, two, lds, w, lane);
    else wide_tile<128, 4, 3, GATED>(a, i0, j0, rows, three, lds, w, lane);
}

// ---------------------------------------------------------------- gradient before the activation
// grad_pre = grad act'(pre), and the sums of its columns over a block of rows (of the binary32 values).  A wavefront
// takes 512 columns of kGradRows rows, eight a lane.
constexpr int kGradRows = 32, kGradSlice = 512;

__device__ __forceinline__ void load_grad(const LinearGradArgs& a, int64_t at, float (&d)[8]) {
    if (a.grad_f32) {
        const f32x4* g = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.grad) + at);
        const f32x4 lo = g[0], hi = g[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = lo[i];
            d[i + 4] = hi[i];
        }
    } else {
        unpack8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.grad) + at), d);
    }
}

template <bool GATED>
__global__ __launch_bounds__(64) void k_linear_grad(LinearGradArgs a) {
    const int slices = (a.F + kGradSlice - 1) / kGradSlice;
    const int block = (int)(blockIdx.x / slices), col = (int)(blockIdx.x - (unsigned)block * slices) * kGradSlice + threadIdx.x * 8;
    if (col >= a.F) return;
    const int first = block * kGradRows, last = min(a.T, first + kGradRows), M = GATED ? 2 * a.F : a.F;
    float sum[GATED ? 2 : 1][8] = {};
    for (int r = first; r < last; ++r) {
        float d[8], v[8];
        load_grad(a, (int64_t)r * a.F + col, d);
        const int64_t at = (int64_t)r * M + col;
        if constexpr (GATED) {
            float u[8];
            unpack8(*reinterpret_cast<const u32x4*>(a.pre + at), v);
            unpack8(*reinterpret_cast<const u32x4*>(a.pre + at + a.F), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid(v[i]);
                const float dg = d[i] * u[i] * (s * (1.0f + v[i] * (1.0f - s))), du = d[i] * (v[i] * s);
                v[i] = dg;
                u[i] = du;
                sum[0][i] += dg;
                sum[1][i] += du;
            }
            if (a.grad_pre != nullptr) {
                *reinterpret_cast<u32x4*>(a.grad_pre + at) = pack8(v);
                *reinterpret_cast<u32x4*>(a.grad_pre + at + a.F) = pack8(u);
            }
        } else {
            if (a.act != MOE_ACT_NONE) {
                unpack8(*reinterpret_cast<const u32x4*>(a.pre + at), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] *= slope(a.act, v[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[0][i] += d[i];
            if (a.grad_pre != nullptr) *reinterpret_cast<u32x4*>(a.grad_pre + at) = pack8(d);
        }
    }
    if (a.grad_bias == nullptr) return;
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        f32x4* to = reinterpret_cast<f32x4*>(a.partial + (int64_t)block * M + h * a.F + col);
        to[0] = f32x4{sum[h][0], sum[h][1], sum[h][2], sum[h][3]};
        to[1] = f32x4{sum[h][4], sum[h][5], sum[h][6], sum[h][7]};
    }
}

// The blocks' sums, added in their order (in binary64: a column may have any number of rows).
__global__ __launch_bounds__(256) void k_linear_bias(const float* partial, int64_t blocks, int M, float* out, int accumulate) {
    __shared__ double part[4][64];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, c = (int)blockIdx.x * 64 + lane;
    double sum = 0.0;
    if (c < M)
        for (int64_t b = w; b < blocks; b += 4) sum += partial[b * M + c];
    part[w][lane] = sum;
    __syncthreads();
    if (w != 0 || c >= M) return;
    sum = part[0][lane] + part[1][lane] + part[2][lane] + part[3][lane];
    out[c] = (float)(accumulate ? sum + out[c] : sum);
}

template <bool GATED>
hipError_t linear(const LinearArgs& a, hipStream_t s) {
    constexpr int NP = GATED ? 2 : 1;
    auto split = [&](auto ps, auto qs, auto nw, auto ahead) {
        constexpr int PS = decltype(ps)::value * NP, QS = decltype(qs)::value, NW = decltype(nw)::value, A = decltype(ahead)::value;
        const int64_t tiles = (int64_t)((a.F + PS / NP * 16 - 1) / (PS / NP * 16)) * ((a.T + QS * 16 - 1) / (QS * 16));
        k_linear_split<PS, QS, GATED, NW, A><<<dim3((unsigned)((tiles + 31) / 32 * 32)), dim3(64 * NW), 0, s>>>(a);
        return hipGetLastError();
    };
    using std::integral_constant;
    const int cols = kTileP / NP;
    const int64_t wide = (int64_t)((a.F + cols - 1) / cols) * ((a.T + 255) / 256);
    if (wide < 128) {
        if (a.T <= 16) return split(integral_constant<int, 1>(), integral_constant<int, 1>(), integral_constant<int, 8>(), integral_constant<int, 4>());
        return split(integral_constant<int, 4 / NP>(), integral_constant<int, 4>(), integral_constant<int, 8>(), integral_constant<int, 2>());
    }
    const int64_t blocks = (wide + 255) / 256 * 256;
    if (blocks * 64 * kWaves >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    k_linear<GATED><<<dim3((unsigned)blocks), dim3(64 * kWaves), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) { return a.act == MOE_ACT_SWIGLU ? linear<true>(a, s) : linear<false>(a, s); }

int64_t linear_sum_blocks(int64_t T, int64_t) { return (T + kGradRows - 1) / kGradRows; }

hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    const bool gated = a.act == MOE_ACT_SWIGLU;
    const int M = gated ? 2 * a.F : a.F;
    const int64_t rows = linear_sum_blocks(a.T, M), blocks = rows * ((a.F + kGradSlice - 1) / kGradSlice);
    if (blocks * 64 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    if (blocks > 0) {
        if (gated) k_linear_grad<true><<<dim3((unsigned)blocks), dim3(64), 0, s>>>(a);
        else k_linear_grad<false><<<dim3((unsigned)blocks), dim3(64), 0, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.grad_bias == nullptr) return e;
    k_linear_bias<<<dim3((unsigned)((M + 63) / 64)), dim3(256), 0, s>>>(a.partial, rows, M, a.grad_bias, a.accumulate);
    return hipGetLastError();
}

}  // namespace moe

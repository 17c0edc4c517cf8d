// The dense product with its epilogue, out = act(x W^T + bias) + residual, and
// what its backward pass needs beside two products: the gradient before the activation
// and the sums of its columns.
//
// Products are exact and added in binary32; the epilogue works on those sums in binary32 and
// rounds once.  A gated activation takes a gate's column and its up column in the same tile.
#include <type_traits>

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
// Exponentials and reciprocals are the hardware's (one step each); an exponent's own rounding is what is left, |v| half
// steps relative.
__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896341f); }
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-v)); }

// The normal distribution below v: with y = |v| / sqrt(2), erfc(y) = exp(-y^2) t P(t), t = 1 / (1 + 0.3 y), P a minimax
// polynomial fitted to erfc(y) exp(y^2) / t, so that the lower tail keeps its relative precision and the density comes along.
// The fit is 2.3e-8 off at most, relative, and 4.7e-7 (eight half steps) as binary32 computes it; the tail has the exponent's
// rounding besides, three half steps of v^2 / 2: below 3/2 v^2 + 20 half steps as a whole.  The library's erfc takes twice as many
// instructions, and made the gradient of gelu bound by them.
struct Normal {
    float below, density;   // density times sqrt(2 pi)
    __device__ __forceinline__ explicit Normal(float v) {
        constexpr float p[] = {0.16918741f, 0.17072384f, 0.14828606f, 0.215108f, -0.09503003f, 0.5482136f, -0.5126702f, 0.48573738f, -0.12955607f};
        density = exp_of(-0.5f * v * v);
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(v), 0.3f * 0.70710678118654752f, 1.0f));
        float q = p[8];
#pragma unroll
        for (int i = 7; i >= 0; --i) q = __builtin_fmaf(q, t, p[i]);
        const float tail = 0.5f * t * q * density;
        below = v < 0.0f ? tail : 1.0f - tail;
    }
};
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f, kTanhCubic = 0.044715f;   // gelu_tanh: sqrt(2 / pi), and the cube's factor

// (1 + tanh r(v)) / 2 is the sigmoid of 2 r(v)
__device__ __forceinline__ float tanh_gate(float v) { return sigmoid(2.0f * kTanhScale * (v + kTanhCubic * v * v * v)); }

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case MOE_ACT_RELU: return v < 0.0f ? 0.0f : v;   // NaN stays
        case MOE_ACT_SILU: return v * sigmoid(v);
        case MOE_ACT_GELU: return v * Normal(v).below;
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
        case MOE_ACT_GELU: {
            const Normal n(v);
            return n.below + v * n.density * kInvSqrt2Pi;
        }
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

// A wavefront's 16 rows of PS subtiles side by side (gated: a gate's and an up's in turn) go through LDS, 1 KB a
// subtile, so that a lane has eight neighbouring columns of one row.  A row's 16-byte chunk c sits at c ^ row.
template <int PS, bool GATED>
__device__ __forceinline__ void leave(const LinearArgs& a, char* mine, const f32x4 (&v)[PS], int row, int last_row, int col, int lane) {
    constexpr int kRow = PS * 64, kMask = PS * 4 - 1, kChunks = PS * 2 / (GATED ? 2 : 1);   // bytes, 16-byte chunks - 1, eights of outputs
    const int g = lane >> 4, t = lane & 15;
    auto at = [&](int r, int c) { return reinterpret_cast<f32x4*>(mine + r * kRow + ((c ^ (r & kMask)) << 4)); };
#pragma unroll
    for (int p = 0; p < PS; ++p) *at(t, 4 * p + g) = v[p];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
    for (int k = 0; k < 16 * kChunks; k += 64) {
        const int r = (k + lane) / kChunks, c = lane % kChunks;
        const int from = GATED ? (c >> 1) * 8 + (c & 1) * 2 : 2 * c;
        if (row + r < last_row && col + 8 * c < a.F && r < 16) {
            const f32x4 lo = *at(r, from), hi = *at(r, from + 1);
            float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, u[8];
            if constexpr (GATED) {
                const f32x4 ul = *at(r, from + 4), uh = *at(r, from + 5);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = ul[i];
                    u[i + 4] = uh[i];
                }
            }
            finish<GATED>(a, row + r, col + 8 * c, x, u);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
}

// ---------------------------------------------------------------- few rows
// 16 columns and up to 16 rows for a workgroup whose NW wavefronts share out the contraction: the matrix goes straight into
// registers, and nothing is waited for but a wavefront's own loads.  Their sums meet in LDS and are added in the order of the
// wavefronts.  Bound by the matrix and a launch: 1 x 2048 -> 7168, 29 MB, 9.3 us, of which 4.7 would be a bare read.
template <bool GATED, int NW, int AHEAD>
__global__ __launch_bounds__(64 * NW) void k_linear_few(LinearArgs a) {
    constexpr int NP = GATED ? 2 : 1;
    using D = Direct<false, NP, NP>;
    __shared__ f32x4 part[NW][NP][64];
    __shared__ __align__(16) char corners[NW][D::kLds];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i0 = (int)blockIdx.x * 16;
    D d;
    d.corner = corners[w];
    d.ld = a.K * 2;
#pragma unroll
    for (int h = 0; h < NP; ++h)
        d.rp[h] = descriptor(static_cast<const char*>(a.w) + (int64_t)(h * a.F + i0) * d.ld, min(16, a.F - i0) * d.ld);
    d.rq = descriptor(a.x, a.T * d.ld);
    d.set_rows(a.T, (uint32_t)((lane & 15) * d.ld), lane);
    bool todo = true;
    d.template stream<AHEAD>(
        [&](int* first, int* stride, int* end) {
            *first = w;
            *stride = NW;
            *end = (d.ld + kStepBytes - 1) / kStepBytes;
            const bool more = todo;
            todo = false;
            return more;
        },
        [&](const f32x4 (&acc)[NP]) {
#pragma unroll
            for (int p = 0; p < NP; ++p) part[w][p][lane] = acc[p];
        },
        lane);
    __syncthreads();
    const int r = threadIdx.x >> 1, c = threadIdx.x & 1;
    if (r >= a.T || i0 + 8 * c >= a.F) return;
    float v[NP][8];
#pragma unroll
    for (int h = 0; h < NP; ++h) {
        f32x4 lo = part[0][h][c * 32 + r], hi = part[0][h][c * 32 + 16 + r];
#pragma unroll
        for (int k = 1; k < NW; ++k) {
            lo += part[k][h][c * 32 + r];
            hi += part[k][h][c * 32 + 16 + r];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[h][i] = lo[i];
            v[h][i + 4] = hi[i];
        }
    }
    finish<GATED>(a, r, i0 + 8 * c, v[0], v[NP - 1]);
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
    __device__ __forceinline__ void init(const char* gate, const char* up, int ld, int valid, int w, int lane) {
        base[0] = gate;
        base[1] = up;
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
    const int wp = w % WP, wq = w / WP;
#pragma unroll
    for (int q = 0; q < B::QS; ++q)
#pragma unroll
        for (int p0 = 0; p0 < B::PS; p0 += 4) {
            const f32x4 v[4] = {acc[p0][q], acc[p0 + 1][q], acc[p0 + 2][q], acc[p0 + 3][q]};
            leave<4, GATED>(a, scratch + w * 4096, v, j0 + wq * B::QS * 16 + q * 16, j0 + rows, i0 + (wp * B::PS + p0) * (GATED ? 8 : 16), lane);
        }
}

// 256 rows x 256 columns (gated: 128 of each).  Bound by the matrix cores at the clock their power allows: 4096 x 7168 -> 2 x 2048,
// gated, 240 GFLOP in 176 us, 1.37 PFLOP/s.
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

// ---------------------------------------------------------------- small tiles
// Which tile of which part of the contraction a workgroup takes.
struct Part {
    int ti, tj, part;
    int first, last, past;   // steps
    __device__ __forceinline__ bool init(int ni, int nj, int steps, int split, int run) {
        const int64_t at = xcd_run_tile((int)blockIdx.x, run), tiles = (int64_t)ni * nj;
        if (at >= tiles * split) return false;
        part = (int)(at / tiles);
        band_order((int)(at - part * tiles), nj, ni, &tj, &ti);
        past = steps;
        first = (int)((int64_t)part * steps / split);
        last = (int)((int64_t)(part + 1) * steps / split);
        return true;
    }
};

// P matrix rows (gated: half of them gates) x Q rows.  Bound by LDS where two workgroups of 128 x 128 share a compute unit, else by
// the latency of its steps (counters beside StagedBody's operands); times beside plan_tiles().
template <int P, int Q, int WP, int WQ, int AHEAD, bool GATED>
__global__ __launch_bounds__(64 * WP * WQ) void k_linear_tile(LinearArgs a, int split, int run) {
    using OpP = typename std::conditional<GATED, StageGated<P, WP * WQ>, StageKC<P, WP * WQ>>::type;
    using OpQ = StageKC<Q, WP * WQ>;
    using B = StagedBody<P, Q, WP, WQ, AHEAD, OpP, OpQ>;
    constexpr int NP = GATED ? 2 : 1, kCols = P / NP;
    __shared__ __align__(1024) char lds[B::kLds];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, ld = a.K * 2;
    Part at;
    if (!at.init((a.F + kCols - 1) / kCols, (a.T + Q - 1) / Q, (ld + kStepBytes - 1) / kStepBytes, split, run)) return;
    const int i0 = at.ti * kCols, j0 = at.tj * Q, rows = min(Q, a.T - j0);
    const char* mat = static_cast<const char*>(a.w) + (int64_t)i0 * ld;
    OpP lp;
    OpQ lq;
    if constexpr (GATED) lp.init(mat, mat + (int64_t)a.F * ld, ld, min(kCols, a.F - i0), w, lane);
    else lp.init(mat, ld, min(kCols, a.F - i0), w, lane);
    lq.init(static_cast<const char*>(a.x) + (int64_t)j0 * ld, ld, rows, w, lane);
    B::run(lds, lp, lq, at.first, at.last, at.past, w, lane);
    for (int item = threadIdx.x; item < Q * kCols / 8; item += 64 * B::kWaves) {
        const int r = item / (kCols / 8), c = item % (kCols / 8), col = i0 + 8 * c;
        if (r >= rows || col >= a.F) continue;
        const int from = GATED ? (c >> 1) * 8 + (c & 1) * 2 : 2 * c;
        f32x4 v[NP][2];
#pragma unroll
        for (int h = 0; h < NP; ++h) {
            v[h][0] = B::sum(lds, r, from + 4 * h);
            v[h][1] = B::sum(lds, r, from + 4 * h + 1);
        }
        if (split > 1) {
            f32x4* to = reinterpret_cast<f32x4*>(a.partial + ((int64_t)at.part * a.T + j0 + r) * (NP * a.F) + col);
#pragma unroll
            for (int h = 0; h < NP; ++h) {
                to[h * (a.F / 4)] = v[h][0];
                to[h * (a.F / 4) + 1] = v[h][1];
            }
        } else {
            float x[NP][8];
#pragma unroll
            for (int h = 0; h < NP; ++h)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[h][i] = v[h][i >> 2][i & 3];
            finish<GATED>(a, j0 + r, col, x[0], x[NP - 1]);
        }
    }
}

// Eight sums of partial results, added in the order of the parts.
__device__ __forceinline__ void add_parts(const float* from, int64_t stride, int split, float (&v)[8]) {
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    for (int s = 0; s < split; ++s) {
        const f32x4* p = reinterpret_cast<const f32x4*>(from + s * stride);
        lo += p[0];
        hi += p[1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[i + 4] = hi[i];
    }
}

// Bound by memory: four parts of 4096 x 256, 21 MB, 4.7 us.
template <bool GATED>
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs a, int split) {
    const int64_t eights = a.F / 8, item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= a.T * eights) return;
    const int row = (int)(item / eights), col = (int)(item - row * eights) * 8, M = GATED ? 2 * a.F : a.F;
    const float* from = a.partial + (int64_t)row * M + col;
    float v[8], u[8];
    add_parts(from, (int64_t)a.T * M, split, v);
    if constexpr (GATED) add_parts(from + a.F, (int64_t)a.T * M, split, u);
    finish<GATED>(a, row, col, v, u);
}

// ---------------------------------------------------------------- products of the backward pass
// Eight neighbouring results at element o of the output.
__device__ __forceinline__ void put8(const LinearBwdArgs& a, int64_t o, float (&v)[8]) {
    if (a.out_f32) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o);
        f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        if (a.accumulate) {
            lo += d[0];
            hi += d[1];
        }
        d[0] = lo;
        d[1] = hi;
    } else {
        u32x4* d = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + o);
        if (a.accumulate) {
            float old[8];
            unpack8(*d, old);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += old[i];
        }
        *d = pack8(v);
    }
}

// WEIGHTS: the contraction runs over rows of both operands; else along the gradient's rows.  Bound as k_linear_tile is; figures
// beside linear_bwd_here().
template <int P, int Q, int WP, int WQ, int AHEAD, bool WEIGHTS>
__global__ __launch_bounds__(64 * WP * WQ) void k_linear_bwd(LinearBwdArgs a, int split, int run) {
    using OpP = StageMC<P, WP * WQ>;
    using OpQ = typename std::conditional<WEIGHTS, StageMC<Q, WP * WQ>, StageKC<Q, WP * WQ>>::type;
    using B = StagedBody<P, Q, WP, WQ, AHEAD, OpP, OpQ>;
    __shared__ __align__(1024) char lds[B::kLds];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    Part at;
    if (!at.init((a.C + P - 1) / P, (a.R + Q - 1) / Q, (a.X + kStepC - 1) / kStepC, split, run)) return;
    const int i0 = at.ti * P, j0 = at.tj * Q, rows = min(Q, a.R - j0);
    OpP lp;
    OpQ lq;
    lp.init(a.p, a.C * 2, a.X, i0, w, lane);
    if constexpr (WEIGHTS) lq.init(a.q, a.R * 2, a.X, j0, w, lane);
    else lq.init(static_cast<const char*>(a.q) + (int64_t)j0 * a.X * 2, a.X * 2, rows, w, lane);
    B::run(lds, lp, lq, at.first, at.last, at.past, w, lane);
    for (int item = threadIdx.x; item < Q * P / 8; item += 64 * B::kWaves) {
        const int r = item / (P / 8), c = item % (P / 8), col = i0 + 8 * c;
        if (r >= rows || col >= a.C) continue;
        const f32x4 lo = B::sum(lds, r, 2 * c), hi = B::sum(lds, r, 2 * c + 1);
        if (split > 1) {
            f32x4* to = reinterpret_cast<f32x4*>(a.partial + ((int64_t)at.part * a.R + j0 + r) * a.C + col);
            to[0] = lo;
            to[1] = hi;
        } else {
            float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            put8(a, (int64_t)(j0 + r) * a.C + col, v);
        }
    }
}

__global__ __launch_bounds__(256) void k_linear_bwd_join(LinearBwdArgs a, int split) {
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)a.R * a.C;
    if (item * 8 >= n) return;
    float v[8];
    add_parts(a.partial + item * 8, n, split, v);
    put8(a, item * 8, v);
}

// ---------------------------------------------------------------- gradient before the activation
// grad_pre = grad act'(pre), and the sums of its columns (of the binary32 values).  grad_pre is rounded once, to bf16 (off by
// at most 2^-8 of its value), also where the gradient comes in binary32: the matrix instruction of both products takes bf16,
// and as a sum of two such numbers it would cost them twice the operations.  A workgroup of 16 wavefronts takes 128 rows of 128
// columns, eight a lane and four rows a wavefront at once; the sums meet in LDS, and go out at once where that is all rows (the
// sums of 128 rows are 1/64 of what a bf16 gradient takes).  Bound by memory: 8192 x 4096, gelu, 201 MB, 43 us, 4.7 TB/s.
// Whole wavefronts on a row of 512 columns are as fast there (1% faster from 16384 x 4096 on) but leave most of the chip idle
// below 256 workgroups, where the time is that of a wavefront's loads one after the other (both products with it, 1024 x 1024 x
// 1024: 39 us against 27).
constexpr int kGradWaves = 16, kGradRows = 128, kGradSlice = 128;
constexpr int kGradLanes = kGradSlice / 8, kGradAtOnce = kGradWaves * (64 / kGradLanes);   // a row's lanes, rows at once

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
__global__ __launch_bounds__(64 * kGradWaves) void k_linear_grad(LinearGradArgs a) {
    constexpr int NP = GATED ? 2 : 1;
    __shared__ f32x4 part[kGradWaves][2][kGradLanes];
    const int slices = (a.F + kGradSlice - 1) / kGradSlice, w = threadIdx.x >> 6, lane = threadIdx.x & (kGradLanes - 1);
    const int block = (int)(blockIdx.x / slices), col = (int)(blockIdx.x - (unsigned)block * slices) * kGradSlice + lane * 8;
    const int M = NP * a.F;
    float sum[NP][8] = {};
    if (col < a.F) {
        for (int i = 0; i < kGradRows / kGradAtOnce; ++i) {
            const int r = block * kGradRows + i * kGradAtOnce + (int)threadIdx.x / kGradLanes;
            if (r >= a.T) break;
            float d[8], v[8];
            load_grad(a, (int64_t)r * a.F + col, d);
            const int64_t at = (int64_t)r * M + col;
            if constexpr (GATED) {
                float u[8];
                unpack8(*reinterpret_cast<const u32x4*>(a.pre + at), v);
                unpack8(*reinterpret_cast<const u32x4*>(a.pre + at + a.F), u);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float s = sigmoid(v[k]);
                    const float dg = d[k] * u[k] * (s * (1.0f + v[k] * (1.0f - s))), du = d[k] * (v[k] * s);
                    v[k] = dg;
                    u[k] = du;
                    sum[0][k] += dg;
                    sum[1][k] += du;
                }
                if (a.grad_pre != nullptr) {
                    *reinterpret_cast<u32x4*>(a.grad_pre + at) = pack8(v);
                    *reinterpret_cast<u32x4*>(a.grad_pre + at + a.F) = pack8(u);
                }
            } else {
                if (a.act != MOE_ACT_NONE) {
                    unpack8(*reinterpret_cast<const u32x4*>(a.pre + at), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) d[k] *= slope(a.act, v[k]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[0][k] += d[k];
                if (a.grad_pre != nullptr) *reinterpret_cast<u32x4*>(a.grad_pre + at) = pack8(d);
            }
        }
    }
    if (a.grad_bias == nullptr) return;
#pragma unroll
    for (int h = 0; h < NP; ++h) {
#pragma unroll
        for (int step = kGradLanes; step < 64; step *= 2)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[h][k] += __shfl_xor(sum[h][k], step, 64);
        if (h > 0) __syncthreads();
        part[w][0][lane] = f32x4{sum[h][0], sum[h][1], sum[h][2], sum[h][3]};
        part[w][1][lane] = f32x4{sum[h][4], sum[h][5], sum[h][6], sum[h][7]};
        __syncthreads();
        if (w < 2 && (int)(threadIdx.x & 63) < kGradLanes && col < a.F) {   // each of two wavefronts half of a lane's eight
            f32x4 v = part[0][w][lane];
#pragma unroll
            for (int i = 1; i < kGradWaves; ++i) v += part[i][w][lane];
            const int64_t at = h * a.F + col + w * 4;
            if (a.partial != nullptr) {
                *reinterpret_cast<f32x4*>(a.partial + (int64_t)block * M + at) = v;
            } else {
                f32x4* out = reinterpret_cast<f32x4*>(a.grad_bias + at);
                *out = a.accumulate ? *out + v : v;
            }
        }
    }
}

// The workgroups' sums, added in their order (in binary64: a column may have any number of rows).
__global__ __launch_bounds__(1024) void k_linear_bias(const float* partial, int blocks, int M, float* out, int accumulate) {
    __shared__ double part[16][64];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, c = (int)blockIdx.x * 64 + lane;
    double sum = 0.0;
    if (c < M)
        for (int b = w; b < blocks; b += 16) sum += partial[(int64_t)b * M + c];
    part[w][lane] = sum;
    __syncthreads();
    if (w != 0 || c >= M) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += part[i][lane];
    out[c] = (float)(accumulate ? sum + out[c] : sum);
}

template <bool GATED, int P, int Q, int WP, int WQ, int AHEAD>
hipError_t launch_tile(const LinearArgs& a, int split, hipStream_t s) {
    constexpr int kCols = GATED ? P / 2 : P;
    const int64_t tiles = (int64_t)((a.F + kCols - 1) / kCols) * ((a.T + Q - 1) / Q) * split;
    const int run = xcd_run(tiles);
    k_linear_tile<P, Q, WP, WQ, AHEAD, GATED><<<dim3((unsigned)xcd_grid(tiles, run)), dim3(64 * WP * WQ), 0, s>>>(a, split, run);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || split == 1) return e;
    k_linear_join<GATED><<<dim3((unsigned)(((int64_t)a.T * (a.F / 8) + 255) / 256)), dim3(256), 0, s>>>(a, split);
    return hipGetLastError();
}

template <bool WEIGHTS, int P, int Q, int WP, int WQ, int AHEAD>
hipError_t launch_bwd(const LinearBwdArgs& a, int split, hipStream_t s) {
    const int64_t tiles = (int64_t)((a.C + P - 1) / P) * ((a.R + Q - 1) / Q) * split;
    const int run = xcd_run(tiles);
    k_linear_bwd<P, Q, WP, WQ, AHEAD, WEIGHTS><<<dim3((unsigned)xcd_grid(tiles, run)), dim3(64 * WP * WQ), 0, s>>>(a, split, run);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || split == 1) return e;
    k_linear_bwd_join<<<dim3((unsigned)(((int64_t)a.R * a.C / 8 + 255) / 256)), dim3(256), 0, s>>>(a, split);
    return hipGetLastError();
}

// ---------------------------------------------------------------- which kernel
// How a product of `rows` x `cols` results over `steps` steps is shared out: tiles of kTileRows x kTileCols, the contraction
// in `split` parts.  The shortest of what they are expected to take, us: the operands at the rate that full compute units take them
// in (12 TB/s, fitted to the times below; what stands behind it is LDS), or the latency of a workgroup's steps; and the partial
// sums' way to memory and back with a second launch.  Measured, cold matrices, us (tile rows x columns / parts; the choice first):
//   4096 x 7168 -> 256     128 x 128 / 4  31   / 1 90    64 x 64 / 1 38
//   8192 x 4096 -> 64      32 x 64 / 1    19             64 x 64 / 1 24
//   1024 x 4096 -> 4096    128 x 128 / 1  44   / 2 54    64 x 64 / 1 67   256 x 256 105
//   512 x 4096 -> 4096     128 x 128 / 2  32   / 1 41    64 x 64 / 1 37
//   333 x 1000 -> 2056     64 x 64 / 1    10   / 2 15    128 x 128 / 1 17
//   64 x 4096 -> 4096      64 x 64 / 4    13   / 1 23    32 x 64 / 2 13.5
//   32 x 4096 -> 4096      32 x 64 / 4    12   / 1 17    64 x 64 / 4 12
//   24 x 7168 -> 256       32 x 64 / 8    10   / 2 16
//   3000 x 4096 -> 4096    256 x 256      104            128 x 128 / 1 111
//   2048 x 4096 -> 4096    128 x 128 / 1  75             256 x 256 105
struct Plan {
    int tile, split;   // kTile128 .., or kWide
    float us;
};
enum { kTile128, kTile64, kTile32, kTiles, kWide };
constexpr int kTileCols[kTiles] = {128, 64, 64}, kTileRows[kTiles] = {128, 64, 32};
constexpr float kStepUs[kTiles] = {0.65f, 0.33f, 0.2f}, kOperandUs = 1.0f / 12e6f, kPartUs = 8.0f / 5e6f, kJoinUs = 4.0f, kWideUs = 1.6f;

constexpr int64_t kMostTiles = (1 << 23) - 256;   // of up to 512 threads: a launch has fewer than 2^32

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// tiles: how many kinds there are.  cols counts matrix rows (a gated product's are twice its results).
Plan plan_tiles(int64_t rows, int64_t cols, int64_t steps, int tiles) {
    Plan best = {kTile64, 1, 1e30f};
    for (int t = 0; t < tiles; ++t) {
        const int64_t n = ceil_div(rows, kTileRows[t]) * ceil_div(cols, kTileCols[t]);
        if (n >= kMostTiles) continue;
        for (int split = 1; split <= 16 && (split == 1 || steps >= 4 * split); split *= 2) {
            const float traffic = (float)n * steps * (kTileCols[t] + kTileRows[t]) * kStepBytes * kOperandUs;
            const float latency = (float)ceil_div(steps, split) * ceil_div(n * split, 512) * kStepUs[t];
            const float us = (traffic > latency ? traffic : latency) + (split > 1 ? kJoinUs + (float)split * rows * cols * kPartUs : 0.0f);
            if (us < best.us) best = Plan{t, split, us};
        }
    }
    return best;
}

// Up to 12 rows whose matrix a workgroup for each 16 columns reads well (1 x 7168 -> 4096 13.2, in tiles 15.2; 12 x 4096 -> 4096 10.4
// and 11.3), or is short (8 x 1024 -> 1024 5.1 and 6.4); not so 4 x 7168 -> 2048 gated (21.6 and 16.1), 8 x 7168 -> 256 (13.4 and
// 9.7) or 16 x 4096 -> 4096.
bool few_rows(int64_t T, int64_t K, int64_t F) { return T <= 12 && (F >= 2560 || K <= 1024); }

Plan plan_linear(int64_t T, int64_t K, int64_t M) {
    const int64_t steps = ceil_div(K * 2, kStepBytes);
    const Plan p = plan_tiles(T, M, steps, kTiles);
    const float wide = (float)ceil_div(ceil_div(M, kTileP) * ceil_div(T, 256), 256) * steps * kWideUs;
    return wide < p.us ? Plan{kWide, 1, wide} : p;
}

template <bool GATED>
hipError_t linear(const LinearArgs& a, hipStream_t s) {
    const int64_t M = GATED ? 2 * (int64_t)a.F : a.F;
    if (few_rows(a.T, a.K, a.F)) {
        k_linear_few<GATED, 4, 8><<<dim3((unsigned)ceil_div(a.F, 16)), dim3(256), 0, s>>>(a);
        return hipGetLastError();
    }
    const Plan p = plan_linear(a.T, a.K, M);
    if (p.tile == kTile128) return launch_tile<GATED, 128, 128, 2, 4, 2>(a, p.split, s);
    if (p.tile == kTile64) return launch_tile<GATED, 64, 64, 2, 2, 4>(a, p.split, s);
    if (p.tile == kTile32) return launch_tile<GATED, 64, 32, 2, 2, 4>(a, p.split, s);
    const int64_t blocks = ceil_div(ceil_div(M, kTileP) * ceil_div(a.T, 256), 256) * 256;
    k_linear<GATED><<<dim3((unsigned)blocks), dim3(64 * kWaves), 0, s>>>(a);
    return hipGetLastError();
}

template <bool WEIGHTS>
hipError_t linear_bwd(const LinearBwdArgs& a, hipStream_t s) {
    const Plan p = plan_tiles(a.R, a.C, ceil_div(a.X, kStepC), kTile32);
    if (p.tile == kTile128) return launch_bwd<WEIGHTS, 128, 128, 2, 4, 2>(a, p.split, s);
    return launch_bwd<WEIGHTS, 64, 64, 2, 2, 4>(a, p.split, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) { return a.act == MOE_ACT_SWIGLU ? linear<true>(a, s) : linear<false>(a, s); }

bool linear_fits(int64_t T, int64_t M) { return ceil_div(M, kTileP) * ceil_div(T, 256) <= kMostTiles; }
bool linear_bwd_fits(int64_t T, int64_t F) { return ceil_div(T, kGradRows) * ceil_div(F, kGradSlice) <= kMostTiles / 2; }

int64_t linear_workspace(int64_t T, int64_t K, int64_t F, bool gated) {
    if (T == 0 || few_rows(T, K, F)) return 0;
    const int64_t M = gated ? 2 * F : F;
    const Plan p = plan_linear(T, K, M);
    return p.split > 1 ? p.split * T * M * 4 : 0;
}

// Up to 320 tiles of 128 x 128; more fill the chip in the expert products' kernels.  grad_x, us, here and there: 1024 rows, 4096 x
// 4096, 43 and 66, 519 rows, 5120 -> 1368 24 and 71, 77 rows, 528 -> 256 6.6 and 9.3; grad_W of 256 x 7168 over 4096 rows 32 and 45, of
// 4096 x 4096 over 1024 44 and 33, over 1 15 and 11, of 5120 x 1368 over 519 19 and 17.
bool linear_bwd_here(int64_t R, int64_t C) { return ceil_div(R, 128) * ceil_div(C, 128) <= 320; }

int64_t linear_bwd_workspace(int64_t R, int64_t C, int64_t X) {
    if (!linear_bwd_here(R, C)) return 0;
    const Plan p = plan_tiles(R, C, ceil_div(X, kStepC), kTile32);
    return p.split > 1 ? p.split * R * C * 4 : 0;
}

hipError_t launch_linear_bwd(const LinearBwdArgs& a, bool weights, hipStream_t s) { return weights ? linear_bwd<true>(a, s) : linear_bwd<false>(a, s); }

int64_t linear_sum_blocks(int64_t T) { return T <= kGradRows ? 0 : ceil_div(T, kGradRows); }

hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    const bool gated = a.act == MOE_ACT_SWIGLU;
    const int M = gated ? 2 * a.F : a.F;
    const int64_t sums = linear_sum_blocks(a.T);
    if (a.T > 0) {
        const unsigned blocks = (unsigned)(ceil_div(a.T, kGradRows) * ceil_div(a.F, kGradSlice));
        if (gated) k_linear_grad<true><<<dim3(blocks), dim3(64 * kGradWaves), 0, s>>>(a);
        else k_linear_grad<false><<<dim3(blocks), dim3(64 * kGradWaves), 0, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.grad_bias == nullptr || (a.T > 0 && sums == 0)) return e;
    k_linear_bias<<<dim3((unsigned)((M + 63) / 64)), dim3(1024), 0, s>>>(a.partial, (int)sums, M, a.grad_bias, a.accumulate);
    return hipGetLastError();
}

}  // namespace moe

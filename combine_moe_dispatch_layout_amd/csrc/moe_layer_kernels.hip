// The experts of a few tokens in two kernels, from the tokens' rows to the sum of
// their experts' outputs:
//   k_layer_up    act[p] = silu(g) u, (g, u) = W1[e] x[t], for every slot p = (t, j) with an expert e
//   k_layer_down  out[t] = residual[t] + sum over j of w[t, j] W2[e] act[p]
// There is no dispatch: each workgroup finds the slots of its expert in topk_idx, and reads the
// tokens' rows where they stand.
//
// Bound by reading the matrices of the experts that are chosen.  Both kernels stream them straight into
// registers, 16 matrix rows by 128 bytes a step, and use each for up to 16 slots; the contraction
// (k_layer_up) or the experts (k_layer_down) are shared out over the wavefronts of a workgroup and
// joined in LDS, in an order that sizes and routing decide.  One token of 6 of 64 experts, 4096 and 2048 wide, bf16:
// 302 MB in 58 us, 5.2 TB/s (a bare read in this pattern 6.2); 128 tokens of 8 of 256, 7168 and 2048, E4M3: 11.2 GB in 2.04 ms,
// 5.4 TB/s (first kernel 1.31, second 0.73; with 16 column tiles a workgroup 2.07, of which the loads of rows and scales 0.26).
// A compute unit's vector cache has about 700 requests of 64 bytes on their way, and the rows' count among them: hence rows
// come in whole lines, through LDS, and no more of them than a tile has.
//
// Sums are binary32; the activations are rounded once, to bf16, because the second product's matrix instruction takes
// bf16.  E4M3 matrices are widened to bf16 exactly, rows and activations are not quantised.
#include "moe_ep.h"
#include "moe_internal.h"
#include "moe_layer.h"
#include "moe_tiles.h"

namespace moe {
namespace {

constexpr int kRows = 16;        // slots of a tile
constexpr int kFewSlots = 64;    // slots that one wavefront sorts in registers

// The expert of slot p, -1 for none.
__device__ __forceinline__ int expert_of(const LayerArgs& a, int p) {
    const int64_t e = p < a.T * a.k ? a.idx[p] : -1;
    if (e < -1 || e >= a.E) {
        atomicOr(a.err, kErrBadTopk);
        return -1;
    }
    return (int)e;
}

// A tile: up to kRows slots of one expert.
struct Found {
    int e, n;   // expert (-1: no more tiles), slots
    int slot;   // of the lane's row, number lane & 15; valid where that is below n
};

// At most 64 slots: each wavefront holds them, one a lane, and takes the experts in the order of their first slots.
struct FewTiles {
    int expert;        // of the lane's slot
    uint64_t left;     // slots of experts not yet taken
    uint64_t mine;     // slots of the current expert
    int e, n, first;   // it, its slots, slots before the next tile
    __device__ __forceinline__ void init(const LayerArgs& a, int lane) {
        expert = expert_of(a, lane);
        left = __ballot(expert >= 0);
        n = first = 0;
    }
    __device__ __forceinline__ Found next(int lane) {
        if (first >= n) {
            if (left == 0) return Found{-1, 0, 0};
            e = __builtin_amdgcn_readlane(expert, __ffsll((unsigned long long)left) - 1);
            mine = __ballot(expert == e);
            left &= ~mine;
            n = __popcll(mine);
            first = 0;
        }
        // each slot's lane tells the lane of its row; the others tell lane 63, which nobody asks
        const int rank = __popcll(mine & ((1ull << lane) - 1)) - first;
        const bool in = (mine >> lane & 1) && rank >= 0 && rank < kRows;
        const int told = __builtin_amdgcn_ds_permute((in ? rank : 63) * 4, lane);
        const Found f = {e, min(kRows, n - first), __shfl(told, lane & 15, 64)};
        first += kRows;
        return f;
    }
};

// More slots: the workgroup counts each expert's in LDS.
struct Counts {
    int count[MOE_MAX_EXPERTS];
    uint16_t expert[MOE_LAYER_MAX_ROWS];   // of each slot, 0xffff for none

    // Also gives the calling thread's slots (tid, tid + NT, ..): their experts, and their numbers among their expert's, in an
    // order that is this workgroup's own.
    template <int NT>
    __device__ __forceinline__ void init(const LayerArgs& a, int (&ex)[MOE_LAYER_MAX_ROWS / NT], int (&rank)[MOE_LAYER_MAX_ROWS / NT]) {
        const int P = a.T * a.k, tid = threadIdx.x;
        for (int e = tid; e < a.E; e += NT) count[e] = 0;
#pragma unroll
        for (int i = 0; i < MOE_LAYER_MAX_ROWS / NT; ++i) {
            ex[i] = i * NT + tid < P ? expert_of(a, i * NT + tid) : -1;
            expert[i * NT + tid] = (uint16_t)ex[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MOE_LAYER_MAX_ROWS / NT; ++i) rank[i] = ex[i] >= 0 ? atomicAdd(&count[ex[i]], 1) : 0;
        __syncthreads();
    }
    // Slots and tiles of the lane's run of experts, and of all lanes' up to it.
    struct Run {
        int first, last;          // experts
        int slots, tiles;         // of them
        int slots_to, tiles_to;   // inclusive sums over the lanes
    };
    __device__ __forceinline__ Run run(const LayerArgs& a, int lane) const {
        const int per = (a.E + 63) / 64;
        Run r = {min(lane * per, a.E), min((lane + 1) * per, a.E), 0, 0, 0, 0};
        for (int e = r.first; e < r.last; ++e) {
            r.slots += count[e];
            r.tiles += (count[e] + kRows - 1) / kRows;
        }
        r.slots_to = r.slots;
        r.tiles_to = r.tiles;
#pragma unroll
        for (int step = 1; step < 64; step <<= 1) {
            const int x = __shfl_up(r.slots_to, step, 64), y = __shfl_up(r.tiles_to, step, 64);
            if (lane >= step) {
                r.slots_to += x;
                r.tiles_to += y;
            }
        }
        return r;
    }
    // One tile.  The workgroups that share an expert's tiles each find their own, so its slots are taken in ascending order.
    __device__ __forceinline__ Found tile(const LayerArgs& a, int want, int lane) const {
        const Run r = run(a, lane);
        const uint64_t here = __ballot(want < r.tiles_to);
        if (here == 0) return Found{-1, 0, 0};
        int left = want - (r.tiles_to - r.tiles), e = r.first;
        for (; e < r.last - 1; ++e) {
            const int n = (count[e] + kRows - 1) / kRows;
            if (left < n) break;
            left -= n;
        }
        const int owner = __ffsll((unsigned long long)here) - 1;
        e = __builtin_amdgcn_readlane(e, owner);
        const int from = __builtin_amdgcn_readlane(left, owner) * kRows;
        Found f = {e, min(kRows, count[e] - from), 0};
        int before = -from;   // the tile's number of the next of the expert's slots
        for (int p = 0; p < a.T * a.k && before < kRows; p += 64) {
            const uint64_t some = __ballot(expert[p + lane] == e);
            const int rank = before + __popcll(some & ((1ull << lane) - 1)), t = lane & 15;
            const bool in = (some >> lane & 1) && rank >= 0 && rank < kRows;
            const int told = __shfl(__builtin_amdgcn_ds_permute((in ? rank : 63) * 4, p + lane), t, 64);
            const int next = before + __popcll(some);
            if (t >= before && t < next) f.slot = told;
            before = next;
        }
        return f;
    }
};

// All of them, sorted by expert.  Which of an expert's slots comes first is left to the order of atomics: one
// workgroup has them all, and results do not depend on it (a slot's sums are its own, wherever in a tile it sits).
struct ManyTiles {
    static constexpr int kMaxTiles = MOE_LAYER_MAX_ROWS + MOE_LAYER_MAX_ROWS / kRows;
    Counts counts;
    uint16_t start[MOE_MAX_EXPERTS], sorted[MOE_LAYER_MAX_ROWS];
    uint16_t tile_e[kMaxTiles], tile_first[kMaxTiles], tile_n[kMaxTiles];
    int tiles;

    template <int NT>
    __device__ __forceinline__ void init(const LayerArgs& a) {
        constexpr int kOwn = MOE_LAYER_MAX_ROWS / NT;
        const int tid = threadIdx.x, lane = tid & 63;
        int ex[kOwn], rank[kOwn];
        counts.init<NT>(a, ex, rank);
        if (tid < 64) {
            const Counts::Run r = counts.run(a, lane);
            if (lane == 63) tiles = r.tiles_to;
            int to = r.slots_to - r.slots, tt = r.tiles_to - r.tiles;
            for (int e = r.first; e < r.last; ++e) {
                const int n = counts.count[e];
                start[e] = (uint16_t)to;
                for (int i = 0; i < n; i += kRows, ++tt) {
                    tile_e[tt] = (uint16_t)e;
                    tile_first[tt] = (uint16_t)(to + i);
                    tile_n[tt] = (uint16_t)min(kRows, n - i);
                }
                to += n;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (ex[i] >= 0) sorted[start[ex[i]] + rank[i]] = (uint16_t)(i * NT + tid);
        __syncthreads();
    }
    __device__ __forceinline__ Found at(int i, int lane) const {
        if (i >= tiles) return Found{-1, 0, 0};
        const int n = tile_n[i], t = lane & 15;
        return Found{tile_e[i], n, sorted[tile_first[i] + min(t, n - 1)]};
    }
};

// The hardware's exponential: its argument's rounding, |g| half steps of binary32, is all that matters, beside the rounding to bf16
// that follows.
__device__ __forceinline__ float silu(float g) { return g * (1.0f / (1.0f + __expf(-g))); }

// One tile against `cols` times 16 gate columns and the up columns that belong to them, the contraction shared out over the
// wavefronts.  (Measured with 16 column tiles, 128 tokens, E4M3, both kernels 2.07 ms: the rows held in registers by sixteen
// wavefronts, so that only the matrix is read, 2.24; two column tiles at a time 2.09 to 2.13, and one token 73 us against 59.)
template <bool FP8, int NW, int AHEAD>
__global__ __launch_bounds__(64 * NW) void k_layer_up(LayerArgs a, int cols) {
    constexpr int kSize = FP8 ? 1 : 2;
    using D = Direct<FP8, 2, 2>;
    union Shared {
        Counts counts;
        f32x4 part[2][NW][2][64];
        __device__ Shared() {}
    };
    __shared__ Shared sh;
    __shared__ __align__(16) char corners[NW][D::kLds];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int all = (a.I + 15) / 16, runs = (all + cols - 1) / cols, tile = (int)blockIdx.x / runs;
    int col = ((int)blockIdx.x - tile * runs) * cols;
    const int last_col = min(col + cols, all);
    Found f;
    if (a.T * a.k <= kFewSlots) {
        FewTiles few;
        few.init(a, lane);
        f = few.next(lane);
        for (int i = 0; i < tile && f.e >= 0; ++i) f = few.next(lane);
    } else {
        int ex[MOE_LAYER_MAX_ROWS / (64 * NW)], rank[MOE_LAYER_MAX_ROWS / (64 * NW)];
        sh.counts.template init<64 * NW>(a, ex, rank);
        f = sh.counts.tile(a, tile, lane);
        __syncthreads();   // the sums go where the counts are
    }
    const int e = __builtin_amdgcn_readfirstlane(f.e), n = __builtin_amdgcn_readfirstlane(f.n);
    if (e < 0) return;
    const int g = lane >> 4, t = lane & 15;
    D d;
    d.corner = corners[w];
    d.ld = a.H * kSize;
    const char* mat = static_cast<const char*>(a.w1) + (int64_t)e * 2 * a.I * d.ld;
    d.rq = descriptor(a.x, a.T * a.H * 2);
    d.set_rows(n, (uint32_t)(f.slot / a.k) * (uint32_t)(a.H * 2), lane);
    int done_col = col, side = 0;
    d.template stream<AHEAD>(
        [&](int* first, int* stride, int* end) {
            *first = w;
            *stride = NW;
            *end = (d.ld + kStepBytes - 1) / kStepBytes;
            if (col >= last_col) return false;
            const int i0 = col++ * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                d.rp[h] = descriptor(mat + (int64_t)(h * a.I + i0) * d.ld, min(16, a.I - i0) * d.ld);
                if constexpr (FP8) d.set_scales(h, a.s1 + ((int64_t)e * (2 * a.I / 128) + (h * a.I + i0) / 128) * (a.H / 128));
            }
            return true;
        },
        [&](const f32x4 (&acc)[2]) {
            sh.part[side][w][0][lane] = acc[0];
            sh.part[side][w][1][lane] = acc[1];
            __syncthreads();   // the next item's go to the other side, so one barrier an item is enough
            const int i = done_col * 16 + 4 * g;
            if (done_col % NW == w && t < n && i < a.I) {   // the wavefronts take turns to join
                f32x4 gate = sh.part[side][0][0][lane], up = sh.part[side][0][1][lane];
#pragma unroll
                for (int j = 1; j < NW; ++j) {
                    gate += sh.part[side][j][0][lane];
                    up += sh.part[side][j][1][lane];
                }
                f32x4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = silu(gate[r]) * up[r];
                *reinterpret_cast<u32x2*>(a.act + (int64_t)f.slot * a.I + i) = bf16_pack(v);
            }
            ++done_col;
            side ^= 1;
        },
        lane);
}

// 16 output columns of every token.  The tiles (times `split` parts of their contraction) go round the
// wavefronts; what a slot contributes stays in LDS until all are done, and each token adds its own in the order of its slots.
template <bool FP8, int NW, int AHEAD>
__global__ __launch_bounds__(64 * NW, 4) void k_layer_down(LayerArgs a) {
    using D = Direct<FP8, 1>;
    constexpr int kSize = FP8 ? 1 : 2, NT = 64 * NW;
    extern __shared__ f32x4 slots[];   // [split][slots][4]
    __shared__ ManyTiles many;
    __shared__ __align__(16) char corners[NW][D::kLds];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int P = a.T * a.k, h0 = (int)blockIdx.x * 16, g = lane >> 4, t = lane & 15;
    const bool small = P <= kFewSlots;
    FewTiles few;
    if (small) few.init(a, lane);
    else many.init<NT>(a);
    D d;
    d.corner = corners[w];
    d.ld = a.I * kSize;
    d.rq = descriptor(a.act, P * a.I * 2);
    const int steps = (d.ld + kStepBytes - 1) / kStepBytes;
    Found f = {-1, 0, 0};
    int have = -1, item = w;                       // tile that f is; next item
    int put_n = 0, put_at = 0, next_n = 0, next_at = 0;   // slots of the item whose sums come next, and of the one loaded after it
    d.template stream<AHEAD>(
        [&](int* first, int* stride, int* end) {
            const int tile = item / a.split, part = item - tile * a.split;
            item += NW;
            if (small) {
                for (; have < tile && (have < 0 || f.e >= 0); ++have) f = few.next(lane);
            } else {
                f = many.at(tile, lane);
            }
            put_n = next_n;
            put_at = next_at;
            *first = part * steps / a.split;
            *stride = 1;
            *end = (part + 1) * steps / a.split;
            const int e = __builtin_amdgcn_readfirstlane(f.e), n = __builtin_amdgcn_readfirstlane(f.n);
            if (e < 0) return false;
            next_n = n;
            next_at = (part * P + f.slot) * 4 + g;
            d.set_rows(n, (uint32_t)f.slot * (uint32_t)(a.I * 2), lane);
            d.rp[0] = descriptor(static_cast<const char*>(a.w2) + ((int64_t)e * a.H + h0) * d.ld, min(16, a.H - h0) * d.ld);
            if constexpr (FP8) d.set_scales(0, a.s2 + ((int64_t)e * (a.H / 128) + h0 / 128) * (a.I / 128));
            return true;
        },
        [&](const f32x4 (&acc)[1]) {
            if (t < put_n) slots[put_at] = acc[0];
        },
        lane);
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 4; i += NT) {
        const int tok = i >> 2, c = i & 3, h = h0 + 4 * c;
        if (h >= a.H) continue;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < a.k; ++j) {
            const int p = tok * a.k + j;
            const int64_t e = a.idx[p];
            if (e < 0 || e >= a.E) continue;
            f32x4 y = slots[p * 4 + c];
            for (int q = 1; q < a.split; ++q) y += slots[(q * P + p) * 4 + c];
            v += y * a.w[p];
        }
        const int64_t at = (int64_t)tok * a.H + h;
        if (a.residual != nullptr) {
            const u32x2 old = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.residual) + at);
            v += f32x4{__uint_as_float(old.x << 16), __uint_as_float(old.x & 0xffff0000u), __uint_as_float(old.y << 16),
                       __uint_as_float(old.y & 0xffff0000u)};
        }
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) = bf16_pack(v);
    }
}

template <bool FP8>
hipError_t launch(const LayerArgs& args, hipStream_t s) {
    LayerArgs a = args;
    const int P = a.T * a.k;
    const int tiles = (P < a.E ? P : a.E) + P / kRows;   // at most
    const int up = (a.I + 15) / 16, down = (a.H + 15) / 16;   // at most 2048 each
    // Column tiles of a workgroup, so that finding its slots does not count: as many as leave more than ten workgroups a compute
    // unit, of which four run at once.  Both kernels, E4M3, of 256 experts: 128 tokens x 8, 8 column tiles, 2.03 ms (16 2.06, 4 2.00;
    // one, first kernel, 1.51 against 1.32); 32 tokens, 8, 1.25 (16 1.31, 4 1.22).  bf16, of 64: 64 tokens x 6, 4, 670 us (2 680).
    int cols = 1;
    while (cols < 16 && (int64_t)tiles * ((up + 2 * cols - 1) / (2 * cols)) > 10 * 256) cols *= 2;
    k_layer_up<FP8, 4, FP8 ? 2 : 4><<<dim3((unsigned)(tiles * ((up + cols - 1) / cols))), dim3(256), 0, s>>>(a, cols);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // 64 slots take little LDS, so two workgroups of eight wavefronts share a compute unit; the sums of 1024 slots are 64 KB,
    // and one of sixteen takes it.
    const bool few = P <= kFewSlots;
    const int waves = few ? 8 : 16;
    a.split = 1;   // every wavefront has work
    while (a.split < waves && tiles * a.split < waves) a.split *= 2;
    const size_t lds = (size_t)a.split * P * 64;
    if (few) k_layer_down<FP8, 8, FP8 ? 2 : 4><<<dim3((unsigned)down), dim3(512), lds, s>>>(a);
    else k_layer_down<FP8, 16, FP8 ? 2 : 4><<<dim3((unsigned)down), dim3(1024), lds, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer(const LayerArgs& a, bool fp8, hipStream_t s) { return fp8 ? launch<true>(a, s) : launch<false>(a, s); }

}  // namespace moe

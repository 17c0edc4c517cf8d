// Matrix products of the experts over the ragged receive rows, on the matrix
// cores of gfx950.
//
// All three products are one contraction D[j][i] = sum_c P(i, c) Q(j, c), where
// i is the contiguous dimension of the output:
//   forward           P = W[e] (i = n, c = k)   Q = rows     (j = row, c = k)
//   backward_rows     P = W[e] (i = k, c = n)   Q = grad_out (j = row, c = n)
//   backward_weights  P = rows (i = k, c = row) Q = grad_out (j = n,  c = row)
// An operand whose contraction index is contiguous in memory ("KC") is read
// from LDS with 16-byte loads; one whose i or j index is contiguous ("MC") with
// transposing 8-byte loads.  P feeds the matrix instruction's first operand, so
// a lane ends up with four consecutive i of one j.
//
// Tiles travel from memory to LDS without passing through registers (buffer
// loads with an LDS destination), in a ring of stages of 128 contraction bytes.
// Those loads write LDS in lane order, so the bank swizzle is applied to the
// address each lane reads from.  Out-of-range lanes read zeros (the buffer
// descriptor ends with the tile's valid rows; a lane whose contraction index is
// past the end gets an address past any descriptor), which is what pads ragged
// rows and contraction tails.
#include "moe_expert.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kStepBytes = 128;          // contraction bytes of a KC stage row: 64 bf16 or 128 fp8
constexpr int kStepC = 64;               // contraction elements of a bf16 stage
constexpr int kTileP = 256;              // i extent of a tile
constexpr uint32_t kOob = 0x80000000u;   // past the end of every descriptor (they hold under 2^31 bytes)
constexpr int kScaleBytes = 1024 + 256;  // fp8: 256 row scales and the tile's weight scales, per stage

__device__ __forceinline__ uint16_t bf16_bits(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);   // round to nearest even
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const void* p, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : (bytes > 0x7fffffff ? 0x7fffffff : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)n, 0x00020000);
}

// ---------------------------------------------------------------- segments
struct Tile {
    int e, row, rows;   // expert, first row within its segment, rows of the tile
    int64_t start;      // packed row of the segment's first row
    int tiles;          // row tiles of the launch
};

__device__ __forceinline__ int64_t seg_base(const Segments& s, int e, int64_t start, bool padded) {
    return padded ? (int64_t)e * s.cap + s.first : start;
}

__device__ __forceinline__ int seg_rows(const Segments& s, int lo, int hi) {
    if (lo < 0 || hi < lo || hi > s.max_rows) {
        atomicOr(s.err, kErrBounds);
        return 0;
    }
    return min(hi - lo, s.seg_cap);
}

// Row tile t of the launch, where expert e has ceil(rows / bq) of them.  Every
// wavefront of the block scans the offsets by itself (E <= 1024: at most 16
// per lane).
__device__ __forceinline__ Tile find_tile(const Segments& s, int t, int bq) {
    const int lane = threadIdx.x & 63;
    const int per = (s.E + 63) / 64;
    const int e0 = min(lane * per, s.E), e1 = min(e0 + per, s.E);
    int own = 0;
    for (int e = e0; e < e1; ++e) own += (seg_rows(s, s.eoff[e], s.eoff[e + 1]) + bq - 1) / bq;
    int incl = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int u = __shfl_up(incl, off, 64);
        if (lane >= off) incl += u;
    }
    Tile r;
    r.tiles = __builtin_amdgcn_readlane(incl, 63);
    const uint64_t here = __ballot(t < incl);
    const int owner = here ? __ffsll((unsigned long long)here) - 1 : 63;
    int rest = t - (incl - own), fe = -1, frow = 0, frows = 0, fstart = 0;
    for (int e = e0; e < e1; ++e) {
        const int lo = s.eoff[e], n = seg_rows(s, lo, s.eoff[e + 1]), m = (n + bq - 1) / bq;
        if (fe < 0) {
            if (rest < m) {
                fe = e;
                frow = rest * bq;
                frows = min(bq, n - frow);
                fstart = lo;
            } else {
                rest -= m;
            }
        }
    }
    r.e = __builtin_amdgcn_readlane(fe, owner);
    r.row = __builtin_amdgcn_readlane(frow, owner);
    r.rows = __builtin_amdgcn_readlane(frows, owner);
    r.start = __builtin_amdgcn_readlane(fstart, owner);
    if (here == 0) r.e = -1;
    return r;
}

// ---------------------------------------------------------------- operands
// KC operand: `rows` rows of 128 contraction bytes a stage.  Row r, 16-byte
// chunk c sits at r * 128 + ((c ^ key(r)) << 4).  P's key pairs with the row
// order of its fragments (see frag_row), Q's with consecutive rows: in both,
// the eight lanes that read together meet eight different keys.
template <bool ISP>
__device__ __forceinline__ int kc_key(int r) {
    return ISP ? ((r & 3) | ((r >> 1) & 4)) : (r & 7);
}

// Fragment rows of P: row i of the 16-row subtile s stands for tile row
// 32 (s / 2) + 8 (i / 4) + 4 (s % 2) + i % 4, so that a lane's four values of
// subtiles s and s + 1 are eight consecutive outputs (one 16-byte store).
__device__ __forceinline__ int p_frag_row(int s, int i) { return 32 * (s >> 1) + 8 * (i >> 2) + 4 * (s & 1) + (i & 3); }

template <int ROWS, bool ISP>
struct LoadKC {
    static constexpr int kBytes = ROWS * kStepBytes;
    static constexpr int kInstr = kBytes / 1024 >= kWaves ? kBytes / 1024 / kWaves : 1;
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t voff[kInstr];
    uint32_t chunk;   // byte offset of the lane's chunk within a stage row
    int kbytes, lds;
    __device__ __forceinline__ void init(const void* base, int64_t ld, int valid, int kb, int w, int lane) {
        rsrc = descriptor(base, (int64_t)valid * ld);
        kbytes = kb;
        lds = (w * kInstr * 1024) & (kBytes - 1);   // a small tile's loads are repeated by several waves
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int r = (lds >> 7) + i * 8 + (lane >> 3);
            const int c = (lane & 7) ^ kc_key<ISP>(r);
            if (i == 0) chunk = c * 16;
            voff[i] = (uint32_t)(r * ld) + c * 16;
        }
    }
    // all of a lane's chunks have the same column only where the key repeats every 8 rows or the
    // instruction index does not change it; P's key depends on r & 8, so keep it per instruction
    __device__ __forceinline__ void issue(char* stage, int step) const {
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const uint32_t col = ISP ? chunk ^ ((i & 1) << 6) : chunk;
            const uint32_t v = (int)col + step * kStepBytes < kbytes ? voff[i] + step * kStepBytes : kOob;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, LDS_PTR(void, stage + lds + i * 1024), 16, v, 0, 0, 0);
        }
    }
    __device__ __forceinline__ static bf16x8 frag(const char* stage, int row, int c) {
        return *reinterpret_cast<const bf16x8*>(stage + row * kStepBytes + ((c ^ kc_key<ISP>(row)) << 4));
    }
    __device__ __forceinline__ static i32x8 frag8(const char* stage, int row, int g) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(stage + row * kStepBytes + (((2 * g) ^ kc_key<ISP>(row)) << 4));
        const i32x4 hi =
            *reinterpret_cast<const i32x4*>(stage + row * kStepBytes + (((2 * g + 1) ^ kc_key<ISP>(row)) << 4));
        return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
};

// MC operand: 64 contraction rows of 256 bf16 a stage.  Contraction row c,
// 32-byte unit u (16 columns) sits at c * 512 + ((u ^ key(c)) << 5).  A
// transposing load takes, for 16 lanes, four contraction rows of 16 columns;
// the 32 lanes that read together meet eight different keys.
__device__ __forceinline__ int mc_key(int c) { return (c & 3) | ((c >> 1) & 4); }

struct LoadMC {
    static constexpr int kBytes = kStepC * 512;
    static constexpr int kInstr = kBytes / 1024 / kWaves;
    const char* base;
    int64_t ld, left;   // bytes of a contraction row; bytes from base to the operand's end
    uint32_t voff[kInstr];
    int lds;
    // base: first contraction row, at the tile's first column; cols: columns from there to the row's end
    __device__ __forceinline__ void init(const void* b, int64_t row_bytes, int64_t crows, int64_t col0, int w, int lane) {
        base = static_cast<const char*>(b) + col0 * 2;
        ld = row_bytes;
        left = crows * row_bytes - col0 * 2;
        lds = w * kInstr * 1024;
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int c = (w * kInstr + i) * 2 + (lane >> 5), p = lane & 31;
            const int chunk = (((p >> 1) ^ mc_key(c)) << 1) | (p & 1);
            voff[i] = col0 * 2 + chunk * 16 < row_bytes ? (uint32_t)(c * row_bytes) + chunk * 16 : kOob;
        }
    }
    __device__ __forceinline__ void issue(char* stage, int step) const {
        const int64_t at = (int64_t)step * kStepC * ld;
        const __amdgpu_buffer_rsrc_t rsrc = descriptor(base + at, left - at);
#pragma unroll
        for (int i = 0; i < kInstr; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, LDS_PTR(void, stage + lds + i * 1024), 16, voff[i], 0, 0, 0);
    }
    // columns 16 sub .. +15 as fragment rows, contraction rows c0 + 8 g .. +7 for lane group g
    __device__ __forceinline__ static bf16x8 frag(const char* stage, int sub, int c0, int lane) {
        const int g = lane >> 4, t = lane & 15;
        const int key = (t >> 2) | ((g & 1) << 2);
        const char* at = stage + (c0 + 8 * g + (t >> 2)) * 512 + ((sub ^ key) << 5) + (t & 3) * 8;
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(LDS_PTR(bf16x4, at));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(LDS_PTR(bf16x4, at + 4 * 512));
        return bf16x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
};

// fp8: one row scale for each of 256 rows and the weight scales of the tile's
// two 128-column blocks, for one 128-channel stage.  Waves 0-3 (and again 4-7,
// with the weight scales) issue one 4-byte load per lane.
struct LoadScales {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t voff;
    int kb, lds;
    __device__ __forceinline__ void init(const float* rows, int valid, const float* mats, int nblocks, int kblocks,
                                         int w, int lane) {
        kb = kblocks;
        if (w < 4) {
            rsrc = descriptor(rows, (int64_t)valid * kb * 4);
            voff = (uint32_t)((w * 64 + lane) * kb) * 4;
            lds = w * 256;
        } else {
            rsrc = descriptor(mats, (int64_t)min(nblocks, 2) * kb * 4);
            voff = lane < 2 ? (uint32_t)(lane * kb) * 4 : kOob;
            lds = 1024;
        }
    }
    __device__ __forceinline__ void issue(char* stage, int step) const {
        const uint32_t v = step < kb ? voff + step * 4 : kOob;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, LDS_PTR(void, stage + lds), 4, v, 0, 0, 0);
    }
};

// s_waitcnt vmcnt(N) only
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// Barrier that orders LDS accesses only: loads into LDS stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

extern __shared__ __align__(1024) char g_lds[];

// ---------------------------------------------------------------- tile body
// One tile of kTileP x BQ outputs.  WP x WQ wavefronts; each owns
// (kTileP / WP) x (BQ / WQ) outputs as 16 x 16 subtiles.
template <int BQ, int WP, int STAGES, bool FP8, bool PMC, bool QMC>
struct TileBody {
    static_assert(WP <= kWaves, "");
    static constexpr int WQ = kWaves / WP;
    static constexpr int PS = kTileP / WP / 16, QS = BQ / WQ / 16;
    static_assert(PS % 2 == 0 && QS >= 1, "");
    static constexpr int kPBytes = kTileP * kStepBytes;
    static constexpr int kQBytes = QMC ? LoadMC::kBytes : BQ * kStepBytes;
    static constexpr int kStage = kPBytes + kQBytes + (FP8 ? kScaleBytes : 0);
    static constexpr int kLds = kStage * STAGES;

    using LP = LoadKC<kTileP, true>;
    using LQ = LoadKC<BQ, false>;

    template <class OpP, class OpQ>
    __device__ __forceinline__ static void run(const OpP& lp, const OpQ& lq, const LoadScales& ls, int steps,
                                               f32x4 (&acc)[PS][QS], int w, int lane) {
        constexpr int kLoads = OpP::kInstr + OpQ::kInstr + (FP8 ? 1 : 0);
        const int wp = w % WP, wq = w / WP;
        auto issue = [&](int step, int slot) {
            char* st = g_lds + slot * kStage;
            lp.issue(st, step);
            lq.issue(st + kPBytes, step);
            if constexpr (FP8) ls.issue(st + kPBytes + kQBytes, step);
        };
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
            for (int q = 0; q < QS; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        lds_barrier();   // the previous tile's reads are done
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) issue(s, s);
        int cur = 0, nxt = STAGES - 1;
        for (int step = 0; step < steps; ++step) {
            wait_loads<(STAGES - 2) * kLoads>();
            lds_barrier();
            issue(step + STAGES - 1, nxt);   // past the end: reads nothing, writes zeros
            const char* sp = g_lds + cur * kStage;
            const char* sq = sp + kPBytes;
            const int g = lane >> 4, t = lane & 15;
            if constexpr (FP8) {
                const float* sc = reinterpret_cast<const float*>(sq + kQBytes);
                const float sw = sc[256 + wp * (kTileP / WP) / 128];
                i32x8 fq[QS];
                float s[QS];
#pragma unroll
                for (int q = 0; q < QS; ++q) {
                    const int row = wq * QS * 16 + q * 16 + t;
                    fq[q] = LQ::frag8(sq, row, g);
                    s[q] = sc[row] * sw;
                }
#pragma unroll
                for (int p = 0; p < PS; ++p) {
                    const i32x8 fp = LP::frag8(sp, wp * PS * 16 + p_frag_row(p, t), g);
#pragma unroll
                    for (int q = 0; q < QS; ++q) {
                        const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            fp, fq[q], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[p][q][r] = __builtin_fmaf(d[r], s[q], acc[p][q][r]);
                    }
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    bf16x8 fq[QS];
#pragma unroll
                    for (int q = 0; q < QS; ++q) {
                        if constexpr (QMC) fq[q] = LoadMC::frag(sq, wq * QS + q, kk * 32, lane);
                        else fq[q] = LQ::frag(sq, wq * QS * 16 + q * 16 + t, kk * 4 + g);
                    }
#pragma unroll
                    for (int p = 0; p < PS; ++p) {
                        bf16x8 fp;
                        if constexpr (PMC) fp = LoadMC::frag(sp, wp * PS + p, kk * 32, lane);
                        else fp = LP::frag(sp, wp * PS * 16 + p_frag_row(p, t), kk * 4 + g);
#pragma unroll
                        for (int q = 0; q < QS; ++q)
                            acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp, fq[q], acc[p][q], 0, 0, 0);
                    }
                }
            }
            cur = cur == STAGES - 1 ? 0 : cur + 1;
            nxt = nxt == STAGES - 1 ? 0 : nxt + 1;
        }
        wait_loads<0>();   // nothing may still be on its way into LDS when it is reused
    }

    // bf16 stores of the tile: out points at the tile's first output, ld its row length; i < ni, j < nj
    __device__ __forceinline__ static void store(uint16_t* out, int64_t ld, int ni, int nj, const f32x4 (&acc)[PS][QS],
                                                 int w, int lane) {
        const int wp = w % WP, wq = w / WP, g = lane >> 4, t = lane & 15;
#pragma unroll
        for (int q = 0; q < QS; ++q) {
            const int j = wq * QS * 16 + q * 16 + t;
            if (j >= nj) continue;
            uint16_t* row = out + (int64_t)j * ld;
#pragma unroll
            for (int p = 0; p < PS; p += 2) {
                const f32x4 x = acc[p][q], y = acc[p + 1][q];
                auto pk = [](float lo, float hi) { return (uint32_t)bf16_bits(lo) | ((uint32_t)bf16_bits(hi) << 16); };
                if constexpr (!PMC) {
                    const int i = wp * PS * 16 + 16 * p + 8 * g;
                    if (i < ni)
                        *reinterpret_cast<i32x4*>(row + i) =
                            i32x4{(int)pk(x[0], x[1]), (int)pk(x[2], x[3]), (int)pk(y[0], y[1]), (int)pk(y[2], y[3])};
                } else {
                    const int i = wp * PS * 16 + 16 * p + 4 * g;
                    if (i < ni) *reinterpret_cast<u32x2*>(row + i) = u32x2{pk(x[0], x[1]), pk(x[2], x[3])};
                    if (i + 16 < ni) *reinterpret_cast<u32x2*>(row + i + 16) = u32x2{pk(y[0], y[1]), pk(y[2], y[3])};
                }
            }
        }
    }
};

// ---------------------------------------------------------------- rows products
// A tile of the forward or the rows gradient: rows [row, row + rows) of expert
// e against output columns [i0, i0 + 256).
template <int BQ, int WP, int STAGES, bool FP8, bool PMC>
__device__ __forceinline__ void rows_tile(const ExpertGemmArgs& a, const Tile& tl, int i0, int w, int lane) {
    using B = TileBody<BQ, WP, STAGES, FP8, PMC, false>;
    constexpr int kSize = FP8 ? 1 : 2;
    const int cdim = PMC ? a.N : a.K, idim = PMC ? a.K : a.N;
    const int64_t qrow = seg_base(a.seg, tl.e, tl.start, a.q_padded) + tl.row;
    const int64_t orow = seg_base(a.seg, tl.e, tl.start, a.out_padded) + tl.row;
    const int ni = min(kTileP, idim - i0);
    const char* wmat = static_cast<const char*>(a.p) + (int64_t)tl.e * a.N * a.K * kSize;
    const int64_t qld = (int64_t)cdim * kSize;
    typename B::LQ lq;
    lq.init(static_cast<const char*>(a.q) + qrow * qld, qld, tl.rows, (int)qld, w, lane);
    LoadScales ls;
    f32x4 acc[B::PS][B::QS];
    const int steps = (cdim * kSize + kStepBytes - 1) / kStepBytes;
    if constexpr (FP8) {
        const int kb = a.K / 128, nb = (a.N + 127) / 128;
        ls.init(a.q_scales + qrow * kb, tl.rows, a.p_scales + ((int64_t)tl.e * nb + i0 / 128) * kb, nb - i0 / 128, kb, w,
                lane);
    }
    if constexpr (PMC) {
        LoadMC lp;
        lp.init(wmat, (int64_t)a.K * 2, a.N, i0, w, lane);
        B::run(lp, lq, ls, steps, acc, w, lane);
    } else {
        typename B::LP lp;
        lp.init(wmat + i0 * qld, qld, ni, (int)qld, w, lane);
        B::run(lp, lq, ls, steps, acc, w, lane);
    }
    B::store(static_cast<uint16_t*>(a.out) + orow * idim + i0, idim, ni, tl.rows, acc, w, lane);
}

// Stages of a tile's ring: what fits in 160 KB of LDS.
constexpr int kLdsBytes = 160 * 1024 - 1024;

template <bool FP8, bool PMC>
__global__ __launch_bounds__(kThreads) void k_expert_rows(ExpertGemmArgs a) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int ntiles = ((PMC ? a.K : a.N) + kTileP - 1) / kTileP;
    // block b runs on XCD b % 8: give each XCD a contiguous run of tiles
    const int b = blockIdx.x;
    const Tile first = find_tile(a.seg, 0, 256);
    const int total = first.tiles * ntiles;
    const int per = (total + 7) / 8;
    if (b / 8 >= per) return;
    const int t = (b % 8) * per + b / 8;
    if (t >= total) return;
    const Tile tl = find_tile(a.seg, t / ntiles, 256);
    if (tl.e < 0) return;
    const int i0 = (t % ntiles) * kTileP;
    if (tl.rows > 128) rows_tile<256, 2, 2, FP8, PMC>(a, tl, i0, w, lane);
    else if (tl.rows > 64) rows_tile<128, 2, 3, FP8, PMC>(a, tl, i0, w, lane);
    else if (tl.rows > 32) rows_tile<64, 4, 3, FP8, PMC>(a, tl, i0, w, lane);
    else rows_tile<32, 8, 4, FP8, PMC>(a, tl, i0, w, lane);
}

// ---------------------------------------------------------------- weights gradient
__global__ __launch_bounds__(kThreads) void k_expert_weights_grad(ExpertGemmArgs a) {
    using B = TileBody<256, 2, 2, false, true, true>;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int kt = (a.K + kTileP - 1) / kTileP, nt = (a.N + 255) / 256;
    const int b = blockIdx.x;
    const int e = b / (kt * nt), rest = b % (kt * nt);
    const int i0 = (rest % kt) * kTileP, j0 = (rest / kt) * 256;
    const int lo = a.seg.eoff[e];
    const int rows = seg_rows(a.seg, lo, a.seg.eoff[e + 1]);
    const int64_t prow = seg_base(a.seg, e, lo, a.p_padded), qrow = seg_base(a.seg, e, lo, a.q_padded);
    LoadMC lp, lq;
    lp.init(static_cast<const char*>(a.p) + (rows ? prow * a.K * 2 : 0), (int64_t)a.K * 2, rows, i0, w, lane);
    lq.init(static_cast<const char*>(a.q) + (rows ? qrow * a.N * 2 : 0), (int64_t)a.N * 2, rows, j0, w, lane);
    f32x4 acc[B::PS][B::QS];
    LoadScales ls;
    B::run(lp, lq, ls, (rows + kStepC - 1) / kStepC, acc, w, lane);
    const int ni = min(kTileP, a.K - i0), nj = min(256, a.N - j0);
    const int64_t at = ((int64_t)e * a.N + j0) * a.K + i0;
    const int wp = w % 2, wq = w / 2, g = lane >> 4, t = lane & 15;
    if (a.accumulate || a.out_f32) {
#pragma unroll
        for (int q = 0; q < B::QS; ++q) {
            const int j = wq * B::QS * 16 + q * 16 + t;
#pragma unroll
            for (int p = 0; p < B::PS; ++p) {
                const int i = wp * B::PS * 16 + 16 * p + 4 * g;
                if (j >= nj || i >= ni) continue;
                const int64_t o = at + (int64_t)j * a.K + i;
                if (a.out_f32) {
                    f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o);
                    *d = a.accumulate ? *d + acc[p][q] : acc[p][q];
                } else {
                    u32x2* d = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + o);
                    const u32x2 old = *d;
                    f32x4 v = acc[p][q];
                    v[0] += __uint_as_float(old.x << 16);
                    v[1] += __uint_as_float(old.x & 0xffff0000u);
                    v[2] += __uint_as_float(old.y << 16);
                    v[3] += __uint_as_float(old.y & 0xffff0000u);
                    *d = u32x2{(uint32_t)bf16_bits(v[0]) | ((uint32_t)bf16_bits(v[1]) << 16),
                               (uint32_t)bf16_bits(v[2]) | ((uint32_t)bf16_bits(v[3]) << 16)};
                }
            }
        }
    } else {
        B::store(static_cast<uint16_t*>(a.out) + at, a.K, ni, nj, acc, w, lane);
    }
}

hipError_t allow_lds(const void* f) {
    return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
}

template <bool FP8, bool PMC>
hipError_t launch_rows(const ExpertGemmArgs& a, int64_t pairs, hipStream_t s) {
    const int64_t ntiles = ((PMC ? a.K : a.N) + kTileP - 1) / kTileP;
    const int64_t mtiles = pairs / 256 + (pairs < a.seg.E ? pairs : a.seg.E);   // at least one expert per ragged end
    const int64_t blocks = (mtiles * ntiles + 7) / 8 * 8;
    hipError_t e = allow_lds(reinterpret_cast<const void*>(&k_expert_rows<FP8, PMC>));
    if (e != hipSuccess) return e;
    k_expert_rows<FP8, PMC><<<dim3((unsigned)blocks), dim3(kThreads), kLdsBytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertGemmArgs& a, bool fp8, int64_t pairs, hipStream_t s) {
    return fp8 ? launch_rows<true, false>(a, pairs, s) : launch_rows<false, false>(a, pairs, s);
}

hipError_t launch_expert_gemm_bwd_rows(const ExpertGemmArgs& a, int64_t pairs, hipStream_t s) {
    return launch_rows<false, true>(a, pairs, s);
}

hipError_t launch_expert_gemm_bwd_weights(const ExpertGemmArgs& a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.seg.E * ((a.K + kTileP - 1) / kTileP) * ((a.N + 255) / 256);
    hipError_t e = allow_lds(reinterpret_cast<const void*>(&k_expert_weights_grad));
    if (e != hipSuccess) return e;
    k_expert_weights_grad<<<dim3((unsigned)blocks), dim3(kThreads), kLdsBytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe

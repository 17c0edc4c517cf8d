// What the matrix products are built from, on the matrix cores of gfx950: operands on
// their way from memory to LDS to fragments, and one tile of 256 columns.  Included
// by the kernels of the expert products, of the dense product and of the layer of a
// few tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_ep.h"

namespace moe {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int kStepBytes = 128;          // contraction bytes of a KC stage row: 64 bf16 or 128 fp8
constexpr int kStepC = 64;               // contraction elements of a bf16 stage
constexpr int kTileP = 256;              // i extent of a tile
constexpr int kNonTemporal = 2;          // cache policy of a buffer access
constexpr uint32_t kOob = 0x80000000u;   // past the end of every descriptor (they hold under 2^31 bytes)

__device__ __forceinline__ uint32_t bf16_bits(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);   // round to nearest even
}
__device__ __forceinline__ u32x2 bf16_pack(f32x4 v) {
    return u32x2{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
}

// A descriptor covers one stage of one tile, at most 256 rows of 2 * MOE_MAX_FEATURES bytes, or all rows of a few tokens.
static_assert(256ll * 2 * MOE_MAX_FEATURES < kOob && 2ll * MOE_LAYER_MAX_ROWS * MOE_MAX_FEATURES < kOob, "");
__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, max(bytes, 0), 0x00020000);
}

// ---------------------------------------------------------------- order of tiles
// Block b runs on XCD b % 8, and about 256 blocks (32 for each XCD) run together: blocks of one
// XCD take 32 consecutive tiles of each run of 256, so that they share operand panels in its L2.
__device__ __forceinline__ int64_t xcd_tile(int b) {
    const int i = b >> 3;
    return ((int64_t)(i >> 5) << 8) + ((b & 7) << 5) + (i & 31);
}

// The same for many small blocks, four neighbouring tiles on one XCD: of the row tiles of a matrix (4 experts
// x 64 rows in tiles of 32, 4096 x 4096 bf16: 49 us, 73 with neighbours spread over the XCDs), or of columns
// that share lines of the output.
__device__ __forceinline__ int xcd_tile4(int b) { return (b & ~31) | ((b & 7) << 2) | ((b >> 3) & 3); }

// The same where the tiles are known on the host: each XCD takes `run` consecutive ones at a time.  What the tiles of an XCD
// share is read from memory once: 4096 rows of 7168 against 256 columns in tiles of 64 x 64, 8 rows of tiles an XCD, 36 us,
// 40 with 4 neighbours an XCD.
constexpr int kMostRun = 32;
inline int xcd_run(int64_t tiles) { return tiles >= 8 * kMostRun ? kMostRun : (int)((tiles + 7) / 8); }
inline int64_t xcd_grid(int64_t tiles, int run) { return (tiles + 8 * run - 1) / (8 * run) * (8 * run); }
__device__ __forceinline__ int64_t xcd_run_tile(int b, int run) {
    const int i = b >> 3;
    return (int64_t)(i / run) * (8 * run) + (b & 7) * run + i % run;
}

// Order of the tiles of one matrix with `nj` row tiles and `ni` column tiles: bands of kBand row
// tiles, column by column, so that 32 consecutive tiles touch about 4 + 8 panels.
constexpr int kBand = 4;
__device__ __forceinline__ void band_order(int l, int nj, int ni, int* j, int* i) {
    const int band = l / (kBand * ni), rest = l - band * kBand * ni;
    const int height = min(kBand, nj - band * kBand);
    *i = rest / height;
    *j = band * kBand + rest - *i * height;
}

// ---------------------------------------------------------------- operands
// KC operand: ROWS rows of 128 contraction bytes a stage.  Row r, 16-byte chunk c sits at
// r * 128 + ((c ^ (r & 7)) << 4): the eight lanes that read together meet eight different chunks.
// TAIL: rows need not be whole steps.
template <int ROWS, int NW, bool TAIL>
struct LoadKC {
    static constexpr int kBytes = ROWS * kStepBytes;
    static constexpr int kInstr = (kBytes / 1024 + NW - 1) / NW;
    const char* base;
    int bytes;        // of the valid rows
    uint32_t voff[kInstr];
    uint32_t chunk;   // byte offset of the lane's chunk within a stage row
    int kbytes, lds[kInstr];
    __device__ __forceinline__ void init(const void* b, int ld, int valid, int kb, int w, int lane) {
        base = static_cast<const char*>(b);
        bytes = valid * ld;
        kbytes = kb;
        chunk = ((lane & 7) ^ (lane >> 3)) * 16;   // an instruction covers eight rows
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            // where the wavefronts' loads do not divide the tile, some are made twice
            lds[i] = (w * kInstr + i) % (kBytes / 1024) * 1024;
            voff[i] = (lds[i] / kStepBytes + (lane >> 3)) * ld + chunk;
        }
    }
    // The descriptor moves along the rows, so a lane's offsets stay the same.  What it would read past
    // a row's end is the next row: columns behind a last step of fewer than 128 bytes are masked.
    struct Step {
        __amdgpu_buffer_rsrc_t rsrc;
        int left;
    };
    __device__ __forceinline__ Step step_of(int step) const {
        const int at = step * kStepBytes;
        return Step{descriptor(base + at, at < kbytes ? bytes - at : 0), kbytes - at};
    }
    __device__ __forceinline__ void issue(char* stage, const Step& st, int i) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rsrc, LDS_PTR(void, stage + lds[i]), 16,
                                                 !TAIL || (int)chunk < st.left ? voff[i] : kOob, 0, 0, 0);
    }
    __device__ __forceinline__ static bf16x8 frag(const char* stage, int row, int c) {
        return *reinterpret_cast<const bf16x8*>(stage + (row * kStepBytes + ((c ^ (row & 7)) << 4)));
    }
    // fp8: a lane group's 32 of the 128 channels are chunks g and g + 4 (both operands agree, so the
    // order within the contraction is free): with chunks 2 g and 2 g + 1 half the LDS cycles are conflicts
    __device__ __forceinline__ static i32x8 frag8(const char* stage, int row, int g) {
        const int at = row * kStepBytes, key = row & 7;
        const i32x4 lo = *reinterpret_cast<const i32x4*>(stage + (at + ((g ^ key) << 4)));
        const i32x4 hi = *reinterpret_cast<const i32x4*>(stage + (at + (((g + 4) ^ key) << 4)));
        return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
};

// MC operand: 64 contraction rows of W bf16 a stage.  Contraction row c,
// 32-byte unit u (16 columns) sits at c * 2 W + ((u ^ key(c)) << 5).  A
// transposing load takes, for 16 lanes, four contraction rows of 16 columns;
// the 32 lanes that read together meet eight different keys.
__device__ __forceinline__ int mc_key(int c) { return (c & 3) | ((c >> 1) & 4); }

template <int NW, int W = 256>
struct LoadMC {
    static constexpr int kRow = W * 2, kLanes = kRow / 16;   // bytes of a stage row, lanes that load it
    static constexpr int kBytes = kStepC * kRow;
    static constexpr int kInstr = kBytes / 1024 / NW;
    const char* base;
    int ld, crows, before;   // bytes of a contraction row, contraction rows, bytes of a row before the tile
    uint32_t voff[kInstr];
    int lds;
    __device__ __forceinline__ void init(const void* b, int row_bytes, int n, int col0, int w, int lane) {
        before = col0 * 2;
        base = static_cast<const char*>(b) + before;
        ld = row_bytes;
        crows = n;
        lds = w * kInstr * 1024;
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int c = (w * kInstr + i) * (64 / kLanes) + lane / kLanes, p = lane % kLanes;
            const int chunk = (((p >> 1) ^ mc_key(c)) << 1) | (p & 1);
            voff[i] = before + chunk * 16 < row_bytes ? (uint32_t)(c * row_bytes) + chunk * 16 : kOob;
        }
    }
    struct Step {
        __amdgpu_buffer_rsrc_t rsrc;
    };
    __device__ __forceinline__ Step step_of(int step) const {
        const int c0 = step * kStepC;
        return Step{descriptor(base + (int64_t)c0 * ld, min(crows - c0, kStepC) * ld - before)};
    }
    __device__ __forceinline__ void issue(char* stage, const Step& st, int i) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rsrc, LDS_PTR(void, stage + (lds + i * 1024)), 16, voff[i], 0, 0,
                                                 0);
    }
    // columns 16 sub .. +15 as fragment rows, contraction rows c0 + 8 g .. +7 for lane group g
    __device__ __forceinline__ static bf16x8 frag(const char* stage, int sub, int c0, int lane) {
        const int g = lane >> 4, t = lane & 15;
        const int key = (t >> 2) | ((g & 1) << 2);
        const int at = (c0 + 8 * g + (t >> 2)) * kRow + ((sub ^ key) << 5) + (t & 3) * 8;
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(LDS_PTR(bf16x4, stage + at));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(LDS_PTR(bf16x4, stage + (at + 4 * kRow)));
        return bf16x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
};

// The steps of a tile in the order they are taken: from `start` to the end, then from 0.  Rows of
// matrices whose length is a power of two lie on few memory channels at one column; tiles that start
// at different columns spread over all of them.
struct Steps {
    int n, start;
    // Arithmetic instead of conditions: for those the compiler branches, and moves the scaling of the
    // matrix results past the branch, into more registers than there are.
    __device__ __forceinline__ static int not_below(int a, int b) { return (b - 1 - a) >> 31; }   // a >= b ? -1 : 0
    __device__ __forceinline__ static int select(int mask, int yes, int no) { return no ^ ((no ^ yes) & mask); }
    // step of the s-th turn; past the end a step that reads nothing
    __device__ __forceinline__ int at(int s) const {
        const int k = s + start;
        return select(not_below(s, n), n, k - (n & not_below(k, n)));
    }
    // turn s's run of four steps 4 i .. 4 i + 3, counted in the order they are taken (start is 0, or
    // both start and n are multiples of 4)
    __device__ __forceinline__ int four(int s) const { return s >> 2; }
};

// fp8: the scales of the tile's rows and of its two 128-column blocks, for four steps at a time (one
// load a lane and step costs 9% of the prefill product).  Two runs of four are held: row r's at
// (run % 2) * 4096 + r * 16, the blocks' at 8192 + (run % 2) * 1024.  A run that passes a row's end
// reads the next row's, which no step uses; past the last row the loads return zeros, dword by dword.
struct LoadScales {
    static constexpr int kBytes = 2 * 4096 + 2 * 1024;
    __amdgpu_buffer_rsrc_t rsrc;
    char* lds;
    uint32_t voff;
    int at, slot, dump;
    // wavefronts 0-3 load the rows', 4-7 all the blocks'; dump: where 1 KB relative to `to` is free
    __device__ __forceinline__ void init(const float* rows, int valid, const float* mats, int nblocks, int kblocks, char* to,
                                         int unused, int w, int lane) {
        lds = to;
        dump = unused;
        rsrc = w < 4 ? descriptor(rows, valid * kblocks * 4) : descriptor(mats, min(nblocks, 2) * kblocks * 4);
        voff = (uint32_t)((w < 4 ? w * 64 + lane : lane) * kblocks * 4);
        at = w < 4 ? w * 1024 : 8192;
        slot = w < 4 ? 4096 : 1024;
    }
    // The loads of turn s where it begins a run; else loads that read nothing.
    __device__ __forceinline__ void issue(const Steps& order, int s) const {
        const int k = order.at(s);
        const int begins = ~Steps::not_below(s, order.n) & (((k & 3) - 1) >> 31);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, LDS_PTR(void, lds + Steps::select(begins, at + (order.four(s) & 1) * slot, dump)), 16,
            (voff + k * 4) | (kOob & ~begins), 0, 0, 0);
    }
    // turn s's scale of a row times that of a column block
    __device__ __forceinline__ float read(const Steps& order, int s, int row, int block) const {
        const int run = order.four(s) & 1, k = (order.at(s) & 3) * 4;
        return *reinterpret_cast<const float*>(lds + (run * 4096 + k + row * 16)) *
               *reinterpret_cast<const float*>(lds + (8192 + run * 1024 + k + block * 16));
    }
};

// s_waitcnt vmcnt(N) only
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// Barrier that orders LDS accesses only.  The compiler counts loads into LDS as LDS accesses: where it cannot tell
// that none in flight belongs to this fence it puts s_waitcnt vmcnt(0) before the barrier, whatever wait_loads() left in
// flight.  So it is in every loop of the narrow kernels, in two of three steps of the three-stage tiles, and at the
// first barrier of a tile: right, but with one step in flight where the stages could hold two or three.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// One stage: P's tile and Q's.
struct Stage {
    char *p, *q;
};

// ---------------------------------------------------------------- tile body
// One tile of kTileP x BQ outputs.  WP x WQ wavefronts; each owns
// (kTileP / WP) x (BQ / WQ) outputs as PS x QS subtiles of 16 x 16.
//
// A step's matrix instructions are issued in groups, one P fragment times the QS Q fragments each; P
// fragments are read kAhead groups before they are used, bf16's Q fragments half a step before.  After
// the group whose reads are the last from the stage, one barrier says that every wavefront is done
// with it and that the next stage has arrived; the remaining groups issue the loads that refill the
// freed stage, for STAGES steps on, and read the first fragments of the next.  What is waited for are
// loads that had STAGES - 1 steps' time to arrive, or one step's where lds_barrier() waits for all of
// them (two of three steps with three stages).  Groups are kept in this order (the
// scheduler is fenced off between them): with all loads right behind the barrier the wavefronts
// queue for the address unit while the matrix cores are idle.
template <int NW, int BQ, int WP, int STAGES, bool FP8, bool PMC, bool QMC>
struct TileBody {
    static_assert(WP <= NW, "");
    static constexpr int WQ = NW / WP;
    static constexpr int PS = kTileP / WP / 16, QS = BQ / WQ / 16;
    static_assert((PS == 2 || PS % 4 == 0) && QS >= 1, "");

    using LP = LoadKC<kTileP, NW, !FP8>;
    using LQ = LoadKC<BQ, NW, !FP8>;
    using MC = LoadMC<NW>;
    using Frag = typename std::conditional<FP8, i32x8, bf16x8>::type;

    static constexpr int kHalves = FP8 ? 1 : 2;      // matrix instructions of one step along the contraction
    static constexpr int kGroups = kHalves * PS;
    static constexpr int kRing = FP8 || PS < 4 ? 2 : 4;   // P fragments held
    static constexpr int kAhead = kRing - 1;
    static_assert(kAhead <= PS, "the first half's Q fragments are replaced in the second half");

    __device__ __forceinline__ static Frag read_p(const Stage& st, int i, int w, int lane) {
        const int wp = w % WP, g = lane >> 4, t = lane & 15, h = i / PS, p = i % PS;
        if constexpr (FP8) return LP::frag8(st.p, wp * PS * 16 + p * 16 + t, g);
        else if constexpr (PMC) return MC::frag(st.p, wp * PS + p, h * 32, lane);
        else return LP::frag(st.p, wp * PS * 16 + p * 16 + t, h * 4 + g);
    }
    __device__ __forceinline__ static Frag read_q(const Stage& st, int h, int q, int w, int lane) {
        const int wq = w / WP, g = lane >> 4, t = lane & 15;
        if constexpr (FP8) return LQ::frag8(st.q, wq * QS * 16 + q * 16 + t, g);
        else if constexpr (QMC) return MC::frag(st.q, wq * QS + q, h * 32, lane);
        else return LQ::frag(st.q, wq * QS * 16 + q * 16 + t, h * 4 + g);
    }
    __device__ __forceinline__ static float read_scale(const LoadScales& ls, const Steps& order, int turn, int q, int w,
                                                       int lane) {
        return ls.read(order, turn, (w / WP) * QS * 16 + q * 16 + (lane & 15), (w % WP) * (kTileP / WP) / 128);
    }

    // One turn, in stage `cur`.  qc: Q fragments of its first half, read already, and at the end the
    // next turn's; sc: fp8's scales, likewise.
    template <class OpP, class OpQ>
    __device__ __forceinline__ static void step_of(const Stage& cur, const Stage& nxt, int turn, const Steps& order,
                                                   const OpP& lp, const OpQ& lq, const LoadScales& ls, Frag (&pr)[kRing],
                                                   Frag (&qc)[QS], float (&sc)[QS], f32x4 (&acc)[PS][QS], int w, int lane) {
        constexpr int kLoadsP = OpP::kInstr, kLoads = OpP::kInstr + OpQ::kInstr + (FP8 ? 1 : 0);
        constexpr int kBefore = kGroups - kAhead;                  // groups before the barrier
        constexpr int kQGroups = PS < kBefore ? PS : kBefore;      // they read the second half's Q
        const int next = order.at(turn + STAGES);   // past the end it reads nothing and writes zeros
        const auto sp = lp.step_of(next);
        const auto sq = lq.step_of(next);
        Frag qn[QS];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            if (i == kBefore) {
                wait_loads<(STAGES - 2) * kLoads>();
                lds_barrier();
            }
            if (i < kBefore) {
                pr[(i + kAhead) % kRing] = read_p(cur, i + kAhead, w, lane);
                if (!FP8 && i < kQGroups) {
#pragma unroll
                    for (int q = i * QS / kQGroups; q < (i + 1) * QS / kQGroups; ++q) qn[q] = read_q(cur, 1, q, w, lane);
                }
            } else {
                const int j = i - kBefore;
                pr[(i + kAhead) % kRing] = read_p(nxt, j, w, lane);
                if constexpr (!FP8) {
#pragma unroll
                    for (int q = j * QS / kAhead; q < (j + 1) * QS / kAhead; ++q) qc[q] = read_q(nxt, 0, q, w, lane);
                }
#pragma unroll
                for (int l = j * kLoads / kAhead; l < (j + 1) * kLoads / kAhead; ++l) {
                    if (l < kLoadsP) lp.issue(cur.p, sp, l);
                    else if (l < kLoadsP + OpQ::kInstr) lq.issue(cur.q, sq, l - kLoadsP);
                    else ls.issue(order, turn + STAGES);
                }
            }
            const int p = i % PS;
            if constexpr (FP8) {
                constexpr int kAtOnce = 5;   // unscaled results held
#pragma unroll
                for (int q0 = 0; q0 < QS; q0 += kAtOnce) {
                    f32x4 d[kAtOnce];
#pragma unroll
                    for (int q = q0; q < QS && q < q0 + kAtOnce; ++q) {
                        d[q - q0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pr[i % kRing], qc[q], f32x4{0.f, 0.f, 0.f, 0.f},
                                                                                     0, 0, 0, 0, 0, 0);
                        if (i == kGroups - 1) {   // this fragment was used for the last time
                            __builtin_amdgcn_sched_barrier(0);
                            qc[q] = read_q(nxt, 0, q, w, lane);
                        }
                    }
#pragma unroll
                    for (int q = q0; q < QS && q < q0 + kAtOnce; ++q) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[p][q][r] = __builtin_fmaf(d[q - q0][r], sc[q], acc[p][q][r]);
                        if (i == kGroups - 1) sc[q] = read_scale(ls, order, turn + 1, q, w, lane);
                    }
                    if (q0 + kAtOnce < QS) __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int q = 0; q < QS; ++q)
                    acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pr[i % kRing], i < PS ? qc[q] : qn[q], acc[p][q],
                                                                       0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // begin() starts the loads of a tile's first steps, run() does the rest.
    template <class OpP, class OpQ>
    __device__ __forceinline__ static void begin(const Stage (&st)[STAGES], const OpP& lp, const OpQ& lq,
                                                 const LoadScales& ls, const Steps& order) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s) {
            const int step = order.at(s);
            const auto sp = lp.step_of(step);
            const auto sq = lq.step_of(step);
#pragma unroll
            for (int l = 0; l < OpP::kInstr; ++l) lp.issue(st[s].p, sp, l);
#pragma unroll
            for (int l = 0; l < OpQ::kInstr; ++l) lq.issue(st[s].q, sq, l);
            if constexpr (FP8) ls.issue(order, s);
        }
    }
    template <class OpP, class OpQ>
    __device__ __forceinline__ static void run(const Stage (&st)[STAGES], const OpP& lp, const OpQ& lq, const LoadScales& ls,
                                               const Steps& order, f32x4 (&acc)[PS][QS], int w, int lane) {
        constexpr int kLoads = OpP::kInstr + OpQ::kInstr + (FP8 ? 1 : 0);
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
            for (int q = 0; q < QS; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        Frag pr[kRing], qc[QS];
        float sc[QS];
        wait_loads<(STAGES - 1) * kLoads>();   // the first stage's; lds_barrier() waits for the others' too
        lds_barrier();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) pr[i] = read_p(st[0], i, w, lane);
#pragma unroll
        for (int q = 0; q < QS; ++q) {
            qc[q] = read_q(st[0], 0, q, w, lane);
            if constexpr (FP8) sc[q] = read_scale(ls, order, 0, q, w, lane);
        }
        // A stage is known at compile time, so the loop takes STAGES steps a turn; leaving it in the
        // middle would give the accumulators two sets of registers.
        int step = 0;
        for (; step + STAGES - 1 < order.n; step += STAGES) {
#pragma unroll
            for (int s = 0; s < STAGES; ++s)
                step_of(st[s], st[(s + 1) % STAGES], step + s, order, lp, lq, ls, pr, qc, sc, acc, w, lane);
        }
        if (step < order.n) {
            step_of(st[0], st[1], step, order, lp, lq, ls, pr, qc, sc, acc, w, lane);
            if (STAGES > 2 && step + 1 < order.n)
                step_of(st[1], st[2 % STAGES], step + 1, order, lp, lq, ls, pr, qc, sc, acc, w, lane);
        }
        wait_loads<0>();   // nothing may be on its way into LDS when the stages are used again
    }

    // bf16 stores of the tile: out points at its first output, ld is its row length; i < ni, j < nj.  A
    // lane holds four columns of one row: 16 rows of kCols columns at a time go through LDS, so that a
    // store writes whole 128-byte lines (direct 8-byte stores reach them in four parts).  A row's
    // 16-byte chunk c sits at c ^ row.  The stores pass the caches (non-temporal) where rows are whole lines; else
    // two tiles share lines, which meet in L2 (gradients of 64 matrices of 4104 x 4096: 0.55 ms, 1.23 past the
    // caches; of 4096 x 4096 0.39 past them, 0.44 not).
    static constexpr int kCols = PS >= 4 ? 64 : PS * 16, kChunks = kCols / 8;
    __device__ __forceinline__ static void store(uint16_t* out, int64_t ld, int ni, int nj, const f32x4 (&acc)[PS][QS],
                                                 char* scratch, int w, int lane) {
        const int wp = w % WP, wq = w / WP, g = lane >> 4, t = lane & 15;
        char* mine = scratch + w * 2048;
        const auto rsrc = descriptor(out, ((nj - 1) * (int)ld + ni) * 2);
        const bool whole = ld % 64 == 0;
#pragma unroll
        for (int q = 0; q < QS; ++q) {
#pragma unroll
            for (int p0 = 0; p0 < PS; p0 += kCols / 16) {
#pragma unroll
                for (int p = 0; p < kCols / 16; ++p) {
                    const f32x4 v = acc[p0 + p][q];
                    const int c = 2 * p + (g >> 1);
                    *reinterpret_cast<u32x2*>(mine + t * kCols * 2 + (((c ^ t) & (kChunks - 1)) << 4) + (g & 1) * 8) =
                        bf16_pack(v);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
                for (int k = 0; k < kCols / 32; ++k) {
                    const int r = k * (64 / kChunks) + lane / kChunks, c = lane % kChunks;
                    const i32x4 v = *reinterpret_cast<const i32x4*>(mine + r * kCols * 2 + (((c ^ r) & (kChunks - 1)) << 4));
                    const int j = wq * QS * 16 + q * 16 + r, i = (wp * PS + p0) * 16 + c * 8;
                    const int at = j < nj && i < ni ? (j * (int)ld + i) * 2 : (int)kOob;   // past the end nothing is stored
                    if (whole) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, at, 0, kNonTemporal);
                    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, at, 0, 0);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            }
        }
    }
};

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)off, 0, 0));
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)off, 0, 0));
}

// ---------------------------------------------------------------- matrices straight into registers
// PS subtiles of 16 matrix rows against up to 16 bf16 rows for one wavefront: a step is 128 bytes of each matrix row, in bf16
// (64 channels) or E4M3 codes (128, widened to bf16, which holds every code exactly).  NP panels of the matrix (a gate's and
// an up's) take PS / NP subtiles each.  E4M3: a step's sums are multiplied by the scale of its 128 x 128 block before they are
// added.
//
// What bounds reading a matrix this way is how much a compute unit's vector cache has on its way: some 700 requests of 64
// bytes, those that hit or read nothing among them.  So the rows, of which there are few, are not read as the matrix
// instruction wants them (four or two loads for 16 rows, whether they are there or not): a load brings the step of four
// (bf16: eight) rows, and a wavefront's corner of LDS, which no one else uses and nobody waits for, turns it into fragments.
template <bool FP8, int PS, int NP = 1>
struct Direct {
    static_assert(PS % NP == 0, "");
    static constexpr int kPer = PS / NP;
    static constexpr int kRowBytes = FP8 ? 256 : 128, kGroup = 1024 / kRowBytes, kGroups = 16 / kGroup;   // a row's step; rows of a load, loads
    static constexpr int kLds = 16 * kRowBytes;   // bytes of a wavefront's corner
    struct Step {
        i32x4 p[PS][2], q[kGroups];
        float m[NP];
    };
    __amdgpu_buffer_rsrc_t rp[NP], rq;
    // E4M3: the panels' scales, one a step, in scalar loads (as vector loads they took a tenth of the time)
    const __attribute__((address_space(4))) float* scales[NP];
    uint32_t row[kGroups];   // byte offset of the rows that the lane loads, with its place in them
    int groups;              // loads that the rows take
    int ld;                  // bytes of a matrix row
    char* corner;

    // n rows; from: byte offset of row lane & 15, anything from n on.
    __device__ __forceinline__ void set_rows(int n, uint32_t from, int lane) {
        groups = (n + kGroup - 1) / kGroup;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int r = j * kGroup + lane * 16 / kRowBytes;
            const uint32_t of = __shfl(from, r, 64);
            row[j] = r < n ? of + lane * 16 % kRowBytes : kOob;
        }
    }
    __device__ __forceinline__ void set_scales(int panel, const float* of) {
        scales[panel] = (const __attribute__((address_space(4))) float*)of;
    }
    // Past the end of a row a step's lanes load zeros, for both operands.
    __device__ __forceinline__ void load(Step& x, int step, int lane) const {
        const int g = lane >> 4, t = lane & 15;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int at = step * kStepBytes + g * 16 + c * 64;
            const uint32_t off = at < ld ? (uint32_t)(t * ld + at) : kOob;
#pragma unroll
            for (int p = 0; p < PS; ++p) x.p[p][c] = load16(rp[p / kPer], off + (uint32_t)(p % kPer * 16 * ld));
        }
        if constexpr (FP8) {
#pragma unroll
            for (int n = 0; n < NP; ++n) x.m[n] = scales[n][min(step, ld / kStepBytes - 1)];
        }
        const int at = step * kRowBytes;
        const bool in = at + lane * 16 % kRowBytes < (FP8 ? 2 * ld : ld);
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
            if (j == 0 || j < groups) x.q[j] = load16(rq, in ? row[j] + at : kOob);
    }
    // Row r's 16-byte chunk c sits at c ^ r of the row's.
    __device__ __forceinline__ char* place(int r, int c) const {
        return corner + r * kRowBytes + (((c ^ r) & (kRowBytes / 16 - 1)) << 4);
    }
    // eight E4M3 codes as bf16
    __device__ __forceinline__ static bf16x8 widen(int lo, int hi) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
        return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
    __device__ __forceinline__ void multiply(const Step& x, f32x4 (&acc)[PS], int loaded, int lane) const {
        constexpr int kFrags = FP8 ? 4 : 2;
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
            if (j == 0 || j < loaded) *reinterpret_cast<i32x4*>(place(j * kGroup + lane * 16 / kRowBytes, lane & (kRowBytes / 16 - 1))) = x.q[j];
        const int g = lane >> 4, t = lane & 15;
        bf16x8 q[kFrags];   // of rows that are not there, whatever the corner holds: their sums are not used
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
            q[i] = *reinterpret_cast<const bf16x8*>(place(t, FP8 ? 2 * g + (i >> 1) * 8 + (i & 1) : g + 4 * i));
#pragma unroll
        for (int p = 0; p < PS; ++p) {
            if constexpr (FP8) {
                f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(x.p[p][i / 2][i % 2 * 2], x.p[p][i / 2][i % 2 * 2 + 1]), q[i], d, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[p][r] = __builtin_fmaf(d[r], x.m[p / kPer], acc[p][r]);
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.p[p][c]), q[c], acc[p], 0, 0, 0);
            }
        }
    }
    // One item after another, the next one's loads behind the last of this one's, so that nothing runs dry between
    // them, AHEAD steps on their way; the loads stay in order (the scheduler is fenced off), so that a use waits for its own
    // only.  next(first, stride, end) points this at the next item (descriptors, rows) and says which steps; false: there is
    // none.  done(acc) gets the sums of the item before.
    template <int AHEAD, class Next, class Done>
    __device__ __forceinline__ void stream(Next next, Done done, int lane) {
        int first, stride, end;
        bool more = next(&first, &stride, &end);
        if (!more) return;
        const int past = (ld + kStepBytes - 1) / kStepBytes;
        Step ring[AHEAD];
        auto fetch = [&](int u, int step) {
            load(ring[u], step < end ? step : past, lane);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) fetch(u, first + u * stride);
        while (more) {
            f32x4 acc[PS];
#pragma unroll
            for (int p = 0; p < PS; ++p) acc[p] = f32x4{0.f, 0.f, 0.f, 0.f};
            const int loaded = groups;   // of this item; next() sets the following one's
            for (bool last = false; !last;) {
                first += AHEAD * stride;
                last = first >= end;
                if (last) {
                    more = next(&first, &stride, &end);
                    if (!more) end = first;   // nothing
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    multiply(ring[u], acc, loaded, lane);
                    fetch(u, first + u * stride);
                }
            }
            done(acc);
        }
    }
};

// ---------------------------------------------------------------- operands through registers into LDS
// For tiles that are too few, or too small, to hide a step's latency: operands are loaded into registers several steps
// ahead (each use waits for its own loads alone) and stored to LDS, which holds two steps.  What bounds many tiles of 128 x 128
// is LDS more than anything else (counters of 2048 x 4096 -> 4096, two workgroups a compute unit: LDS works in 57% of the cycles,
// the matrix cores in 44%, a third of the wavefronts' time is waiting to issue to LDS; operands come at 14 TB/s).  One workgroup a
// compute unit alternates between the two (4096 x 7168 -> 256 in four parts: 40% and 30%, operands at 9 TB/s), and tiles of 64 x 64 wait
// for their steps' latency (64 x 4096 -> 4096 in four parts: 21% and 10%).  There are no bank conflicts.  A third step in LDS, so that fragments are read a barrier ahead, made no difference but for fewer
// workgroups a compute unit.

// R rows of 128 contraction bytes a step for NW wavefronts, in LoadKC's order.
template <int R, int NW>
struct StageKC {
    static constexpr int kN = R / 8 / NW, kBytes = R * kStepBytes;
    static_assert(kN >= 1 && kN * 8 * NW == R, "");
    const char* base;
    int bytes, kbytes;
    uint32_t voff[kN], chunk, at;
    __device__ __forceinline__ void init(const void* b, int ld, int valid, int w, int lane) {
        base = static_cast<const char*>(b);
        bytes = valid * ld;
        kbytes = ld;
        chunk = (lane & 7) * 16;
        at = w * kN * 1024 + (lane >> 3) * kStepBytes + (((lane & 7) ^ (lane >> 3)) << 4);
#pragma unroll
        for (int i = 0; i < kN; ++i) voff[i] = (uint32_t)(((w * kN + i) * 8 + (lane >> 3)) * ld) + chunk;
    }
    __device__ __forceinline__ void load(i32x4 (&r)[kN], int step) const {
        const int from = step * kStepBytes;
        const auto rsrc = descriptor(base + from, from < kbytes ? bytes - from : 0);
        const bool in = (int)chunk < kbytes - from;
#pragma unroll
        for (int i = 0; i < kN; ++i) r[i] = load16(rsrc, in ? voff[i] : kOob);
    }
    __device__ __forceinline__ void store(char* to, const i32x4 (&r)[kN]) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) *reinterpret_cast<i32x4*>(to + at + i * 1024) = r[i];
    }
    __device__ __forceinline__ static bf16x8 frag(const char* stage, int sub, int half, int lane) {
        const int row = sub * 16 + (lane & 15);
        return *reinterpret_cast<const bf16x8*>(stage + (row * kStepBytes + (((half * 4 + (lane >> 4)) ^ (row & 7)) << 4)));
    }
};

// The same of R matrix rows whose subtiles of 16 are a gate's and an up's in turn, each from a panel of its own: a wavefront
// loads one subtile.
template <int R, int NW>
struct StageGated : StageKC<R, NW> {
    using KC = StageKC<R, NW>;
    static_assert(KC::kN == 2, "");
    __device__ __forceinline__ void init(const char* gate, const char* up, int ld, int valid, int w, int lane) {
        KC::init(w & 1 ? up : gate, ld, valid, w >> 1, lane);
        KC::at += (w - (w >> 1)) * KC::kN * 1024;   // where subtile w is in the stage
    }
};

// 64 contraction rows of W columns a step.  Contraction row c's 32-byte unit u (16 columns) sits at u ^ key(c), so that the
// eight rows that a transposing load's 32 lanes read lie in different banks (rows of 256 bytes all begin in the same, of 128
// in two).
template <int W, int NW>
struct StageMC {
    static_assert(W == 64 || W == 128, "");
    static constexpr int kRow = W * 2, kLanes = kRow / 16, kBytes = kStepC * kRow, kN = kBytes / 1024 / NW;
    static_assert(kN >= 1 && kN * 1024 * NW == kBytes, "");
    const char* base;
    int ld, crows, before;   // bytes of a contraction row, contraction rows, bytes of a row before the tile
    uint32_t voff[kN], at[kN];
    __device__ __forceinline__ static int key(int c) { return W == 64 ? (c >> 1 & 1) | (c >> 2 & 2) : (c & 3) | (c >> 1 & 4); }
    __device__ __forceinline__ void init(const void* b, int row_bytes, int n, int col0, int w, int lane) {
        before = col0 * 2;
        base = static_cast<const char*>(b) + before;
        ld = row_bytes;
        crows = n;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = (w * kN + i) * (64 / kLanes) + lane / kLanes, p = lane % kLanes;
            voff[i] = before + p * 16 < row_bytes ? (uint32_t)(c * row_bytes) + p * 16 : kOob;
            at[i] = c * kRow + (((p >> 1) ^ key(c)) << 5) + (p & 1) * 16;
        }
    }
    __device__ __forceinline__ void load(i32x4 (&r)[kN], int step) const {
        const int c0 = step * kStepC;
        const auto rsrc = descriptor(base + (int64_t)c0 * ld, min(crows - c0, kStepC) * ld - before);
#pragma unroll
        for (int i = 0; i < kN; ++i) r[i] = load16(rsrc, voff[i]);
    }
    __device__ __forceinline__ void store(char* to, const i32x4 (&r)[kN]) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) *reinterpret_cast<i32x4*>(to + at[i]) = r[i];
    }
    __device__ __forceinline__ static bf16x8 frag(const char* stage, int sub, int half, int lane) {
        const int g = lane >> 4, t = lane & 15, c = half * 32 + 8 * g + (t >> 2);
        const int from = c * kRow + ((sub ^ key(c)) << 5) + (t & 3) * 8;
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(LDS_PTR(bf16x4, const_cast<char*>(stage) + from));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(LDS_PTR(bf16x4, const_cast<char*>(stage) + (from + 4 * kRow)));
        return bf16x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
};

// A tile of P x Q outputs by WP x WQ wavefronts, AHEAD steps of loads on their way.
template <int P, int Q, int WP, int WQ, int AHEAD, class OpP, class OpQ>
struct StagedBody {
    static constexpr int kWaves = WP * WQ, PS = P / WP / 16, QS = Q / WQ / 16;
    static constexpr int kStage = OpP::kBytes + OpQ::kBytes, kSums = P * Q * 4;
    static constexpr int kLds = 2 * kStage > kSums ? 2 * kStage : kSums;
    static_assert(PS >= 1 && QS >= 1 && AHEAD % 2 == 0, "");

    // Steps [first, last) of the contraction; afterwards the tile's sums are in LDS.
    __device__ __forceinline__ static void run(char* lds, const OpP& lp, const OpQ& lq, int first, int last, int past, int w, int lane) {
        const int wp = w % WP, wq = w / WP;
        f32x4 acc[PS][QS];
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
            for (int q = 0; q < QS; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        i32x4 rp[AHEAD][OpP::kN], rq[AHEAD][OpQ::kN];
        auto fetch = [&](int slot, int step) {   // past the end zeros
            step = step < last ? step : past;
            lp.load(rp[slot], step);
            lq.load(rq[slot], step);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) fetch(s, first + s);
        lp.store(lds, rp[0]);
        lq.store(lds + OpP::kBytes, rq[0]);
        fetch(0, first + AHEAD);
        lds_barrier();
        for (int step = first; step < last; step += AHEAD) {   // whole rounds of both buffers and of the registers
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) {
                const char* cur = lds + (s & 1) * kStage;
                char* nxt = lds + ((s + 1) & 1) * kStage;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    bf16x8 pf[PS], qf[QS];
#pragma unroll
                    for (int p = 0; p < PS; ++p) pf[p] = OpP::frag(cur, wp * PS + p, h, lane);
#pragma unroll
                    for (int q = 0; q < QS; ++q) qf[q] = OpQ::frag(cur + OpP::kBytes, wq * QS + q, h, lane);
#pragma unroll
                    for (int p = 0; p < PS; ++p)
#pragma unroll
                        for (int q = 0; q < QS; ++q) acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[p], qf[q], acc[p][q], 0, 0, 0);
                    if (h == 0) {   // the next step goes into the other buffer, which everyone left at the last barrier
                        lp.store(nxt, rp[(s + 1) % AHEAD]);
                        lq.store(nxt + OpP::kBytes, rq[(s + 1) % AHEAD]);
                        fetch((s + 1) % AHEAD, step + s + 1 + AHEAD);
                    }
                }
                lds_barrier();
            }
        }
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
            for (int q = 0; q < QS; ++q)
                *reinterpret_cast<f32x4*>(lds + sum_at((wq * QS + q) * 16 + (lane & 15), (wp * PS + p) * 4 + (lane >> 4))) = acc[p][q];
        lds_barrier();
    }
    // Of row j's sums, 16-byte chunk c (of row j's first 16 chunks, c ^ j).
    __device__ __forceinline__ static int sum_at(int j, int c) { return j * P * 4 + ((c ^ (j & 15)) << 4); }
    __device__ __forceinline__ static f32x4 sum(const char* lds, int j, int c) { return *reinterpret_cast<const f32x4*>(lds + sum_at(j, c)); }
};

}  // namespace
}  // namespace moe

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
// bf16 products are exact and added in binary32.  The E4M3 matrix instructions (the
// 128-channel one used here and the 32-channel one alike) add the products of eight
// neighbouring channels cut, towards zero, to multiples of 2^(m - 13), m the largest
// exponent sum among the eight; groups are then added in binary32.  Kept, because the
// one way past it is to widen the codes to bf16, at half the matrix rate, and what
// it costs is small: 1.5e-5 of the result for normal codes, where the rounding of the
// output to bf16 costs 1.7e-3.  Block sums are scaled and added in binary32.
//
// Tiles travel from memory to LDS without passing through registers (buffer
// loads with an LDS destination), in two or three stages of 128 contraction
// bytes.  Those loads write LDS in lane order, so the bank swizzle is applied to
// the address each lane reads from.  Out-of-range lanes read zeros (the buffer
// descriptor ends with the tile's valid rows; a lane whose contraction index is
// past the end gets an address past any descriptor), which is what pads ragged
// rows and contraction tails.
//
// From many tiles to few: k_expert_rows (256 columns x up to 256 rows, one
// workgroup a compute unit, scheduled by hand) and k_expert_weights_grad (256 x
// 256, persistent); k_expert_rows_narrow and k_expert_grad_narrow (128 x 128, 128
// x 32 and 64 x 64, two workgroups a compute unit); k_expert_rows_few (16 or 32 columns x
// up to 32 rows, one wavefront, no LDS).  launch_rows() chooses.
//
// What bounds them (MI355X; a large copy moves 4.76 TB/s, a large library
// product does 1.39 PFLOP/s NT, 1.21 NN, 1.08 TN in bf16 and 3.05 in plain fp8):
//   many rows an expert   the matrix cores and the power they may draw: 8192^3
//                         takes 0.78 ms forward (1.41 PFLOP/s, 67-70% of the cycles on the
//                         matrix cores at a clock that falls to 1.5-1.9 GHz), 1.52 ms for both
//                         gradients (1.45 PFLOP/s), 0.50 ms in fp8 with block scales (2.18)
//   few rows an expert    reading the matrices: 1 row an expert 6.2 TB/s, 64 rows 5.6, 128
//                         rows 5.2, 256 rows 4.0 of matrix bytes; what is lost there is the time
//                         of flight of a stage, so smaller tiles get a third stage (of which
//                         most barriers leave one in flight, see lds_barrier())
// Tried and dropped: reading the next steps' lines into L2 ahead (each line once
// 8192^3 0.90 ms against 0.83, shared among the tiles that need it 0.81 against
// 0.80: loads return in order), 32 x 32 x 16 matrix instructions (1.78 PFLOP/s
// from registers alone against 2.01), stages of 64 contraction bytes (15.0 TB/s
// into LDS against 18.4), raised wave priority around the matrix instructions
// (1-3% slower), bands of 2, 8 or 16 row tiles (0-3% slower), tiles of hot and
// cold experts in turn (no change), experts' rows in equal tiles (288 rows 4%
// faster, 416 6% slower), four wavefronts of 128 x 128 (the compiler moves
// accumulators about), staggered workgroups in the weights gradient (no change).
#include "moe_ep.h"
#include "moe_expert.h"
#include "moe_internal.h"

#include <type_traits>

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

// Every descriptor covers one stage of one tile, at most 256 rows of 2 * MOE_MAX_FEATURES bytes.
static_assert(256ll * 2 * MOE_MAX_FEATURES < kOob, "");
__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, max(bytes, 0), 0x00020000);
}

// ---------------------------------------------------------------- segments
struct Tile {
    int e, row, rows;   // expert, first row within its segment, rows of the tile
    int64_t start;      // packed row of the segment's first row
    int col;            // column tile
    bool alone;         // the expert's only row tile
};

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

// Order of the tiles of one matrix with `nj` row tiles and `ni` column tiles: bands of kBand row
// tiles, column by column, so that 32 consecutive tiles touch about 4 + 8 panels.
constexpr int kBand = 4;
__device__ __forceinline__ void band_order(int l, int nj, int ni, int* j, int* i) {
    const int band = l / (kBand * ni), rest = l - band * kBand * ni;
    const int height = min(kBand, nj - band * kBand);
    *i = rest / height;
    *j = band * kBand + rest - *i * height;
}

__device__ __forceinline__ int64_t seg_base(const Segments& s, int e, int64_t start, bool padded) {
    return padded ? (int64_t)e * s.cap + s.first : start;
}

__device__ __forceinline__ int seg_rows(const Segments& s, int lo, int hi) {
    if (!s.ascending(lo, hi)) {
        atomicOr(s.err, kErrBounds);
        return 0;
    }
    return min(hi - lo, s.seg_cap);
}

// Tile t of the launch, where expert e has ceil(rows / bq) x ni of them; e = -1 past the last.
// Every wavefront of the block scans the offsets by itself (E <= 1024: at most 16 per lane).
__device__ __forceinline__ Tile find_tile(const Segments& s, int64_t t, int bq, int ni) {
    constexpr int kPer = (MOE_MAX_EXPERTS + 63) / 64;
    const int lane = threadIdx.x & 63;
    const int per = (s.E + 63) / 64;
    const int e0 = lane * per;
    int off[kPer + 1], own = 0;
#pragma unroll
    for (int u = 0; u <= kPer; ++u)
        if (u <= per) off[u] = s.eoff[min(e0 + u, s.E)];
    int rows[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        if (u >= per) break;
        rows[u] = seg_rows(s, off[u], off[u + 1]);   // past the last expert: none
        own += (rows[u] + bq - 1) / bq;
    }
    int incl = own;
#pragma unroll
    for (int step = 1; step < 64; step <<= 1) {
        const int u = __shfl_up(incl, step, 64);
        if (lane >= step) incl += u;
    }
    const int band = (int)(t / ni);   // row tiles before t's expert are at most this many
    Tile r;
    const uint64_t here = __ballot(band < incl);
    r.e = -1;
    if (here == 0) return r;
    const int owner = __ffsll((unsigned long long)here) - 1;
    int before = incl - own, fe = -1, fbefore = 0, fn = 0, flo = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        if (u >= per) break;
        const int m = (rows[u] + bq - 1) / bq;
        if (fe < 0 && band < before + m) {
            fe = e0 + u;
            fbefore = before;
            fn = rows[u];
            flo = off[u];
        }
        before += m;
    }
    r.e = __builtin_amdgcn_readlane(fe, owner);
    r.start = __builtin_amdgcn_readlane(flo, owner);
    const int n = __builtin_amdgcn_readlane(fn, owner);
    int j;
    band_order((int)(t - (int64_t)__builtin_amdgcn_readlane(fbefore, owner) * ni), (n + bq - 1) / bq, ni, &j, &r.col);
    r.row = j * bq;
    r.alone = n <= bq;
    r.rows = min(bq, n - r.row);
    return r;
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

// ---------------------------------------------------------------- rows products
constexpr int kThreeFp8 = 128;   // rows of the largest fp8 tile with three stages

// A tile of the forward or the rows gradient: rows [row, row + rows) of expert
// e against output columns [i0, i0 + 256).
template <int NW, int BQ, int WP, int STAGES, bool FP8, bool PMC>
__device__ __forceinline__ void rows_tile(const ExpertGemmArgs& a, const Tile& tl, int i0, const Stage (&st)[STAGES],
                                          char* scratch, char* scales, int w, int lane) {
    using B = TileBody<NW, BQ, WP, STAGES, FP8, PMC, false>;
    constexpr int kSize = FP8 ? 1 : 2;
    const int cdim = PMC ? a.N : a.K, idim = PMC ? a.K : a.N;
    const int64_t qrow = seg_base(a.seg, tl.e, tl.start, a.q_padded) + tl.row;
    const int64_t orow = seg_base(a.seg, tl.e, tl.start, a.out_padded) + tl.row;
    const int ni = min(kTileP, idim - i0);
    const char* wmat = static_cast<const char*>(a.p) + (int64_t)tl.e * a.N * a.K * kSize;
    const int64_t qld = (int64_t)cdim * kSize;
    typename B::LQ lq;
    lq.init(static_cast<const char*>(a.q) + qrow * qld, (int)qld, tl.rows, (int)qld, w, lane);
    LoadScales ls;
    f32x4 acc[B::PS][B::QS];
    // Tiles that share a matrix panel in L2 start together.  Only lengths of whole runs of four steps
    // are started elsewhere: others spread over the channels by themselves, and no run is cut short, so
    // that LoadScales never needs a third.  (64 experts x 4 rows, 4096 x 4096 bf16: 371 us, 437 us
    // without.)
    const int n = (cdim * kSize + kStepBytes - 1) / kStepBytes;
    const Steps steps = {n, !PMC && tl.alone && n % 4 == 0 ? ((int)(blockIdx.x & 31) * n / 32) & ~3 : 0};
    if constexpr (FP8) {
        const int kb = a.K / 128, nb = (a.N + 127) / 128;
        ls.init(a.q_scales + qrow * kb, tl.rows, a.p_scales + ((int64_t)tl.e * nb + i0 / 128) * kb, nb - i0 / 128, kb,
                scales, BQ > kThreeFp8 ? -1024 : kThreeFp8 * 16, w, lane);
    }
    if constexpr (PMC) {
        LoadMC<NW> lp;
        lp.init(wmat, a.K * 2, a.N, i0, w, lane);
        B::begin(st, lp, lq, ls, steps);
        B::run(st, lp, lq, ls, steps, acc, w, lane);
    } else {
        typename B::LP lp;
        lp.init(wmat + i0 * qld, (int)qld, ni, (int)qld, w, lane);
        B::begin(st, lp, lq, ls, steps);
        B::run(st, lp, lq, ls, steps, acc, w, lane);
    }
    lds_barrier();   // the epilogue's LDS was a stage
    B::store(static_cast<uint16_t*>(a.out) + orow * idim + i0, idim, ni, tl.rows, acc, scratch, w, lane);
}

// ---------------------------------------------------------------- few rows
// A token or a few: one wavefront multiplies 16 or 32 columns with up to 32 rows, and no operand passes
// through LDS, so nothing is waited for but the wavefront's own loads.  The lanes of a matrix
// instruction read 64 contiguous bytes of 16 matrix rows; 512 bytes of each row are on their way.
// What bounds it is reading the matrices (201 MB alone take 35-39 us, 5.2-5.8 TB/s), and from about 16 rows
// on the loads of the rows, which every wavefront repeats.  A token with 6 experts of 4096 x 4096 bf16 takes
// 38 us (5.4 TB/s; 51 in the narrow tiles below), with 6 of 2048 x 7168 32 us (76), with 2 of 4096 x 4096 16 us (44).

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)off, 0, 0));
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)off, 0, 0));
}

// PS x QS subtiles of 16 x 16.
template <bool FP8, int PS, int QS>
struct FewBody {
    // contraction bytes of one matrix instruction, and instructions that are loaded for ahead
    static constexpr int kUnit = FP8 ? 128 : 64, kRing = 512 / kUnit, kChunks = kUnit / 64;
    struct Unit {
        i32x4 p[PS][kChunks], q[QS][kChunks];
        float m, s[QS];   // fp8: scale of the column block, of the rows
    };
    __amdgpu_buffer_rsrc_t rp, rq, rm, rs;
    int ld;   // bytes of a row

    // Unit u of the lane's columns and rows; zeros past the row's end, as past the last row.  fp8 takes
    // chunks g and g + 4 of 128 channels, for both operands.
    __device__ __forceinline__ void load(Unit& x, int u, int lane) const {
        const int at = u * kUnit + (lane >> 4) * 16, t = lane & 15;
        const bool in = at < ld;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const uint32_t off = in ? (uint32_t)(t * ld + at + c * 64) : kOob, sub = (uint32_t)(16 * ld);
#pragma unroll
            for (int p = 0; p < PS; ++p) x.p[p][c] = load16(rp, off + p * sub);
#pragma unroll
            for (int q = 0; q < QS; ++q) x.q[q][c] = load16(rq, off + q * sub);
        }
        if constexpr (FP8) {
            x.m = load4(rm, in ? (uint32_t)u * 4 : kOob);
#pragma unroll
            for (int q = 0; q < QS; ++q) x.s[q] = load4(rs, in ? (uint32_t)((t + 16 * q) * (ld / 128) + u) * 4 : kOob);
        }
    }
    __device__ __forceinline__ static i32x8 join(const i32x4 (&v)[kChunks]) {
        return i32x8{v[0].x, v[0].y, v[0].z, v[0].w, v[kChunks - 1].x, v[kChunks - 1].y, v[kChunks - 1].z, v[kChunks - 1].w};
    }
    __device__ __forceinline__ void run(f32x4 (&acc)[PS][QS], int lane) const {
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
            for (int q = 0; q < QS; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        // The loads stay in this order (the scheduler is fenced off), so that a use waits for its own only.
        Unit ring[kRing];
#pragma unroll
        for (int u = 0; u < kRing; ++u) {
            load(ring[u], u, lane);
            __builtin_amdgcn_sched_barrier(0);
        }
        for (int first = 0; first * kUnit < ld; first += kRing) {
#pragma unroll
            for (int u = 0; u < kRing; ++u) {
                Unit& x = ring[u];
#pragma unroll
                for (int p = 0; p < PS; ++p)
#pragma unroll
                    for (int q = 0; q < QS; ++q) {
                        if constexpr (FP8) {
                            const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                join(x.p[p]), join(x.q[q]), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
                            const float sc = x.s[q] * x.m;
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[p][q][r] = __builtin_fmaf(d[r], sc, acc[p][q][r]);
                        } else {
                            acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8, x.p[p][0]), __builtin_bit_cast(bf16x8, x.q[q][0]), acc[p][q], 0, 0, 0);
                        }
                    }
                load(x, first + kRing + u, lane);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
};

template <bool FP8, int PS, int QS>
__device__ __forceinline__ void few_tile(const ExpertGemmArgs& a, const Tile& tl, int lane) {
    constexpr int kSize = FP8 ? 1 : 2;
    const int i0 = tl.col * PS * 16;
    const int64_t qrow = seg_base(a.seg, tl.e, tl.start, a.q_padded) + tl.row;
    const int64_t orow = seg_base(a.seg, tl.e, tl.start, a.out_padded) + tl.row;
    FewBody<FP8, PS, QS> b;
    b.ld = a.K * kSize;
    b.rp = descriptor(static_cast<const char*>(a.p) + ((int64_t)tl.e * a.N + i0) * b.ld, min(PS * 16, a.N - i0) * b.ld);
    b.rq = descriptor(static_cast<const char*>(a.q) + qrow * b.ld, tl.rows * b.ld);
    if constexpr (FP8) {
        const int kb = a.K / 128, nb = (a.N + 127) / 128;
        b.rm = descriptor(a.p_scales + ((int64_t)tl.e * nb + i0 / 128) * kb, kb * 4);
        b.rs = descriptor(a.q_scales + qrow * kb, tl.rows * kb * 4);
    }
    f32x4 acc[PS][QS];
    b.run(acc, lane);
#pragma unroll
    for (int p = 0; p < PS; ++p)
#pragma unroll
        for (int q = 0; q < QS; ++q) {
            const int i = i0 + 16 * p + 4 * (lane >> 4), j = q * 16 + (lane & 15);
            if (i < a.N && j < tl.rows)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + (orow + j) * a.N + i) = bf16_pack(acc[p][q]);
        }
}

// Tiles of 16 * PS columns and up to 16 * QS rows.
template <bool FP8, int PS, int QS>
__global__ __launch_bounds__(64, 2) void k_expert_rows_few(ExpertGemmArgs a) {
    const Tile tl = find_tile(a.seg, xcd_tile4((int)blockIdx.x), 16 * QS, (a.N + PS * 16 - 1) / (PS * 16));
    if (tl.e < 0) return;
    if (QS > 1 && tl.rows > 16) few_tile<FP8, PS, QS>(a, tl, threadIdx.x);
    else few_tile<FP8, PS, 1>(a, tl, threadIdx.x);
}

// ---------------------------------------------------------------- narrow tiles
// Narrow tiles for products with too few 256-column tiles to occupy the chip: 128 columns x 32 or 128 rows, or 64 x
// 64; two workgroups a compute unit (64 to 80 KB of stages each), so that one computes while the other waits.  Steps are not
// scheduled by hand.  4096 x 4096 bf16, 1 expert: 512 rows 46 us (0.38 PFLOP/s, 64 x 64), 2048 rows
// 76 us (0.90, 128 x 128); bound by the latency of a step.  LDS holds one step ahead (128 x 128), two (fp8, 128 x 32) or
// three, but one is in flight: the barrier of a step waits for all loads (see lds_barrier()).
template <bool FP8, int P, int Q, int NW, int STAGES>
struct NarrowBody {
    using LP = LoadKC<P, NW, !FP8>;
    using LQ = LoadKC<Q, NW, !FP8>;
    static constexpr int WP = P / 32, WQ = NW / WP, QS = Q / 16 / WQ;   // a wavefront owns 32 columns x 16 QS rows
    static_assert(WP * WQ == NW && QS * WQ * 16 == Q && NW >= 4, "");
    static constexpr int kRowScales = (Q + 63) / 64 * 256;              // bytes; then the column block's
    static constexpr int kScales = FP8 ? kRowScales + 256 : 0;
    static constexpr int kStage = (P + Q) * kStepBytes + kScales;
    static constexpr int kLds = kStage * STAGES;

    // Scales of one stage: the rows', and the one of the tile's 128-column block.
    struct Scales {
        __amdgpu_buffer_rsrc_t rsrc;
        uint32_t voff;
        int kb, lds;
        __device__ __forceinline__ void init(const float* rows, int valid, const float* mat, int kblocks, int w, int lane) {
            kb = kblocks;
            const int part = w & 3;   // wavefront 0 loads 64 rows', 1 the next 64's, if there are, 2 and 3 the block's
            const bool r = part * 256 < kRowScales;
            rsrc = r ? descriptor(rows, valid * kb * 4) : descriptor(mat, kb * 4);
            voff = r ? (uint32_t)((part * 64 + lane) * kb) * 4 : lane == 0 ? 0 : kOob;
            lds = r ? part * 256 : kRowScales;
        }
        __device__ __forceinline__ void issue(char* stage, int step) const {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, LDS_PTR(void, stage + lds), 4, step < kb ? voff + step * 4 : kOob, 0,
                                                     0, 0);
        }
    };

    __device__ __forceinline__ static void run(char* lds, const LP& lp, const LQ& lq, const Scales& ls, const Steps& order,
                                               f32x4 (&acc)[2][QS], int w, int lane) {
        constexpr int kLoads = LP::kInstr + LQ::kInstr + (FP8 ? 1 : 0);
        const int g = lane >> 4, t = lane & 15, wp = w % WP, wq = w / WP;
        auto fill = [&](int turn, int slot) {
            char* st = lds + slot * kStage;
            const int step = order.at(turn);   // past the end it reads nothing
            const auto sp = lp.step_of(step);
            const auto sq = lq.step_of(step);
#pragma unroll
            for (int l = 0; l < LP::kInstr; ++l) lp.issue(st, sp, l);
#pragma unroll
            for (int l = 0; l < LQ::kInstr; ++l) lq.issue(st + P * kStepBytes, sq, l);
            if constexpr (FP8) ls.issue(st + (P + Q) * kStepBytes, step);
        };
#pragma unroll
        for (int q = 0; q < QS; ++q) acc[0][q] = acc[1][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) fill(s, s);
        int cur = 0, nxt = STAGES - 1;
        for (int turn = 0; turn < order.n; ++turn) {
            wait_loads<(STAGES - 2) * kLoads>();
            lds_barrier();   // this step has arrived, and everyone is done with the one before
            fill(turn + STAGES - 1, nxt);
            const char* sp = lds + cur * kStage;
            const char* sq = sp + P * kStepBytes;
            if constexpr (FP8) {
                const char* sc = sq + Q * kStepBytes;
                i32x8 pf[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) pf[p] = LP::frag8(sp, wp * 32 + p * 16 + t, g);
#pragma unroll
                for (int q = 0; q < QS; ++q) {
                    const int row = (wq * QS + q) * 16 + t;
                    const i32x8 qf = LQ::frag8(sq, row, g);
                    const float s =
                        *reinterpret_cast<const float*>(sc + row * 4) * *reinterpret_cast<const float*>(sc + kRowScales);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            pf[p], qf, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[p][q][r] = __builtin_fmaf(d[r], s, acc[p][q][r]);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    bf16x8 pf[2];
#pragma unroll
                    for (int p = 0; p < 2; ++p) pf[p] = LP::frag(sp, wp * 32 + p * 16 + t, h * 4 + g);
#pragma unroll
                    for (int q = 0; q < QS; ++q) {
                        const bf16x8 qf = LQ::frag(sq, (wq * QS + q) * 16 + t, h * 4 + g);
#pragma unroll
                        for (int p = 0; p < 2; ++p)
                            acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[p], qf, acc[p][q], 0, 0, 0);
                    }
                }
            }
            cur = cur == STAGES - 1 ? 0 : cur + 1;
            nxt = nxt == STAGES - 1 ? 0 : nxt + 1;
        }
        wait_loads<0>();   // nothing may be on its way into LDS when the workgroup ends
    }
};

template <bool FP8, int P, int Q, int NW, int STAGES>
__global__ __launch_bounds__(64 * NW) void k_expert_rows_narrow(ExpertGemmArgs a) {
    using B = NarrowBody<FP8, P, Q, NW, STAGES>;
    __shared__ __align__(1024) char lds[B::kLds];
    constexpr int kSize = FP8 ? 1 : 2;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Tile tl = find_tile(a.seg, xcd_tile4((int)blockIdx.x), Q, (a.N + P - 1) / P);
    if (tl.e < 0) return;
    const int i0 = tl.col * P, ni = min(P, a.N - i0);
    const int64_t qrow = seg_base(a.seg, tl.e, tl.start, a.q_padded) + tl.row;
    const int64_t orow = seg_base(a.seg, tl.e, tl.start, a.out_padded) + tl.row;
    const int64_t ld = (int64_t)a.K * kSize;
    typename B::LP lp;
    typename B::LQ lq;
    typename B::Scales ls;
    lp.init(static_cast<const char*>(a.p) + ((int64_t)tl.e * a.N + i0) * ld, (int)ld, ni, (int)ld, w, lane);
    lq.init(static_cast<const char*>(a.q) + qrow * ld, (int)ld, tl.rows, (int)ld, w, lane);
    if constexpr (FP8) {
        const int kb = a.K / 128, nb = (a.N + 127) / 128;
        ls.init(a.q_scales + qrow * kb, tl.rows, a.p_scales + ((int64_t)tl.e * nb + i0 / 128) * kb, kb, w, lane);
    }
    f32x4 acc[2][B::QS];
    // matrices read by one row tile: workgroups of an XCD start at different columns, as in rows_tile()
    const int n = (int)((ld + kStepBytes - 1) / kStepBytes);
    const Steps steps = {n, tl.alone ? (int)(blockIdx.x >> 3 & 31) * n / 32 : 0};
    B::run(lds, lp, lq, ls, steps, acc, w, lane);
#pragma unroll
    for (int q = 0; q < B::QS; ++q) {
        const int j = (w / B::WP * B::QS + q) * 16 + (lane & 15);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int i = (w % B::WP) * 32 + p * 16 + 4 * (lane >> 4);
            if (j < tl.rows && i < ni)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + (orow + j) * a.N + i0 + i) = bf16_pack(acc[p][q]);
        }
    }
}

constexpr int kTileBytes = 256 * kStepBytes;   // of one operand's stage
constexpr int kWaves = 8;                      // of a workgroup (one workgroup a compute unit)

constexpr int max_of(int a, int b) { return a > b ? a : b; }

template <bool FP8, bool PMC>
__global__ __launch_bounds__(64 * kWaves, kWaves / 4) void k_expert_rows(ExpertGemmArgs a) {
    // Two stages of up to 256 rows, or three of up to kThree; the epilogue uses a part.  The compiler
    // orders LDS reads after the loads into LDS that it takes to reach them: plain reads where it knows
    // one array for both, transposing reads also where it knows none.  Which loads have arrived is what
    // the waits in step_of() say; to keep it from waiting for more, plain reads see one unnamed block
    // and transposing ones an array for each stage and operand.
    constexpr int kThree = PMC ? 64 : FP8 ? kThreeFp8 : 160, kQ = kThree * kStepBytes;
    Stage two[2], three[3];
    char* scales = nullptr;
    if constexpr (PMC) {
        __shared__ __align__(1024) char p0[kTileBytes], p1[kTileBytes], r0[kTileBytes], r1[kTileBytes], q0[kQ], q1[kQ], q2[kQ];
        two[0] = {p0, r0};
        two[1] = {p1, r1};
        three[0] = {p0, q0};
        three[1] = {p1, q1};
        three[2] = {r0, q2};
    } else {
        constexpr int kTiles = max_of(4 * kTileBytes, 3 * (kTileBytes + kQ));
        __shared__ __align__(1024) char lds[kTiles + (FP8 ? LoadScales::kBytes : 0)];
        char* q = lds + 3 * kTileBytes;
        two[0] = {lds, lds + 2 * kTileBytes};
        two[1] = {lds + kTileBytes, q};
        three[0] = {lds, q};
        three[1] = {lds + kTileBytes, q + kQ};
        three[2] = {lds + 2 * kTileBytes, q + 2 * kQ};
        scales = lds + kTiles;
        // LoadScales's unused kilobyte: before the scales of two stages, behind the rows of three
        static_assert(!FP8 || (kTiles >= 4 * kTileBytes + 1024 && kThreeFp8 * 16 + 1024 <= 4096), "");
    }
    static_assert(kTileBytes >= kWaves * 2048, "");
    char* scratch = two[0].p;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int ntiles = ((PMC ? a.K : a.N) + kTileP - 1) / kTileP;
    const Tile tl = find_tile(a.seg, xcd_tile(blockIdx.x), 256, ntiles);
    if (tl.e < 0) return;
    const int i0 = tl.col * kTileP;
    // The smallest tile that holds the rows.  A third stage pays where reading the matrix is the bound
    // (forward, 64 experts of 4096 x 4096: 128 rows 413 us, with two stages 524; 160 rows 447, as 192 rows
    // with two 495); fp8's scales leave it room up to 128 rows, the transposed operand's separate
    // arrays up to 64.
    if (tl.rows > 192) rows_tile<kWaves, 256, 2, 2, FP8, PMC>(a, tl, i0, two, scratch, scales, w, lane);
    else if (tl.rows > (PMC ? 128 : 160)) rows_tile<kWaves, 192, 2, 2, FP8, PMC>(a, tl, i0, two, scratch, scales, w, lane);
    else if (!PMC && !FP8 && tl.rows > 128) rows_tile<kWaves, kThree, 4, 3, FP8, PMC>(a, tl, i0, three, scratch, scales, w, lane);
    else if (FP8 && tl.rows > 128) rows_tile<kWaves, 160, 4, 2, FP8, PMC>(a, tl, i0, two, scratch, scales, w, lane);
    else if (PMC && tl.rows > 64) rows_tile<kWaves, 128, 4, 2, FP8, PMC>(a, tl, i0, two, scratch, scales, w, lane);
    else if (tl.rows > 64) rows_tile<kWaves, PMC ? 64 : 128, 4, 3, FP8, PMC>(a, tl, i0, three, scratch, scales, w, lane);
    else if (tl.rows > 32) rows_tile<kWaves, 64, 4, 3, FP8, PMC>(a, tl, i0, three, scratch, scales, w, lane);
    else rows_tile<kWaves, 32, 8, 3, FP8, PMC>(a, tl, i0, three, scratch, scales, w, lane);
}

// ---------------------------------------------------------------- weights gradient
// Four results at element o of the output, in its type, added to what it holds if asked.
__device__ __forceinline__ void put(const ExpertGemmArgs& a, int64_t o, f32x4 v) {
    if (a.out_f32) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o);
        *d = a.accumulate ? *d + v : v;
        return;
    }
    u32x2* d = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + o);
    if (a.accumulate) {
        const u32x2 old = *d;
        v += f32x4{__uint_as_float(old.x << 16), __uint_as_float(old.x & 0xffff0000u), __uint_as_float(old.y << 16),
                   __uint_as_float(old.y & 0xffff0000u)};
    }
    *d = bf16_pack(v);
}

// Experts with rows (or without), by number.  A lane knows min(16, ceil(E / 64)) of them.
struct ExpertList {
    uint32_t mask;   // bit u: the lane's expert u is in the list
    int incl;        // experts in the list up to the lane's last
    int per;
    __device__ __forceinline__ void init(const Segments& s, bool with_rows, int lane) {
        constexpr int kPer = (MOE_MAX_EXPERTS + 63) / 64;
        per = (s.E + 63) / 64;
        int off[kPer + 1];
#pragma unroll
        for (int u = 0; u <= kPer; ++u)
            if (u <= per) off[u] = s.eoff[min(lane * per + u, s.E)];
        mask = 0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (u >= per) break;
            if (lane * per + u < s.E && (seg_rows(s, off[u], off[u + 1]) > 0) == with_rows) mask |= 1u << u;
        }
        incl = __popc(mask);
#pragma unroll
        for (int step = 1; step < 64; step <<= 1) {
            const int u = __shfl_up(incl, step, 64);
            if (lane >= step) incl += u;
        }
    }
    __device__ __forceinline__ int count() const { return __builtin_amdgcn_readlane(incl, 63); }
    // The n-th, n < count().
    __device__ __forceinline__ int at(int n) const {
        const int owner = __ffsll((unsigned long long)__ballot(n < incl)) - 1;
        uint32_t m = __builtin_amdgcn_readlane(mask, owner);
        for (int skip = n - __builtin_amdgcn_readlane(incl, owner) + __popc(m); skip > 0; --skip) m &= m - 1;
        return owner * per + __ffs(m) - 1;
    }
};

// Tiles of 256 x 256 over the matrices of experts with rows; those of the others are zeroed as one run of
// memory (160 experts of 2320 x 624 with 2 rows in all: 463 MB, 90 us, as tiles of zeros 225).  With few rows an
// expert it is bound by writing the gradients: 64 matrices of 4096 x 4096 take 0.39 ms at 4 rows each (5.5 TB/s
// written), 0.54 at 128, 1.64 at 768 (1.01 PFLOP/s), 3.6 at 2048 (1.21).  That is bf16, written, of matrices of 256
// tiles, so that every workgroup gets one tile of each expert.  Other matrices share out less evenly: 49,152 rows over 64
// experts with popularity falling as rank^-1.2, 1536 x 2048, 0.40 ms, 0.33 with equal popularity; 128 experts 0.50 and 0.44;
// 2816 x 2048 0.62 and 0.59.  Other results cost more, for put() loads, adds and stores 32 times one after the other,
// behind the next tile's loads: skewed 4096 x 4096 1.78 ms, fp32 2.18, added to bf16 2.57, added to fp32 2.94; at 128 rows
// each 0.66, 1.21, 1.64 and 2.01.
constexpr int kWeightsGradBlocks = 256;
constexpr int kZeroChunk = 64 * 1024;   // bytes of zeros a workgroup writes in turn

__global__ __launch_bounds__(64 * kWaves, kWaves / 4) void k_expert_weights_grad(ExpertGemmArgs a) {
    using B = TileBody<kWaves, 256, 2, 2, false, true, true>;
    __shared__ __align__(1024) char p0[kTileBytes], p1[kTileBytes], q0[kTileBytes], q1[kTileBytes];
    __shared__ __align__(1024) char scratch[kWaves * 2048];
    const Stage st[2] = {{p0, q0}, {p1, q1}};
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int kt = (a.K + kTileP - 1) / kTileP, nt = (a.N + 255) / 256;
    ExpertList list;
    list.init(a.seg, true, lane);
    const int64_t tiles = (int64_t)list.count() * kt * nt;
    auto zero = [&] {
        if (a.accumulate || list.count() == a.seg.E) return;
        ExpertList none;
        none.init(a.seg, false, lane);
        const int64_t bytes = (int64_t)a.N * a.K * (a.out_f32 ? 4 : 2), chunks = (bytes + kZeroChunk - 1) / kZeroChunk;
        for (int64_t c = blockIdx.x; c < none.count() * chunks; c += kWeightsGradBlocks) {
            const int n = (int)(c / chunks);
            const int64_t from = (c - n * chunks) * kZeroChunk, to = min(from + kZeroChunk, bytes);
            char* out = static_cast<char*>(a.out) + none.at(n) * bytes;
            for (int64_t b = from + threadIdx.x * 16; b < to; b += 64 * kWaves * 16)
                __builtin_nontemporal_store(i32x4{0, 0, 0, 0}, reinterpret_cast<i32x4*>(out + b));
        }
    };
    // half of the workgroups begin with the zeros, so that they are written while the others multiply
    const bool first = (blockIdx.x >> 3) & 1;
    if (first) zero();
    LoadMC<kWaves> lp, lq;
    LoadScales ls;   // none
    Steps steps;
    int e, i0, j0;
    auto start = [&](int64_t t, int ln) {
        const int n = (int)(t / (kt * nt));
        e = list.at(n);
        int ti, tj;
        band_order((int)(t - (int64_t)n * kt * nt), nt, kt, &tj, &ti);
        i0 = ti * kTileP;
        j0 = tj * 256;
        const int lo = a.seg.eoff[e];
        const int rows = seg_rows(a.seg, lo, a.seg.eoff[e + 1]);
        const int64_t prow = seg_base(a.seg, e, lo, a.p_padded), qrow = seg_base(a.seg, e, lo, a.q_padded);
        lp.init(static_cast<const char*>(a.p) + (rows ? prow * a.K * 2 : 0), a.K * 2, rows, i0, w, ln);
        lq.init(static_cast<const char*>(a.q) + (rows ? qrow * a.N * 2 : 0), a.N * 2, rows, j0, w, ln);
        steps = Steps{(rows + kStepC - 1) / kStepC, 0};
        B::begin(st, lp, lq, ls, steps);
    };
    // Each workgroup takes every kWeightsGradBlocks-th tile, and starts the next one's loads before it
    // stores (the next tile's first barrier waits for those loads and for the stores).
    int64_t t = xcd_tile(blockIdx.x);
    if (t < tiles) start(t, lane);
    while (t < tiles) {
        f32x4 acc[B::PS][B::QS];
        B::run(st, lp, lq, ls, steps, acc, w, lane);
        const int64_t at = ((int64_t)e * a.N + j0) * a.K + i0;
        const int ni = min(kTileP, a.K - i0), nj = min(256, a.N - j0);
        t += kWeightsGradBlocks;
        int ln = lane;
        asm volatile("" : "+v"(ln));   // what depends on the lane is computed anew: kept over the loop it would spill
        if (t < tiles) {
            lds_barrier();   // everyone is done with the stages
            start(t, ln);
        }
        if (a.accumulate || a.out_f32) {
            const int wp = w % 2, wq = w / 2, g = ln >> 4, tt = ln & 15;
#pragma unroll
            for (int q = 0; q < B::QS; ++q) {
                const int j = wq * B::QS * 16 + q * 16 + tt;
#pragma unroll
                for (int p = 0; p < B::PS; ++p) {
                    const int i = wp * B::PS * 16 + 16 * p + 4 * g;
                    if (j < nj && i < ni) put(a, at + (int64_t)j * a.K + i, acc[p][q]);
                }
            }
        } else {
            B::store(static_cast<uint16_t*>(a.out) + at, a.K, ni, nj, acc, scratch, w, ln);
        }
    }
    if (!first) zero();
}

// ---------------------------------------------------------------- gradients of few tiles
// The gradients in 128 x 128 tiles, two workgroups a compute unit, for the cases that the forward product's
// narrow tiles are for.  Rows gradient, against 256 columns, us: 4096 x 4096, 1 expert with 512 rows 51 and 87, 4 with
// 256 55 and 100, 1 with 2048 69 and 101.  Weights gradient: 1 x 4096 rows, 1024 x 1024, 50 and 75; 24 x 580 rows, 168 x
// 440, 11 and 23; 8 x 300 rows, 1024 x 512, 8.4 and 16.  Up to kNarrowTiles of them, which run together; the rows
// gradient only where 256 columns leave compute units idle.
constexpr int kNarrowGrad = 128;

template <bool WEIGHTS>
__device__ __forceinline__ void grad_narrow(const ExpertGemmArgs& a, const Stage (&st)[2], int w, int lane) {
    constexpr int T = kNarrowGrad, WP = T / 32, WQ = kWaves / WP, QS = T / 16 / WQ;
    using LP = LoadMC<kWaves, T>;
    using LQ = typename std::conditional<WEIGHTS, LP, LoadKC<T, kWaves, true>>::type;
    static_assert(LP::kBytes == T * kStepBytes && LQ::kBytes == T * kStepBytes, "");
    const int kt = (a.K + T - 1) / T;
    LP lp;
    LQ lq;
    int steps, i0, ni, nj;
    int64_t at;   // first output
    if constexpr (WEIGHTS) {
        const int nt = (a.N + T - 1) / T, t = xcd_tile4((int)blockIdx.x), e = t / (kt * nt);
        if (e >= a.seg.E) return;
        int ti, tj;
        band_order(t - e * kt * nt, nt, kt, &tj, &ti);
        i0 = ti * T;
        const int j0 = tj * T, lo = a.seg.eoff[e];
        const int rows = seg_rows(a.seg, lo, a.seg.eoff[e + 1]);   // none: the tile is zeroed
        const int64_t prow = seg_base(a.seg, e, lo, a.p_padded), qrow = seg_base(a.seg, e, lo, a.q_padded);
        lp.init(static_cast<const char*>(a.p) + (rows ? prow * a.K * 2 : 0), a.K * 2, rows, i0, w, lane);
        lq.init(static_cast<const char*>(a.q) + (rows ? qrow * a.N * 2 : 0), a.N * 2, rows, j0, w, lane);
        steps = (rows + kStepC - 1) / kStepC;
        nj = a.N - j0;
        at = ((int64_t)e * a.N + j0) * a.K + i0;
    } else {
        const Tile tl = find_tile(a.seg, xcd_tile4((int)blockIdx.x), T, kt);
        if (tl.e < 0) return;
        i0 = tl.col * T;
        const int64_t qrow = seg_base(a.seg, tl.e, tl.start, a.q_padded) + tl.row;
        lp.init(static_cast<const char*>(a.p) + (int64_t)tl.e * a.N * a.K * 2, a.K * 2, a.N, i0, w, lane);
        lq.init(static_cast<const char*>(a.q) + qrow * a.N * 2, a.N * 2, tl.rows, a.N * 2, w, lane);
        steps = (a.N + kStepC - 1) / kStepC;
        nj = tl.rows;
        at = (seg_base(a.seg, tl.e, tl.start, a.out_padded) + tl.row) * a.K + i0;
    }
    ni = a.K - i0;
    const int g = lane >> 4, t = lane & 15, wp = w % WP, wq = w / WP;
    f32x4 acc[2][QS];
#pragma unroll
    for (int q = 0; q < QS; ++q) acc[0][q] = acc[1][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto fill = [&](const Stage& to, int step) {
        const auto sp = lp.step_of(step);
        const auto sq = lq.step_of(step);
#pragma unroll
        for (int l = 0; l < LP::kInstr; ++l) lp.issue(to.p, sp, l);
#pragma unroll
        for (int l = 0; l < LQ::kInstr; ++l) lq.issue(to.q, sq, l);
    };
    auto one = [&](const Stage& cur, const Stage& nxt, int step) {
        wait_loads<0>();
        lds_barrier();          // this step has arrived, and everyone is done with the one before
        fill(nxt, step + 1);    // past the end it reads nothing
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 pf[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) pf[p] = LP::frag(cur.p, wp * 2 + p, h * 32, lane);
#pragma unroll
            for (int q = 0; q < QS; ++q) {
                bf16x8 qf;
                if constexpr (WEIGHTS) qf = LQ::frag(cur.q, wq * QS + q, h * 32, lane);
                else qf = LQ::frag(cur.q, (wq * QS + q) * 16 + t, h * 4 + g);
#pragma unroll
                for (int p = 0; p < 2; ++p) acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[p], qf, acc[p][q], 0, 0, 0);
            }
        }
    };
    fill(st[0], 0);
    int step = 0;
    for (; step + 1 < steps; step += 2) {
        one(st[0], st[1], step);
        one(st[1], st[0], step + 1);
    }
    if (step < steps) one(st[0], st[1], step);
    wait_loads<0>();   // nothing may be on its way into LDS when the workgroup ends
#pragma unroll
    for (int q = 0; q < QS; ++q) {
        const int j = (wq * QS + q) * 16 + t;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int i = wp * 32 + p * 16 + 4 * g;
            if (j < nj && i < ni) put(a, at + (int64_t)j * a.K + i, acc[p][q]);
        }
    }
}

template <bool WEIGHTS>
__global__ __launch_bounds__(64 * kWaves, kWaves / 2) void k_expert_grad_narrow(ExpertGemmArgs a) {
    constexpr int kBytes = kNarrowGrad * kStepBytes;
    __shared__ __align__(1024) char p0[kBytes], p1[kBytes], q0[kBytes], q1[kBytes];
    const Stage st[2] = {{p0, q0}, {p1, q1}};
    grad_narrow<WEIGHTS>(a, st, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), threadIdx.x & 63);
}

// Upper bound on the tiles of a launch: every `bq` rows, and one ragged end for each expert with rows.
int64_t tile_bound(const ExpertGemmArgs& a, int64_t pairs, int bq, int64_t ni) {
    return (pairs / bq + (pairs < a.seg.E ? pairs : a.seg.E)) * ni;
}

// A grid holds under 2^32 threads.
bool grid_fits(int64_t blocks, int threads) { return blocks * threads < ((int64_t)1 << 32); }

// Which kernel a forward product runs on, from the numbers of its tiles, were its rows spread evenly over the
// experts (as many as there are rows, at most): the smallest tiles that still run together.  Cold matrices, us, against the
// best of the others.
//   128 columns x 32 rows, a mean of up to 32 rows, between half of the workgroups that run together and all:
//     4096 x 4096 bf16, 10 / 12 / 16 experts of 1 row 63 / 72 / 94 against 68 / 78 / 97, 8 of 16 rows 56 against 62, 9 of 32
//     rows 66 against 76; fp8, 2048 x 7168, 8 x 8 rows 23 against 27.  More only in fp8 and with few rows: 7168 x 4096,
//     256 x 4 rows 1211 against 1274, popularity falling as rank^-1.2 1322 against 1337 (mean 8), 1661 against 1404 (mean 30);
//     bf16, 4096 x 4096, 64 x 4 rows 350 against 353, falling popularity (mean 8) 375 against 363.
//   16 (fp8: 32) columns x 16 rows of one wavefront, a mean of up to 8 rows:
//     bf16   4096 x 4096, 1 row each, 2 / 6 / 8 / 10 experts: 16 / 37 / 57 / 68 against 44 / 51 / 56 / 63
//     fp8    2048 x 7168, 1 row each, 6 / 8 / 10 / 12 experts: 20 / 24 / 30 / 35 against 20 / 23 / 39 / 46; 2048 x 2048, 16 x 1
//            row 15 against 17; 7168 x 4096, 16 x 1 row 87 against 84.  fp8 takes them once more, from where 128 columns x 32
//            rows begin a second round of workgroups (more than 512) to where that has made up for it: 1 row each, 560 / 704 /
//            760 tiles of 128 x 32, out of cold caches, in columns 2048: rows of 6144 143 / 160 / 172 against 168 / 174 / 176,
//            4224 116 / 128 / 136 against 132 / 136 / 139, 8192 184 / 207 / 217 against 199 / 207 / 211, 12288 248 / 282 / 305
//            against 272 / 282 / 286; alike at 1024, 2048, 3968, 5120, 7168, 10240 and 16384 and with 8 rows each.  Rows of
//            4096 bytes lose by it, 126 / 140 / 146 against 125 / 130 / 131: these tiles all start at one column.
//   32 columns x 32 rows of one wavefront: 4096 x 4096 bf16, 2 / 4 / 6 experts of 32 rows 19 / 41 / 62 against 45 / 48 / 53, of
//     16 rows 16 / 34 / 54 against 44 / 48 / 52; 1 expert of 64 rows 18 against 42.
//   64 x 64: 4096 x 4096 bf16, 1 x 512 rows 46, 128 x 128 57, 256 columns 90; beyond, 9 x 64 rows 108 / 82 / 83.
//   128 x 128, where 256 columns would leave compute units idle: 4096 x 4096 bf16, 4 x 256 rows 64 against 103, 1 x 2048
//     rows 76 against 102; with more tiles, 12 x 256 rows 171 against 128; where 256 columns fill the chip, 16 x 64 rows
//     about 130 against 101.  fp8 with half of a tile's rows idle: 9 x 64 rows 57 against 48.
constexpr int kFewMean = 8;
constexpr int64_t kFew = 1024, kFewFp8 = 2816, kFewTiles = 640, kNarrowTiles = 512, kWideTiles = 256;

template <bool FP8, int PS, int QS>
hipError_t launch_few(const ExpertGemmArgs& a, int64_t pairs, hipStream_t s) {
    const int64_t blocks = (tile_bound(a, pairs, 16 * QS, (a.N + PS * 16 - 1) / (PS * 16)) + 31) / 32 * 32;
    k_expert_rows_few<FP8, PS, QS><<<dim3((unsigned)blocks), dim3(64), 0, s>>>(a);
    return hipGetLastError();
}

template <bool FP8, int P, int Q, int NW, int STAGES>
hipError_t launch_narrow(const ExpertGemmArgs& a, int64_t pairs, hipStream_t s) {
    const int64_t blocks = (tile_bound(a, pairs, Q, (a.N + P - 1) / P) + 31) / 32 * 32;
    k_expert_rows_narrow<FP8, P, Q, NW, STAGES><<<dim3((unsigned)blocks), dim3(64 * NW), 0, s>>>(a);
    return hipGetLastError();
}

template <bool WEIGHTS>
hipError_t launch_grad_narrow(const ExpertGemmArgs& a, int64_t tiles, hipStream_t s) {
    k_expert_grad_narrow<WEIGHTS><<<dim3((unsigned)((tiles + 31) / 32 * 32)), dim3(64 * kWaves), 0, s>>>(a);
    return hipGetLastError();
}

template <bool FP8, bool PMC>
hipError_t launch_rows(const ExpertGemmArgs& a, int64_t pairs, hipStream_t s) {
    const int64_t ntiles = ((PMC ? a.K : a.N) + kTileP - 1) / kTileP;
    const int64_t tiles = tile_bound(a, pairs, 256, ntiles);
    const int64_t active = pairs < a.seg.E ? pairs : a.seg.E, mean = (pairs + active - 1) / active;
    const int64_t idim = PMC ? a.K : a.N;
    // tiles of bq rows x cols columns, were the rows spread evenly
    auto even = [&](int64_t bq, int64_t cols) { return active * ((mean + bq - 1) / bq) * ((idim + cols - 1) / cols); };
    const bool idle = even(128, 128) <= kNarrowTiles && even(256, 256) < kWideTiles;
    if constexpr (PMC) {
        constexpr int T = kNarrowGrad;
        if (idle) return launch_grad_narrow<false>(a, tile_bound(a, pairs, T, (a.K + T - 1) / T), s);
    } else {
        auto narrow32 = [&] { return launch_narrow<FP8, 128, 32, 4, FP8 ? 3 : 4>(a, pairs, s); };
        const int64_t n32 = even(32, 128);
        auto few = [&] { return launch_few<FP8, FP8 ? 2 : 1, 1>(a, pairs, s); };
        if (mean <= kFewMean && even(32, 32) <= kFew) return few();
        if (mean <= 32 && n32 >= kNarrowTiles / 2 && n32 <= kNarrowTiles) return narrow32();
        if (FP8 && mean <= kFewMean && even(32, 32) <= kFewFp8) return few();
        if (even(32, 32) <= kFewTiles) return launch_few<FP8, 2, 2>(a, pairs, s);
        if (even(64, 64) <= kNarrowTiles) return launch_narrow<FP8, 64, 64, 4, 4>(a, pairs, s);
        if (idle && (!FP8 || mean > 64)) return launch_narrow<FP8, 128, 128, 8, 2>(a, pairs, s);
        if (FP8 && mean <= kFewMean) return narrow32();
    }
    const int64_t blocks = (tiles + 255) / 256 * 256;
    if (!grid_fits(blocks, 64 * kWaves)) return hipErrorInvalidConfiguration;
    k_expert_rows<FP8, PMC><<<dim3((unsigned)blocks), dim3(64 * kWaves), 0, s>>>(a);
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
    constexpr int T = kNarrowGrad;
    const int64_t tiles = (int64_t)a.seg.E * ((a.K + T - 1) / T) * ((a.N + T - 1) / T);
    if (tiles <= kNarrowTiles) return launch_grad_narrow<true>(a, tiles, s);
    k_expert_weights_grad<<<dim3(kWeightsGradBlocks), dim3(64 * kWaves), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe

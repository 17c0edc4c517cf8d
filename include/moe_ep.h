/*
 * moe_ep.h -- C ABI of libmoe_ep.so: MoE token dispatch-layout, dispatch and
 * combine for one AMD Instinct MI355X (gfx950).
 *
 * What the library computes (the pages describe it in prose only):
 *  - "DeepEP cross-node optimisation guide" (cyqw.cn), opening paragraph: the
 *    all-to-all GPU kernels of an expert-parallel MoE library are "dispatch"
 *    (send each token's hidden vector to the experts its router picked) and
 *    "combine" (bring the expert outputs back and reduce them), with FP8
 *    support.
 *  - Same page, "Core API example": dispatch takes hidden_states, topk_idx,
 *    num_max_dispatch_tokens_per_rank and num_experts; combine takes the expert
 *    outputs, topk_weights and the handle returned by dispatch.
 *  - Same page, figure caption in "Technical analysis": the layout (per-expert
 *    and per-rank counts, token->rank map) is computed once and reused.
 *  - Same page, "Low-latency mode key features" and "Performance tuning":
 *    buffers are preallocated (with a size-hint call) and fixed-size, so no
 *    allocation happens at run time.
 *  - DeepTech release article on DeepEP (010bt.com), paragraph defining EP:
 *    different experts live on different ranks.  Here expert e lives on
 *    virtual rank e / (E / R).
 * With a single GPU the transfer to peer ranks is a local copy: dispatch
 * writes the per-destination-rank send buffers and the receive layout the
 * experts read, combine reads expert outputs from that receive layout.
 *
 * Conventions for every call:
 *  - Pointers are DEVICE pointers unless marked "host".  The caller allocates
 *    and owns every buffer passed in or out (size them with moe_size_hint:
 *    all sizes are static upper bounds, so no call ever needs a host sync).
 *  - `stream` is a hipStream_t (NULL = the legacy default stream).  Every
 *    data-path call only enqueues work on that stream and returns; it never
 *    blocks and never allocates device memory.
 *  - A context is bound to the HIP device current at moe_ctx_create and to
 *    one stream at a time; it is not thread-safe.  Calls made on another
 *    device return MOE_ERR_INVALID_ARG.
 *  - Argument errors are reported synchronously by the return value and leave
 *    nothing enqueued.  Data errors found by the kernels are recorded in a
 *    sticky device word that moe_poll_error reads: an expert id outside
 *    [-1, E) (the slot is treated as empty, -1), a row index outside its
 *    buffer or a low-latency window overflow (the row is not placed), a reused
 *    layout made from other routing (the changed tokens are dropped, see
 *    moe_dispatch), Inf or NaN in an fp8 dispatch or activation (those blocks'
 *    codes and scales are unspecified), a logit that is NaN or +infinite (moe_route:
 *    that expert is not chosen) and expert offsets of a handle that are
 *    not ascending or pass num_tokens * topk (the products take those experts to have no
 *    rows; the activation computes the rows before the last offset, none if that
 *    one is out of range).
 *  - bf16 buffers are passed as raw 16-bit storage; fp8 buffers hold OCP
 *    E4M3FN codes, one byte per channel.
 *  - With MOE_EP_LOG=1 in the environment when a context is created, each
 *    kernel launch of that context is logged on stderr (host side only; no
 *    effect on results).
 */
#ifndef MOE_EP_H
#define MOE_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_EP_ABI_VERSION 7   /* 3: moe_timing_launches; 4: stale-layout and non-finite
                                  flags, moe_dispatch_noalloc; 5: moe_dispatch_layout_prefetch;
                                  6: expert products and gated activation, MOE_KERNEL_COUNT 10;
                                  7: router, dense product, layer of a few tokens, MOE_KERNEL_COUNT 15 */

/* ---------------------------------------------------------------- status */
typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* NULL pointer, bad size, wrong device, bad config value */
    MOE_ERR_UNSUPPORTED = 2,   /* outside the supported limits below */
    MOE_ERR_CAPACITY = 3,      /* num_tokens > max_tokens (low-latency: > capacity per source rank);
                                  also from moe_poll_error: a low-latency slot window overflowed
                                  (a token repeated an expert), the rows past it were not placed */
    MOE_ERR_HANDLE = 4,        /* handle not produced by moe_dispatch on a compatible context */
    MOE_ERR_HIP = 5,           /* a HIP runtime call failed */
    MOE_ERR_BAD_TOPK = 6,      /* from moe_poll_error: an expert id outside [-1, E) was seen */
    MOE_ERR_DEVICE_BOUNDS = 7, /* from moe_poll_error: a computed row fell outside its buffer;
                                  the row was dropped */
    MOE_ERR_STALE_LAYOUT = 8,  /* from moe_poll_error: a moe_dispatch with reuse_layout = 1 found
                                  topk_idx entries that differ from the ones its layout was
                                  computed from (rewritten in place in between); every such
                                  token was dropped (pos -1, no rows written) */
    MOE_ERR_NONFINITE = 9      /* from moe_poll_error: an fp8 dispatch (or moe_swiglu_fp8) met Inf
                                  or NaN in a 128-channel block; that block's codes and scale are
                                  unspecified (every other block is exact) */
} moe_status;

/* Human-readable name of a status code (static string, never NULL). */
const char* moe_status_str(moe_status s);

/* ---------------------------------------------------------------- config */
typedef enum moe_quant {
    MOE_QUANT_BF16 = 0,        /* payload rows are the bf16 input rows */
    MOE_QUANT_FP8_E4M3 = 1     /* payload rows are E4M3FN codes + one fp32 dequant scale
                                  per 128 channels (kdjingpai.com DeepEP tutorial,
                                  "Function 3: FP8 operation optimisation"; guide,
                                  production setting "FP8 dispatch") */
} moe_quant;

typedef enum moe_layout {
    MOE_LAYOUT_CONTIGUOUS = 0, /* normal (high-throughput) mode: packed rank-major send
                                  buffer + contiguous expert-major receive rows */
    MOE_LAYOUT_PADDED_LL = 1   /* low-latency mode: fixed slots, receive buffer
                                  [R][E/R][max_tokens*R][row], no send buffer */
} moe_layout;

/* Supported limits (checked by moe_ctx_create / moe_size_hint). */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_RANKS   64
#define MOE_MAX_TOPK    32
#define MOE_MAX_HIDDEN  32768
#define MOE_MAX_FEATURES 65536   /* columns and rows of an expert's weight matrix */

typedef struct moe_config {
    int32_t max_tokens;   /* M >= 1: upper bound on num_tokens of every call; in
                             MOE_LAYOUT_PADDED_LL it is also the per-source-rank slot
                             capacity (the pages' num_max_dispatch_tokens_per_rank) */
    int32_t hidden;       /* H: channels per token; multiple of 8 (bf16), of 128 (fp8) */
    int32_t num_experts;  /* E, 1..MOE_MAX_EXPERTS, multiple of num_ranks */
    int32_t num_ranks;    /* R, 1..MOE_MAX_RANKS: virtual EP ranks; expert e -> rank e/(E/R) */
    int32_t topk;         /* k, 1..MOE_MAX_TOPK: slots per token in topk_idx */
    int32_t src_rank;     /* s0 in [0, R): this GPU's rank (selects its low-latency slots) */
    int32_t quant;        /* moe_quant */
    int32_t layout;       /* moe_layout */
} moe_config;

/* ---------------------------------------------------------------- sizes */
typedef enum moe_buffer_kind {
    MOE_BUF_SEND_ROWS = 0,      /* [max_tokens*min(k,R), row_bytes]; 0 in PADDED_LL */
    MOE_BUF_SEND_SCALES = 1,    /* fp32 [max_tokens*min(k,R), H/128]; 0 unless fp8 and CONTIGUOUS */
    MOE_BUF_RECV_ROWS = 2,      /* CONTIGUOUS: [max_tokens*k, row_bytes];
                                   PADDED_LL: [E, max_tokens*R, row_bytes] */
    MOE_BUF_RECV_SCALES = 3,    /* fp32, same row count as RECV_ROWS, H/128 per row; 0 for bf16 */
    MOE_BUF_EXPERT_OUT = 4,     /* bf16 expert outputs read by combine: RECV_ROWS' row count x 2H */
    MOE_BUF_COMBINE_OUT = 5,    /* bf16 [max_tokens, H] */
    MOE_BUF_HANDLE_POS = 6,     /* int32 [max_tokens, k] */
    MOE_BUF_HANDLE_EXPERT_OFFSETS = 7,  /* int32 [E+1] */
    MOE_BUF_HANDLE_RANK_OFFSETS = 8,    /* int32 [R+1] */
    MOE_BUF_HANDLE_SEND_SRC = 9,        /* int32 [max_tokens*min(k,R)] */
    MOE_BUF_HANDLE_RECV_SRC = 10,       /* int32 [max_tokens*k] */
    MOE_BUF_HANDLE_RECV_COUNTS = 11,    /* int32 [E] */
    MOE_BUF_LAYOUT_EXPERT_COUNTS = 12,  /* int32 [E] */
    MOE_BUF_LAYOUT_RANK_COUNTS = 13,    /* int32 [R] */
    MOE_BUF_LAYOUT_TOKEN_IN_RANK = 14,  /* uint8 [max_tokens, R] */
    MOE_BUF_WORKSPACE = 15,             /* device scratch the context allocates itself */
    MOE_BUF_KIND_COUNT = 16
} moe_buffer_kind;

/* Bytes needed for one buffer kind under `cfg` (host pointers): the pages'
 * size-hint call for preallocated, fixed-size buffers (guide, "Low-latency
 * mode key features": a size hint and pre-allocation; "Performance tuning":
 * buffers made once with low_latency_mode=True, fixed-size buffers instead of
 * queues).  Every size is a static upper bound for num_tokens <= max_tokens.
 * Pure host computation; needs no GPU.  Returns MOE_ERR_INVALID_ARG /
 * UNSUPPORTED for a bad config or kind. */
moe_status moe_size_hint(const moe_config* cfg, int32_t kind, size_t* bytes);

/* ---------------------------------------------------------------- context */
typedef struct moe_ctx moe_ctx;

/* Validate `cfg` (host) and allocate the context and its device workspace
 * (per-tile histograms and scan state, within-tile ranks, error word) on the
 * current HIP device: the pages' preallocated Buffer (guide, "Low-latency mode
 * key features": pre-allocation to avoid run-time allocation; "Performance
 * tuning": the buffer is created once, in low-latency mode with
 * low_latency_mode=True).  The only call that allocates.  On error *out is
 * NULL. */
moe_status moe_ctx_create(const moe_config* cfg, moe_ctx** out);

/* Free the context.  Synchronizes the device first.  NULL is a no-op. */
moe_status moe_ctx_destroy(moe_ctx* ctx);

/* Copy of the configuration the context was created with (host). */
moe_status moe_ctx_config(const moe_ctx* ctx, moe_config* out);

/* Launch-geometry override, for measurement sweeps: 16-byte chunks each lane
 * moves per work item in the dispatch and combine kernels (1, 2, 4, 8 or 16;
 * the combine value also applies to both backward kernels).  0 = the built-in
 * choice: one chunk per lane for the dispatch, two for the combine and the
 * dispatch backward, at most 8 row slices per token for the combine backward,
 * fewer chunks per lane when there are too few tokens to fill the chip.  The
 * fused low-latency dispatch ignores it.  Results do not depend on it. */
moe_status moe_ctx_tune(moe_ctx* ctx, int32_t dispatch_chunks, int32_t combine_chunks);

/* ---------------------------------------------------------------- layout */
/* Dispatch layout (guide, figure caption in "Technical analysis": computed once,
 * reused by dispatch and combine).
 *   topk_idx               int64 [num_tokens, k], row-major; -1 = empty slot
 *   num_tokens_per_expert  int32 [E]:  valid slots routed to expert e
 *   num_tokens_per_rank    int32 [R]:  tokens with at least one expert on rank r
 *   is_token_in_rank       uint8 [num_tokens, R]: 1 iff token t goes to rank r
 *                          (any alignment; 32-bit stores when it is 4-byte
 *                          aligned and R % 4 == 0, byte stores otherwise)
 * Any output pointer may be NULL (not written).  0 <= num_tokens <= max_tokens.
 * Also keeps, in the context's workspace, the scan state a following
 * moe_dispatch(..., reuse_layout = 1) consumes. */
moe_status moe_dispatch_layout(moe_ctx* ctx, const int64_t* topk_idx, int32_t num_tokens,
                               int32_t* num_tokens_per_expert, int32_t* num_tokens_per_rank,
                               uint8_t* is_token_in_rank, void* stream);

/* The dispatch layout, plus a read of the token rows the dispatch reusing
 * this layout will copy (an MI355X-specific addition; the pages' layout call
 * takes topk_idx only).  The layout runs on one workgroup per 256 tokens and is
 * bound by dependent latencies for several microseconds, while HBM is idle; the
 * launch's other workgroups, on the compute units the layout leaves free, read
 * x meanwhile (its first 96 MB), so that the dispatch finds those rows in the
 * 256 MB Infinity Cache instead of HBM.  Outputs, checks and the reused state
 * are those of moe_dispatch_layout; results are identical.
 *   x   bf16 [num_tokens, H], 16-byte aligned, only read; NULL = exactly
 *       moe_dispatch_layout.  Rows of under 2 MB in all are not read.  Under
 *       a workgroup cap (moe_ctx_set_max_workgroups) the extra workgroups,
 *       512 threads each, stay within it (none below a cap of 2).
 * moe_dispatch with reuse_layout = 0 does the same inside its own layout
 * launch. */
moe_status moe_dispatch_layout_prefetch(moe_ctx* ctx, const int64_t* topk_idx, int32_t num_tokens,
                                        const void* x, int32_t* num_tokens_per_expert,
                                        int32_t* num_tokens_per_rank, uint8_t* is_token_in_rank,
                                        void* stream);

/* ---------------------------------------------------------------- dispatch */
/* Output buffers of one dispatch (host struct of device pointers).
 * row_bytes = 2H (bf16) or H (fp8).  Row order:
 *   send:  rank-major; rows [rank_offsets[r], rank_offsets[r+1]) go to rank r,
 *          ascending token index inside each rank.
 *   recv:  CONTIGUOUS: expert-major, rows [expert_offsets[e], expert_offsets[e+1])
 *          for expert e, ordered by (token, slot);
 *          PADDED_LL: row e*cap + s0*M + i (cap = M*R) holds the i-th token
 *          routed to expert e, for i < M; other slots are never written.  A
 *          row with i >= M (possible only when a token repeats an expert)
 *          is not placed: its pos is -1 and moe_poll_error reports
 *          MOE_ERR_CAPACITY.
 * Scales (fp8 only) are fp32 [rows, H/128], row-parallel to the data rows. */
typedef struct moe_dispatch_buffers {
    void*  send_rows;     /* CONTIGUOUS: required; PADDED_LL: must be NULL */
    float* send_scales;   /* fp8 + CONTIGUOUS: required; else NULL */
    void*  recv_rows;     /* required */
    float* recv_scales;   /* fp8: required; else NULL */
} moe_dispatch_buffers;

/* Routing record written by moe_dispatch and read by moe_combine (host struct
 * of caller-owned device buffers, sized by the MOE_BUF_HANDLE_* hints).  The
 * pages' handle is returned by dispatch and passed to combine (guide, "Core
 * API example").  Here the caller owns the storage and the handle carries a
 * tag of the configuration that produced it, instead of a generation counter
 * held by the library: a handle stays valid until the caller reuses its
 * arrays, and moe_combine rejects one from an incompatible configuration
 * (MOE_ERR_HANDLE) rather than reporting a stale generation.
 *   pos[t, j]        row of slot j of token t in the receive layout
 *                    (CONTIGUOUS: expert-major row; PADDED_LL: e*cap + slot),
 *                    -1 for an empty slot or a row that was not placed
 *   expert_offsets   exclusive prefix sum of the per-expert counts (E+1)
 *   rank_offsets     exclusive prefix sum of the per-rank token counts (R+1)
 *   send_src_idx[i]  token of send row i (rank_offsets[R] entries)
 *   recv_src_idx[i]  token of expert-major row i (expert_offsets[E] entries;
 *                    in PADDED_LL the i-th row of expert e is slot s0*M + i -
 *                    expert_offsets[e])
 *   recv_counts[e]   rows received by expert e
 * num_tokens and tag are written by moe_dispatch (host) and checked by
 * moe_combine. */
typedef struct moe_handle {
    int32_t* pos;
    int32_t* expert_offsets;
    int32_t* rank_offsets;
    int32_t* send_src_idx;
    int32_t* recv_src_idx;
    int32_t* recv_counts;
    int32_t  num_tokens;
    uint32_t tag;
} moe_handle;

/* MoE dispatch (guide, "Core API example"; DeepTech article, feature list).
 *   x          bf16 [num_tokens, H] token hidden states
 *   topk_idx   int64 [num_tokens, k]; -1 = empty slot
 *   reuse_layout  0: compute the layout first (one extra kernel; in
 *                    MOE_LAYOUT_PADDED_LL with num_tokens * topk <= 2048 and
 *                    num_tokens <= 512 the
 *                    routing and the copy run as one fused launch instead);
 *                 1: reuse the scan state of the last layout computed on this
 *                    context (by moe_dispatch_layout, or inside a moe_dispatch
 *                    with reuse_layout = 0), which must have seen the same
 *                    topk_idx pointer and num_tokens (checked on the host).
 *                    The contents must not have changed either: the kernel
 *                    compares every entry with the expert id the layout
 *                    recorded, drops each token with a changed entry and sets
 *                    MOE_ERR_STALE_LAYOUT (moe_poll_error)
 *   bufs       output rows (and scales for fp8)
 *   handle     host struct; its device arrays are written, num_tokens/tag set
 * fp8 rows: per token and 128-channel block, a = max|x|, a' = max(a, 1e-4),
 * codes = E4M3(x * (448/a')) with round-to-nearest-even (saturating), stored
 * scale = a'/448.  Every destination gets the same bytes.  The rows must be
 * finite: for a block holding Inf or NaN the codes and scale are unspecified
 * and moe_poll_error reports MOE_ERR_NONFINITE (bf16 rows are copied bit for
 * bit whatever they hold). */
moe_status moe_dispatch(moe_ctx* ctx, const void* x, const int64_t* topk_idx, int32_t num_tokens,
                        int32_t reuse_layout, const moe_dispatch_buffers* bufs,
                        moe_handle* handle, void* stream);

/* ---------------------------------------------------------------- combine */
/* MoE combine (guide, "Core API example" and the production setting's
 * "BF16 combine").
 *   expert_out   bf16 rows in the receive layout of the handle (row pos[t, j])
 *   topk_weights fp32 [num_tokens, k]
 *   out          bf16 [num_tokens, H]
 * out[t, h] = bf16_rne( sum over valid j, ascending, of w[t, j] * y[pos[t, j], h] ),
 * accumulated in fp32 from +0 with separately rounded multiply and add. */
moe_status moe_combine(moe_ctx* ctx, const void* expert_out, const float* topk_weights,
                       const moe_handle* handle, void* out, void* stream);

/* ---------------------------------------------------------------- backward */
/* Gradients of dispatch and combine for training (DeepTech release article,
 * feature list: the high-throughput kernels serve training).  The pages give
 * no formulas; these are the derivatives of the forward definitions above,
 * with the bf16 roundings and the FP8 quantisation passed through as the
 * identity.  Gradients are bf16 in every quant mode.  Both calls read the
 * routing from a handle of the last moe_dispatch (same checks as moe_combine)
 * and return MOE_OK at once when it holds no tokens.
 *
 * moe_dispatch_backward: the adjoint of dispatch's copy into the receive rows.
 *   grad_recv  bf16 rows in the receive layout of the handle (row pos[t, j]
 *              holds the gradient of the copy of token t for slot j)
 *   grad_x     bf16 [num_tokens, H] output
 * grad_x[t, h] = bf16_rne( sum over valid j, ascending, of grad_recv[pos[t, j], h] ),
 * accumulated in fp32 from +0 (combine with every weight 1; a token with no
 * valid slot gets +0).  Send rows carry no gradient of their own: in a
 * multi-GPU exchange they are the transport of the receive rows. */
moe_status moe_dispatch_backward(moe_ctx* ctx, const void* grad_recv, const moe_handle* handle,
                                 void* grad_x, void* stream);

/* moe_combine_backward: gradients of combine with respect to the expert outputs
 * and the weights.
 *   grad_out         bf16 [num_tokens, H] gradient of combine's output
 *   topk_weights     fp32 [num_tokens, k], as passed to moe_combine
 *   expert_out       bf16 rows in the receive layout, as passed to moe_combine
 *   grad_expert_out  bf16 output rows in the receive layout: for each valid
 *                    slot, row pos[t, j] = bf16_rne(w[t, j] * grad_out[t])
 *                    (fp32 product, then one rounding); rows no slot points
 *                    at are not written
 *   grad_weights     fp32 [num_tokens, k] output: the dot product of
 *                    grad_out[t] with expert_out[pos[t, j]] (fp32 sums of the
 *                    exact bf16 products, in a fixed order; 0 for an empty slot) */
moe_status moe_combine_backward(moe_ctx* ctx, const void* grad_out, const float* topk_weights,
                                const void* expert_out, const moe_handle* handle,
                                void* grad_expert_out, float* grad_weights, void* stream);

/* ---------------------------------------------------------------- expert products */
/* What the experts compute between dispatch and combine (an addition: the pages
 * stop at the receive rows).  Expert e multiplies the rows that the dispatch
 * placed for it with its own matrix W[e], bf16 [out_features, in_features],
 * the E matrices one after another.  The rows of an expert are a ragged segment
 * (also empty) that the kernels find from handle->expert_offsets, so no count
 * ever goes to the host.
 *
 * Row order.  Each row buffer is in one of two orders:
 *   MOE_ROWS_RECV    the receive layout of the handle (row pos[t, j]): what
 *                    moe_dispatch writes and moe_combine reads
 *   MOE_ROWS_PACKED  expert-major without gaps: expert e's rows are
 *                    [expert_offsets[e], expert_offsets[e+1])
 * They are the same in MOE_LAYOUT_CONTIGUOUS.  In MOE_LAYOUT_PADDED_LL a packed
 * buffer has max_tokens * topk rows instead of E * max_tokens * R: the first
 * product reads the receive rows and writes packed ones, the activation and
 * the second product's input stay packed, and its output goes back to the
 * receive layout.
 *
 * For every call: rows that no slot points at are neither read nor written (but for
 * those of tokens dropped with MOE_ERR_STALE_LAYOUT: their places stay in the
 * segments, are computed on as the buffers hold them, and enter the weights gradient);
 * the buffers of one call may not overlap, but for moe_swiglu_backward's; a handle
 * from another configuration gives MOE_ERR_HANDLE; with no tokens the call
 * returns MOE_OK at once.  All sums are binary32 (E4M3: but for the sums of eight
 * products, see there) and rounded once, in an order that sizes and routing
 * decide: the same call gives the same bits again.
 * NaN and infinities stay in the rows and columns that hold them.  Features
 * are multiples of 8 (E4M3: see there) and at most MOE_MAX_FEATURES, else
 * MOE_ERR_UNSUPPORTED, as is a product or rows gradient of more tiles of 256 x 256
 * than a launch holds ((num_tokens * topk / 256 + E) * ceil(columns / 256), rounded
 * up to 256s, of 2^23 or more); row buffers and matrices are 16-byte aligned.  The
 * workgroup cap (moe_ctx_set_max_workgroups) leaves compute units to these
 * products and does not apply to them. */
typedef enum moe_rows_order {
    MOE_ROWS_RECV = 0,
    MOE_ROWS_PACKED = 1
} moe_rows_order;

/* out[r, n] = bf16_rne( sum over c of rows[r, c] * W[e][n, c] ), e the expert of row r.
 *   rows     bf16 [rows, in_features] in rows_order
 *   weights  bf16 [E, out_features, in_features]
 *   out      bf16 [rows, out_features] in out_order */
moe_status moe_expert_gemm(moe_ctx* ctx, const void* rows, int32_t rows_order, const void* weights,
                           int32_t in_features, int32_t out_features, const moe_handle* handle,
                           void* out, int32_t out_order, void* stream);

/* The product of E4M3 rows and matrices with binary32 scales: for inference on
 * an FP8 dispatch.
 *   rows           E4M3 codes [rows, in_features]; in_features a multiple of 128
 *   row_scales     fp32 [rows, in_features/128]: recv_scales of the dispatch, or
 *                  moe_swiglu_fp8's out_scales; same order as rows
 *   weights        E4M3 codes [E, out_features, in_features]
 *   weight_scales  fp32 [E, ceil(out_features/128), in_features/128], one for each
 *                  128 x 128 block
 * out[r, n] = bf16_rne( sum over blocks b of row_scales[r, b] * weight_scales[e][n/128, b]
 *                       * (sum over the block's c of rows[r, c] * W[e][n, c]) )
 * Of eight neighbouring channels (8 i to 8 i + 7) the E4M3 matrix instructions add the
 * products cut, towards zero, to multiples of 2^(m - 13), where m is the largest
 * sum of two operands' exponents (floor(log2), at least -6) among the eight: seven
 * of them lose less than 2^(m - 13) each, before the scales.  Codes of one size, as
 * quantisation makes them, lose about 1.5e-5 of the result, a hundredth of what its
 * bf16 rounding does.  All other sums are binary32. */
moe_status moe_expert_gemm_fp8(moe_ctx* ctx, const void* rows, const float* row_scales,
                               int32_t rows_order, const void* weights, const float* weight_scales,
                               int32_t in_features, int32_t out_features, const moe_handle* handle,
                               void* out, int32_t out_order, void* stream);

/* Gradient of moe_expert_gemm with respect to the rows:
 * grad_rows[r, c] = bf16_rne( sum over n of grad_out[r, n] * W[e][n, c] ). */
moe_status moe_expert_gemm_backward_rows(moe_ctx* ctx, const void* grad_out, int32_t out_order,
                                         const void* weights, int32_t in_features,
                                         int32_t out_features, const moe_handle* handle,
                                         void* grad_rows, int32_t rows_order, void* stream);

/* Gradient of moe_expert_gemm with respect to the matrices:
 * grad_weights[e][n, c] = sum over e's rows r of grad_out[r, n] * rows[r, c]
 *   grad_type   type of grad_weights: MOE_GRAD_BF16 (rounded once) or MOE_GRAD_F32
 *   accumulate  0: grad_weights is written (zeros for an expert without rows, also
 *               with no tokens at all); 1: the gradient is added to what it holds
 *               (in binary32, then rounded to grad_type) */
typedef enum moe_grad_type {
    MOE_GRAD_BF16 = 0,
    MOE_GRAD_F32 = 1
} moe_grad_type;
moe_status moe_expert_gemm_backward_weights(moe_ctx* ctx, const void* grad_out, int32_t out_order,
                                            const void* rows, int32_t rows_order,
                                            int32_t in_features, int32_t out_features,
                                            const moe_handle* handle, void* grad_weights,
                                            int32_t grad_type, int32_t accumulate, void* stream);

/* The gated activation between two products: for a row of gate and up values
 * side by side (bf16 [rows, 2 * features], gate first),
 * out[r, c] = bf16_rne( g * s * u ), s = 1 / (1 + exp(-g)), computed in binary32 (where
 * exp(-g) passes its range, g below -88.7, s is 0).  Input and output rows are in
 * the same order.  A gate_up row is one product's output: features is at most
 * MOE_MAX_FEATURES / 2 in this call and the two below, else MOE_ERR_UNSUPPORTED. */
moe_status moe_swiglu(moe_ctx* ctx, const void* gate_up, int32_t features, int32_t order,
                      const moe_handle* handle, void* out, void* stream);

/* The same as E4M3 codes [rows, features] with fp32 scales [rows, features/128] (features
 * a multiple of 128), quantised from the binary32 values by moe_dispatch's
 * rule: a' = max(max|v|, 1e-4) of a block, codes E4M3(v * (448/a')), scale
 * a'/448.  A block with Inf or NaN is reported as in moe_dispatch. */
moe_status moe_swiglu_fp8(moe_ctx* ctx, const void* gate_up, int32_t features, int32_t order,
                          const moe_handle* handle, void* out, float* out_scales, void* stream);

/* Gradient of moe_swiglu (of moe_swiglu_fp8 with the rounding passed through):
 * d gate = d out * u * s * (1 + g * (1 - s)), d up = d out * g * s; grad_gate_up is bf16
 * [rows, 2 * features] and may be gate_up itself. */
moe_status moe_swiglu_backward(moe_ctx* ctx, const void* grad_out, const void* gate_up,
                               int32_t features, int32_t order, const moe_handle* handle,
                               void* grad_gate_up, void* stream);

/* ---------------------------------------------------------------- router */
/* What stands before the dispatch (an addition: the pages begin with topk_idx, and
 * name group-limited gating, which these calls have): the experts and weights of
 * each token from its logits, in the form that moe_dispatch, moe_combine and moe_layer
 * read.  E and k are the context's; num_tokens is at most max_tokens, and below 2^26
 * (MOE_ERR_UNSUPPORTED). */
typedef enum moe_score {
    MOE_SCORE_SOFTMAX = 0,     /* s = softmax of the token's logits, over all its experts */
    MOE_SCORE_SIGMOID = 1      /* s = 1 / (1 + exp(-logit)) */
} moe_score;
typedef enum moe_logit_type {
    MOE_LOGIT_F32 = 0,
    MOE_LOGIT_BF16 = 1
} moe_logit_type;
#define MOE_MAX_GROUPS 64

typedef struct moe_router {    /* host struct */
    int32_t score;             /* moe_score */
    int32_t groups;            /* G, 1..MOE_MAX_GROUPS, divides E: groups of E / G neighbouring experts; 1 = no groups */
    int32_t topk_groups;       /* 1..G: groups that stay; their experts alone can be chosen */
    int32_t group_top;         /* 1 or 2: a group's score is the sum of so many of its largest s + bias */
    int32_t normalize;         /* 1: a token's weights are divided by their sum */
    float   scale;             /* factor of all weights; finite */
} moe_router;

/* topk_idx[t] = the k experts with the largest s + bias, descending, ties to the lowest
 * expert; topk_weights[t, j] = scale * s[topk_idx[t, j]], divided by the sum of the chosen s
 * if asked (bias decides what is chosen and does not enter the weights).
 *   logits        [num_tokens, E] fp32 or bf16; rows `logits_stride` elements apart
 *                 (>= E); aligned to their type
 *   bias          fp32 [E], nullable; not NaN
 *   topk_idx      int64 [num_tokens, k]
 *   topk_weights  fp32 [num_tokens, k]
 * A logit of -inf masks its expert: it is not chosen, has score 0 and adds nothing to its group.
 * So does NaN or +inf, which moe_poll_error reports (MOE_ERR_NONFINITE).  Where fewer than k
 * experts are left the last slots are -1 with weight 0; a token with none has -1 throughout.
 * Without bias and groups experts are compared by their logits, otherwise by
 * s + bias in binary64.  Weights are computed in binary32. */
moe_status moe_route(moe_ctx* ctx, const void* logits, int32_t logit_type, int64_t logits_stride,
                     int32_t num_tokens, const moe_router* router, const float* bias,
                     int64_t* topk_idx, float* topk_weights, void* stream);

/* Gradient of topk_weights with respect to the logits (the choice itself has none):
 *   grad_weights  fp32 [num_tokens, k]; not read for an empty slot
 *   topk_idx      what moe_route gave (or any experts: a slot -1, or of a masked expert, has no
 *                 part; an expert in two slots gets both gradients; an id outside
 *                 [-1, E) is taken as -1 and reported)
 *   grad_logits   fp32 [num_tokens, E], contiguous, written whole */
moe_status moe_route_backward(moe_ctx* ctx, const float* grad_weights, const void* logits,
                              int32_t logit_type, int64_t logits_stride, const int64_t* topk_idx,
                              int32_t num_tokens, const moe_router* router, float* grad_logits,
                              void* stream);

/* ---------------------------------------------------------------- dense product */
/* The product around the experts: the router's logits, the shared expert that
 * every token passes.  Any number of rows (max_tokens does not bound it); of the
 * context only the device and the error word are used. */
typedef enum moe_act {
    MOE_ACT_NONE = 0,
    MOE_ACT_RELU = 1,
    MOE_ACT_SILU = 2,          /* v / (1 + exp(-v)) */
    MOE_ACT_GELU = 3,          /* v / 2 * (1 + erf(v / sqrt(2))) */
    MOE_ACT_GELU_TANH = 4,     /* v / 2 * (1 + tanh(sqrt(2 / pi) * (v + 0.044715 v^3))) */
    MOE_ACT_SWIGLU = 5         /* silu(gate) * up of 2 F columns, gates first */
} moe_act;
typedef enum moe_out_type {
    MOE_OUT_BF16 = 0,
    MOE_OUT_F32 = 1
} moe_out_type;

/* out[r, n] = act( sum over c of x[r, c] * W[n, c] + bias[n] ) + residual[r, n].
 * With M = F, or 2 F for MOE_ACT_SWIGLU:
 *   x          bf16 [num_rows, in_features]
 *   weights    bf16 [M, in_features]
 *   bias       bf16 [M], nullable
 *   residual   bf16 [num_rows, F], nullable; may be out where that is bf16
 *   out        [num_rows, F] of out_type
 *   pre        bf16 [num_rows, M], nullable: receives the sums with their bias, for
 *              moe_linear_backward
 *   workspace  moe_linear_workspace bytes, 16-byte aligned: partial sums of products whose contraction
 *              is shared out; may be NULL if that is 0
 * F is `features`, in_features and F multiples of 8, M and in_features at most MOE_MAX_FEATURES, else
 * MOE_ERR_UNSUPPORTED (as are more tiles of 256 x 256 than 2^23 - 256); buffers 16-byte aligned; only residual and out
 * may overlap.  Sums and epilogue are binary32, each output is rounded once, in an order that the sizes decide. */
moe_status moe_linear(moe_ctx* ctx, const void* x, int32_t num_rows, const void* weights,
                      int32_t in_features, int32_t features, const void* bias, int32_t act,
                      const void* residual, void* out, int32_t out_type, void* pre, void* workspace,
                      void* stream);
/* Bytes of its workspace (host; needs no GPU). */
moe_status moe_linear_workspace(int32_t num_rows, int32_t in_features, int32_t features, int32_t act,
                                size_t* bytes);

/* Gradients of moe_linear.  With d[r, m] the gradient before the activation (grad_out * act'(pre)):
 *   grad_x[r, c] = sum over m of d[r, m] * W[m, c]        bf16 [num_rows, in_features], nullable
 *   grad_weights[m, c] = sum over r of d[r, m] * x[r, c]  [M, in_features] of grad_type, nullable
 *   grad_bias[m] = sum over r of d[r, m]                  fp32 [M], nullable
 * (The residual's gradient is grad_out.)
 *   grad_out    [num_rows, F] of out_type
 *   x, weights  as in moe_linear; weights is read for grad_x, x for grad_weights (else NULL will do)
 *   pre         what moe_linear wrote; not read for MOE_ACT_NONE (may be NULL)
 *   accumulate  1: grad_weights and grad_bias are added to what they hold
 *   workspace   moe_linear_backward_workspace bytes, 16-byte aligned: holds d, rounded to bf16 for the products, also
 *               where grad_out is fp32 (grad_bias adds the binary32 values), and sums; NULL if that is 0
 * With no rows grad_weights and grad_bias are zeroed (or left, with accumulate).  More tiles of 128 rows by 128 of
 * grad_out's columns than 2^22 - 128 are MOE_ERR_UNSUPPORTED. */
moe_status moe_linear_backward(moe_ctx* ctx, const void* grad_out, int32_t out_type, int32_t num_rows,
                               const void* x, const void* weights, int32_t in_features,
                               int32_t features, int32_t act, const void* pre, void* grad_x,
                               void* grad_weights, int32_t grad_type, int32_t accumulate,
                               float* grad_bias, void* workspace, void* stream);
/* Bytes of its workspace (host; needs no GPU). */
moe_status moe_linear_backward_workspace(int32_t num_rows, int32_t in_features, int32_t features,
                                         int32_t act, int32_t out_type, int32_t with_bias,
                                         size_t* bytes);

/* ---------------------------------------------------------------- a few tokens */
/* Everything between the router and the layer's output, for decode-sized
 * batches and inference: what dispatch, expert products, activation and combine
 * give, without receive rows in between.  It is the faster way up to about 16 tokens; from about 32 on those
 * calls are (256 experts of 7168 and 2048 in E4M3, 8 a token, 128 tokens: 1.86 ms against 2.05).  For
 * a slot (t, j) with expert e = topk_idx[t, j]:
 *   (g, u) = W1[e] x[t],   y = W2[e] (silu(g) * u)
 *   out[t] = residual[t] + sum over valid j, ascending, of topk_weights[t, j] * y
 *   x             bf16 [num_tokens, H]
 *   topk_idx      int64 [num_tokens, k]; -1 = empty slot (its weight is not used), an id outside
 *                 [-1, E) is taken as -1 and reported; a repeated expert counts each time
 *   topk_weights  fp32 [num_tokens, k]
 *   w1, w2        bf16 [E, 2 * features, H] (gates first) and [E, H, features]
 *   residual      bf16 [num_tokens, H], nullable; may be out
 *   out           bf16 [num_tokens, H]; a token without an expert gets its residual, or 0
 *   workspace     num_tokens * k * features * 2 bytes, 16-byte aligned: silu(g) * u, rounded to bf16
 * num_tokens is at most max_tokens, and num_tokens * k at most MOE_LAYER_MAX_ROWS, else
 * MOE_ERR_CAPACITY and MOE_ERR_UNSUPPORTED.  features is a multiple of 8 and at most MOE_MAX_FEATURES / 2; buffers are
 * 16-byte aligned (topk_idx 8, topk_weights and scales 4); only residual and out may overlap.  All sums are binary32, y is not
 * rounded, and the order of sums is that of sizes and routing. */
#define MOE_LAYER_MAX_ROWS 1024
moe_status moe_layer(moe_ctx* ctx, const void* x, const int64_t* topk_idx, const float* topk_weights,
                     int32_t num_tokens, const void* w1, const void* w2, int32_t features,
                     const void* residual, void* out, void* workspace, void* stream);

/* The same with matrices of E4M3 codes and a scale for each 128 x 128 block:
 *   w1_scales  fp32 [E, 2 * features / 128, H / 128]
 *   w2_scales  fp32 [E, H / 128, features / 128]
 * H and features multiples of 128.  Rows and activations stay bf16 and the codes are widened exactly, so that nothing is lost
 * by quantising rows; they cost little beside the matrices as long as they are few (with their scales an eighth of the time at
 * 128 tokens of 8 experts, which moe_dispatch, the expert products and moe_combine take 10% less for). */
moe_status moe_layer_fp8(moe_ctx* ctx, const void* x, const int64_t* topk_idx,
                         const float* topk_weights, int32_t num_tokens, const void* w1,
                         const float* w1_scales, const void* w2, const float* w2_scales,
                         int32_t features, const void* residual, void* out, void* workspace,
                         void* stream);

/* ---------------------------------------------------------------- overlap */
/* Resource control (DeepTech release article, feature list: flexible GPU
 * resource control and SM-count control for the high-throughput kernels; the
 * guide's resource-control section sets an SM limit).  At most
 * `max_workgroups` workgroups (0 = no cap, the default) run the dispatch
 * (layout-reusing or two-launch path), combine and backward kernels of this
 * context; each workgroup then loops over more rows, so results are
 * unchanged.  A workgroup is 256 threads for the dispatch and 64 threads per
 * row slice (up to 1024) for the combine backward; the combine and the
 * dispatch backward run one-wavefront workgroups, 4 * max_workgroups of them
 * (the wavefronts of max_workgroups 256-thread workgroups).  The layout's
 * tile workgroups (one per 256 tokens) and the fused low-latency dispatch
 * (the pages: low-latency kernels need no SM control) are not capped; the
 * extra workgroups a layout launch uses to read x are (512 threads each, so
 * max_workgroups / 2 of them).  Capping leaves
 * compute units to kernels on other streams, e.g. GEMMs overlapped with
 * dispatch and combine. */
moe_status moe_ctx_set_max_workgroups(moe_ctx* ctx, int32_t max_workgroups);

/* Issue/complete split (the guide's hook-based communication-computation
 * overlap, "Technical analysis"): enqueue dispatch or combine on a side stream,
 * record a hook there right after it (the issue side returns at once), keep
 * enqueuing compute on the main stream, and call moe_hook_wait on the main
 * stream where the results are first needed (the complete side).  No kernel
 * waits on the device in between.  A hook is a host object bound to the
 * device current at moe_hook_create; it may be recorded again after each
 * wait.  moe_hook_wait with a never-recorded hook returns at once. */
typedef struct moe_hook moe_hook;
moe_status moe_hook_create(moe_hook** out);
moe_status moe_hook_destroy(moe_hook* hook);
moe_status moe_hook_record(moe_hook* hook, void* stream);
moe_status moe_hook_wait(const moe_hook* hook, void* stream);

/* ---------------------------------------------------------------- errors */
/* Synchronize `stream`, read and clear the sticky device error word.
 * Returns MOE_OK, MOE_ERR_BAD_TOPK, MOE_ERR_STALE_LAYOUT, MOE_ERR_CAPACITY,
 * MOE_ERR_DEVICE_BOUNDS or MOE_ERR_NONFINITE (the first set, in that order);
 * *flags (host, may be NULL) receives the raw bits (1: bad expert id, 2: row
 * outside its buffer, 4: low-latency window overflow, 8: stale reused layout,
 * 16: non-finite fp8 input). */
moe_status moe_poll_error(moe_ctx* ctx, void* stream, uint32_t* flags);

/* ---------------------------------------------------------------- timing */
/* Per-kernel timing with HIP events recorded on the launch stream around each
 * kernel the context enqueues.  Off by default.  moe_timing_begin allocates
 * `max_launches` event pairs (host-side HIP objects, not device memory);
 * moe_timing_end synchronizes on the last event, writes per-kernel totals
 * (milliseconds) and launch counts (host arrays of MOE_KERNEL_COUNT entries)
 * and frees the events.  Launches beyond max_launches are not timed. */
typedef enum moe_kernel_id {
    MOE_KERNEL_LAYOUT = 0,   /* count + scan */
    MOE_KERNEL_DISPATCH = 1, /* pack / permute / quantise */
    MOE_KERNEL_COMBINE = 2,  /* gather-reduce */
    MOE_KERNEL_DISPATCH_BWD = 3,  /* dispatch backward (gather-sum) */
    MOE_KERNEL_COMBINE_BWD = 4,   /* combine backward (weighted scatter + dot products) */
    MOE_KERNEL_EXPERT_GEMM = 5,        /* expert products, bf16 and fp8 */
    MOE_KERNEL_EXPERT_BWD_ROWS = 6,
    MOE_KERNEL_EXPERT_BWD_WEIGHTS = 7,
    MOE_KERNEL_SWIGLU = 8,             /* gated activation, bf16 and fp8 */
    MOE_KERNEL_SWIGLU_BWD = 9,
    MOE_KERNEL_ROUTE = 10,
    MOE_KERNEL_ROUTE_BWD = 11,
    MOE_KERNEL_LINEAR = 12,
    MOE_KERNEL_LINEAR_BWD = 13,        /* all launches of a call as one */
    MOE_KERNEL_LAYER = 14,             /* both launches of a call as one */
    MOE_KERNEL_COUNT = 15
} moe_kernel_id;

moe_status moe_timing_begin(moe_ctx* ctx, int32_t max_launches);
moe_status moe_timing_end(moe_ctx* ctx, double* total_ms, int64_t* launches);

/* Per-launch durations of the timing window opened by moe_timing_begin, for
 * percentiles (call before moe_timing_end, which frees the events).  Writes
 * the kernel id (moe_kernel_id) and duration in milliseconds of the first
 * min(capacity, count) timed launches, in launch order, into the host arrays
 * kernel_ids and ms, and the number of timed launches into *count (host).
 * Synchronizes on each launch's end event.  MOE_ERR_INVALID_ARG without an
 * open timing window or with NULL arrays for capacity > 0. */
moe_status moe_timing_launches(moe_ctx* ctx, int32_t* kernel_ids, float* ms, int32_t capacity,
                               int32_t* count);

/* ---------------------------------------------------------------- no allocation */
/* For callers that cannot allocate device memory at all: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Same result
 * as moe_dispatch(reuse_layout = 0) on a context created with *cfg (the same
 * rows, scales and handle arrays; the handle is accepted by moe_combine and
 * the backward calls of any context with an equal configuration), without a
 * context: the layout workspace is a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES per GPU, loaded with the library and held until
 * the process ends, and this call makes no allocation of any kind.
 *   cfg         host; checked like moe_ctx_create.  MOE_ERR_CAPACITY when the
 *               workspace it needs (MOE_BUF_WORKSPACE) exceeds the scratch.
 *   x, topk_idx, num_tokens, bufs, handle: as in moe_dispatch.
 *   error_word  device uint32, nullable: the kernels OR the moe_poll_error
 *               bits into it (the caller clears it); NULL = not reported.
 * The scratch keeps the last call's contents; the words that must start at
 * zero are zeroed on the first call on each device and left zero by every
 * call.  Calls that overlap on one GPU (other streams, other threads) race on
 * the scratch and give wrong results: serialize them.  No launch tuning or
 * workgroup cap applies, and no kernel timing is recorded. */
#define MOE_NOALLOC_SCRATCH_BYTES (8u << 20)
moe_status moe_dispatch_noalloc(const moe_config* cfg, const void* x, const int64_t* topk_idx,
                                int32_t num_tokens, const moe_dispatch_buffers* bufs,
                                moe_handle* handle, uint32_t* error_word, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_EP_H */

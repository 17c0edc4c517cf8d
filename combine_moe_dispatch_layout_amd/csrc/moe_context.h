// The context behind moe_ctx, shared by the host files of the C ABI.  Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdio>
#include <vector>

#include "moe_ep.h"
#include "moe_internal.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {

struct Geometry {
    int El, ksend, ntiles_max, rbits;
    int64_t cap, row_bytes, nb;
    int64_t send_rows, recv_rows;
};

// Workspace layout (device, one allocation, 256-byte aligned pieces).  The
// first pieces -- error word, arrival counter and the grand totals, sized for
// the largest supported E + R -- sit at the same offsets for every
// configuration, so that a workspace shared by calls of different
// configurations (the allocation-free dispatch's static scratch) keeps the
// words that must read zero at the start of a layout zero: each layout zeroes
// the totals it used before it ends.
struct Workspace {
    size_t off_err, off_done, off_sink, off_cnt_e, off_cnt_r, off_eoff, off_roff, off_tile_cnt, off_grand_tot,
        off_erank, off_srank, total;
};

}  // namespace moe

struct moe_ctx {
    moe_config cfg;
    moe::Geometry g;
    moe::Workspace wl;
    int device;
    char* ws;
    uint32_t tag;
    // last layout computed into the workspace, and the mode it ran in
    const int64_t* layout_idx;
    int32_t layout_T;
    int32_t layout_mode;
    bool layout_valid;
    // tuning overrides (0 = heuristic)
    int pack_chunks, combine_chunks;
    // cap on the workgroups of the high-throughput kernels (0 = none)
    int max_blocks;
    // host-side launch log on stderr (environment MOE_EP_LOG=1 at context creation)
    bool log;
    // timing
    bool timing;
    int max_launches;
    std::vector<hipEvent_t> ev0, ev1;
    std::vector<int> kid;

    uint32_t* err() { return reinterpret_cast<uint32_t*>(ws + wl.off_err); }
};

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool on_ctx_device(const moe_ctx* ctx) {
    int dev = -1;
    return hipGetDevice(&dev) == hipSuccess && dev == ctx->device;
}

inline const char* kernel_name(int id) {
    static const char* names[MOE_KERNEL_COUNT] = {"layout", "dispatch", "combine", "dispatch_backward",
                                                  "combine_backward", "expert_gemm", "expert_gemm_backward_rows",
                                                  "expert_gemm_backward_weights", "swiglu", "swiglu_backward"};
    return id >= 0 && id < MOE_KERNEL_COUNT ? names[id] : "?";
}

// Record timing events around one launch when timing is on; log it when asked.
// ctx may be NULL (the allocation-free dispatch): then nothing is recorded.
struct TimedLaunch {
    moe_ctx* ctx;
    hipStream_t s;
    int slot;
    TimedLaunch(moe_ctx* c, hipStream_t st, int id) : ctx(c), s(st), slot(-1) {
        if (c == nullptr) return;
        if (c->log)
            std::fprintf(stderr, "[moe_ep] ctx %p: %s on stream %p (max_workgroups %d)\n", static_cast<void*>(c),
                         kernel_name(id), static_cast<void*>(st), c->max_blocks);
        if (c->timing && (int)c->kid.size() < c->max_launches) {
            slot = (int)c->kid.size();
            c->kid.push_back(id);
            (void)hipEventRecord(c->ev0[slot], st);
        }
    }
    void done() {
        if (slot >= 0) (void)hipEventRecord(ctx->ev1[slot], s);
    }
};

// Compute units of a device (cached per device; 0 if the query fails).
int device_cus(int dev);

}  // namespace moe

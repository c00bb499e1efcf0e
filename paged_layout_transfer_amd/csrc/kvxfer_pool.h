// kvxfer_pool.h -- the pool handle and the host helpers that every file of the library
// shares (not part of the public ABI, never compiled into a kernel).
#pragma once
#include <stdint.h>

#include <vector>

#include "kvxfer.h"
#include "kvxfer_host.h"
#include "kvxfer_internal.h"

namespace kvx {

constexpr int kInflight = 256; // calls in flight per pool before the host waits

// Per-span figures of a validated call.
struct SpanPlan {
    int64_t n_pages, ppc, n_tc, n_chunks, tiles;
};

struct SlotRange {
    int64_t start; // first slot
    int64_t count; // chunks
};

}  // namespace kvx

struct kv_pool {
    kv_pool_desc desc;
    std::vector<void *> bases;
    // allocator: free-block bitmap, lowest ids first
    kvx::BlockBitmap blocks;
    // validation scratch (no allocation on the call path)
    std::vector<kvx::SpanPlan> plans;
    std::vector<kvx::SlotRange> ranges;
    // host image of the static device scratch (kv_transfer_chunks_noalloc), made at create
    std::vector<uint64_t> scr_image;
    // device state, created on the first transfer
    int device = -1;
    uint8_t **d_regions = nullptr;
    int32_t *d_err = nullptr;
    // Span-record arena: each call takes the next free stretch of a circular buffer
    // (pinned host mirror + device copy) and records an event after its kernel; a
    // stretch is reused once that event has passed.  Allocation is sequential, so
    // the oldest call in flight is always the next one in the way.
    uint8_t *d_arena = nullptr;
    uint8_t *h_arena = nullptr;
    kvx::ArenaRing<kvx::kInflight> arena;
    hipEvent_t fl_ev[kvx::kInflight] = {};  // one per arena slot
    bool unfenced = false;  // calls were made with no event behind them: destroy waits for the device
    // staging-memory kind of the last staging base seen
    kvx::StagingKind staging_kind;
    // the declared extents of the regions, staging bases and block tables against
    // the allocations holding them (see check_buffers); the regions are checked until
    // they have passed once
    kvx::ExtentCache extents;
    bool regions_ok = false;
    // timing
    bool timing = false;
    int n_timed = 0;
    std::vector<hipEvent_t> t_ev;
};

namespace kvx {

// True if e is success; otherwise records the failing call for kv_last_hip_error.
bool hip_ok(hipError_t e, const char *where);

// The pool's device state, made on the first call on the device current then;
// KV_ERR_ARG when another device is current now.
int device_setup(kv_pool *p);

// Waits until `device` is idle, whichever is current; KV_ERR_HIP where it cannot be waited for.
int device_wait(int device);

// Reserve a stretch of the pool's record arena for one call (the host waits for the
// calls that still use it), and mark it as used by the work queued on `stream`.
int arena_take(kv_pool *p, int64_t bytes, int64_t *off);
int arena_commit(kv_pool *p, int64_t off, int64_t bytes, hipStream_t stream);

// KV_ERR_RANGE if [q, q + bytes) runs past the allocations the runtime knows there.
int check_extent(ExtentCache &c, const void *q, int64_t bytes, AllocRange *here = nullptr);
// The extents of all of the pool's regions, until they have passed once.
int check_regions(kv_pool *p);

}  // namespace kvx

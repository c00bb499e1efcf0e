// kvxfer_opshost.h -- host helpers that the operators beside the transfers share: launches whose records ride in
// the arguments or the pool's arena, the attention plan, and the checks of its calls' arrays (not part of the
// public ABI, never compiled into a kernel).
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>
#include <vector>

#include "kvxfer_ops.h"
#include "kvxfer_plan.h"
#include "kvxfer_pool.h"

#define HIP_OK(call) kvx::hip_ok((call), #call)

namespace kvx {

constexpr int64_t kMaxKv = 0x7fffffffLL - 4096;  // tiles past the last key still have 31-bit positions
constexpr int64_t kMaxAttnTokens = 1 << 24;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether `stream` is capturing: *out; KV_ERR_CAPTURE if its capture was invalidated.
inline int capturing(hipStream_t stream, bool *out)
{
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (!kvx::hip_ok(hipStreamIsCapturing(stream, &st), "hipStreamIsCapturing")) return KV_ERR_HIP;
    if (st != hipStreamCaptureStatusNone && st != hipStreamCaptureStatusActive) return KV_ERR_CAPTURE;
    *out = st == hipStreamCaptureStatusActive;
    return KV_OK;
}

// Launches with the call's records: in the kernel arguments where they fit (Args::inl), with no event
// behind them, which would cost 3 us of a call's 10 (kv_pool_destroy waits for the device instead);
// or through the pool's arena, whose stretch also fences the call.
template <class Rec, class Args, class Launch>
int launch_with_records(kv_pool *p, const Rec *recs, int32_t n, Args &a, const Rec *Args::*dev, hipStream_t stream,
                        Launch launch)
{
    constexpr int32_t kInline = (int32_t)(sizeof(a.inl) / sizeof(Rec));
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (cap && (n > kInline || p->device < 0)) return KV_ERR_CAPTURE;
    if (int rc = kvx::check_regions(p)) return rc;
    if (int rc = kvx::device_setup(p)) return rc;
    a.*dev = nullptr;
    if (n <= kInline) {
        std::memcpy(a.inl, recs, (size_t)n * sizeof(Rec));
        p->unfenced |= !cap;
        return kvx::hip_ok((hipError_t)launch(), "hipLaunchKernel") ? KV_OK : KV_ERR_HIP;
    }
    const int64_t bytes = ((int64_t)n * (int64_t)sizeof(Rec) + 255) & ~255LL;
    int64_t off = 0;
    if (int rc = kvx::arena_take(p, bytes, &off)) return rc;
    std::memcpy(p->h_arena + off, recs, (size_t)n * sizeof(Rec));
    if (!HIP_OK(hipMemcpyAsync(p->d_arena + off, p->h_arena + off, (size_t)n * sizeof(Rec), hipMemcpyHostToDevice,
                               stream)))
        return KV_ERR_HIP;
    a.*dev = reinterpret_cast<const Rec *>(p->d_arena + off);
    if (!kvx::hip_ok((hipError_t)launch(), "hipLaunchKernel")) {
        (void)hipStreamSynchronize(stream);  // the copy may be in flight: its stretch is free again
        return KV_ERR_HIP;
    }
    return kvx::arena_commit(p, off, bytes, stream);
}

}  // namespace kvx

// A step's plan on the device: one buffer of fixed sections, so that a captured launch finds
// whatever plan is set when it runs, filled through two pinned images used in turn.
struct kv_attn_plan {
    kv_pool *pool = nullptr;
    kv_attn_desc desc{};
    kvx::PlanLimits lim{};
    kvx::Plan plan, next;  // the one set, and the one being made
    std::vector<std::pair<int64_t, int64_t>> rows;  // scratch: rows owned by the sequences
    kvx::ExtentCache extents;
    uint8_t *dev = nullptr, *host[2] = {nullptr, nullptr};
    hipEvent_t sent[2] = {nullptr, nullptr};
    int turn = 0;
    int64_t off_append = 0, off_groups = 0, off_few = 0, off_many = 0, bytes = 0;
    float *part = nullptr;  // partial results, then their maxima and sums
    int device = -1;
};

namespace kvx {

// Whether a token's keys, values and queries are as many as the kernels of rotations and of 4-bit appends count: eight tokens'
// units of eight elements, and sixteen tokens' rows, in 31 bits.
inline bool countable(const kv_pool_desc &d, int64_t q_heads, int64_t dim)
{
    return (2 * (int64_t)d.num_heads + q_heads) * dim <= 1 << 27;
}

// Whether the operators read and write pools of kv_type elements of such a shape; *dim is a head's width.
inline int check_cache(const kv_pool_desc &d, int kv_type, int32_t *dim)
{
    const bool bytes = kv_type == KV_TYPE_E4M3 || kv_type == KV_TYPE_MX4, mx4 = kv_type == KV_TYPE_MX4;
    if (!bytes && kv_type != KV_TYPE_F16 && kv_type != KV_TYPE_BF16) return KV_ERR_ARG;
    const int64_t wide = mx4 ? mx4_dim(d.head_dim) : d.head_dim;
    if (d.num_kv != 2 || d.elem_bytes != (bytes ? 1 : 2) || wide < 1 || wide > KV_MAX_ATTN_DIM) return KV_ERR_ARG;
    if (mx4 && !countable(d, 0, wide)) return KV_ERR_ARG;
    if ((d.head_dim * d.elem_bytes) % (mx4 ? 4 : 16)) return KV_ERR_ALIGN;
    *dim = (int32_t)wide;
    return KV_OK;
}

// What each row of the pool's places is, as the kernels take it (AttnLaunch, ShiftLaunch).
template <class Args>
void set_pages(const kv_pool_desc &d, Args *a)
{
    const uint32_t row = (uint32_t)(d.head_dim * d.elem_bytes);
    const bool hm = d.page_layout == KV_PAGE_HEAD_MAJOR;
    a->block_stride = d.block_stride;
    a->tok_stride = hm ? row : row * (uint32_t)d.num_heads;
    a->head_stride = hm ? row * (uint32_t)d.block_size : row;
    a->num_blocks = (uint32_t)d.num_blocks;
    a->block_size = (uint32_t)d.block_size;
    set_div(a->block_size, &a->bs_magic, &a->bs_shift);
}

// The arguments common to append and attention; the plan's and the layer's part.
inline int launch_base(kv_attn_plan *p, int32_t layer, kvx::AttnLaunch *a)
{
    const kv_pool_desc &d = p->pool->desc;
    if (layer < 0 || layer >= d.num_layers) return KV_ERR_ARG;
    int dev = -1;
    if (!HIP_OK(hipGetDevice(&dev))) return KV_ERR_HIP;
    if (dev != p->device) return KV_ERR_ARG;
    a->head = reinterpret_cast<const kvx::PlanHead *>(p->dev);
    a->append = reinterpret_cast<const kvx::AppendItem *>(p->dev + p->off_append);
    a->groups = reinterpret_cast<const kvx::AttnGroup *>(p->dev + p->off_groups);
    a->k_base = static_cast<uint8_t *>(p->pool->bases[2 * layer]);
    a->v_base = static_cast<uint8_t *>(p->pool->bases[2 * layer + 1]);
    set_pages(d, a);
    a->dim = attn_dim(d, p->desc.kv_type);
    a->mx4 = p->desc.kv_type == KV_TYPE_MX4;
    a->row = (uint32_t)(d.head_dim * d.elem_bytes);
    a->heads = d.num_heads;
    a->group = p->lim.group;
    kvx::set_div((uint32_t)a->group, &a->group_magic, &a->group_shift);
    a->window = p->desc.window;
    a->full = p->lim.full ? 1 : 0;
    a->part_o = p->part;
    a->part_ml = p->part + p->lim.cap_prows * kvx::padded_dim(a->dim);
    a->err = p->pool->d_err;
    return KV_OK;
}

// A strided [n][heads][dim] array of 2-byte elements: alignment, strides, extent.
inline int check_rows(kv_attn_plan *p, const void *q, int64_t n, int32_t heads, int64_t token, int64_t head)
{
    if (!q) return KV_ERR_ARG;
    if (!aligned(q, 16) || token % 8 || head % 8) return KV_ERR_ALIGN;
    if (token < 0 || head < 0) return KV_ERR_ARG;
    const int64_t lim = INT64_MAX / 16;
    if (token > lim / std::max<int64_t>(1, n) || head > lim / heads) return KV_ERR_ARG;
    const int64_t bytes = 2 * ((n - 1) * token + (heads - 1) * head + attn_dim(p->pool->desc, p->desc.kv_type));
    return kvx::check_extent(p->extents, q, bytes);
}

// The new tokens' k and v rows of an append, checked, into the launch's arguments.
inline int append_rows(kv_attn_plan *p, const kv_append_args *x, AttnLaunch *a)
{
    const int32_t heads = p->pool->desc.num_heads;
    if (int rc = check_rows(p, x->k, x->n_tokens, heads, x->k_token_stride, x->k_head_stride)) return rc;
    if (int rc = check_rows(p, x->v, x->n_tokens, heads, x->v_token_stride, x->v_head_stride)) return rc;
    a->n_tokens = x->n_tokens;
    a->k_new = x->k;
    a->v_new = x->v;
    a->k_token = x->k_token_stride;
    a->k_head = x->k_head_stride;
    a->v_token = x->v_token_stride;
    a->v_head = x->v_head_stride;
    a->k_scale = x->k_scale;
    a->v_scale = x->v_scale;
    return KV_OK;
}

// Whether no two elements of the array share memory (an output must not): of its dimensions, in whichever order they lie,
// each steps over all that the smaller ones span.
inline bool apart(int64_t n, int32_t heads, int64_t token, int64_t head, int32_t dim, int64_t layers = 1, int64_t layer = 0)
{
    std::pair<int64_t, int64_t> dims[3] = {{token, n}, {head, heads}, {layer, layers}};  // strides and counts
    std::sort(dims, dims + 3);
    int64_t span = dim;
    for (const auto &[stride, count] : dims) {
        if (count <= 1) continue;
        if (stride < span) return false;
        span += (count - 1) * stride;
    }
    return true;
}

inline bool scale_ok(const kv_attn_plan *p, float s)
{
    return p->desc.kv_type != KV_TYPE_E4M3 || (std::isfinite(s) && s > 0);
}

}  // namespace kvx

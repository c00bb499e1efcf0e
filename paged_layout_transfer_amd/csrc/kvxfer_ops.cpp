// kvxfer_ops.cpp -- host side of the operators on a paged cache beside its transfers: page
// copies and table rewriting, references, forks and compaction, and the attention plan with
// append and attention.  The exported functions are declared and documented in include/kvxfer.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <new>
#include <vector>

#include "kvxfer_ops.h"
#include "kvxfer_plan.h"
#include "kvxfer_pool.h"

#define HIP_OK(call) kvx::hip_ok((call), #call)

namespace {

constexpr int64_t kMaxKv = 0x7fffffffLL - 4096;  // tiles past the last key still have 31-bit positions
constexpr int64_t kMaxAttnTokens = 1 << 24;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether `stream` is capturing: *out; KV_ERR_CAPTURE if its capture was invalidated.
int capturing(hipStream_t stream, bool *out)
{
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (!kvx::hip_ok(hipStreamIsCapturing(stream, &st), "hipStreamIsCapturing")) return KV_ERR_HIP;
    if (st != hipStreamCaptureStatusNone && st != hipStreamCaptureStatusActive) return KV_ERR_CAPTURE;
    *out = st == hipStreamCaptureStatusActive;
    return KV_OK;
}

// Launches with the call's records: in the kernel arguments (n <= KVX_INLINE_COPIES), with no event
// behind them, which would cost 3 us of a call's 10 (kv_pool_destroy waits for the device instead);
// or through the pool's arena, whose stretch also fences the call.
template <class Rec, class Args, class Launch>
int launch_with_records(kv_pool *p, const Rec *recs, int32_t n, Args &a, const Rec *Args::*dev, hipStream_t stream,
                        Launch launch)
{
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (cap && (n > KVX_INLINE_COPIES || p->device < 0)) return KV_ERR_CAPTURE;
    if (int rc = kvx::check_regions(p)) return rc;
    if (int rc = kvx::device_setup(p)) return rc;
    a.*dev = nullptr;
    if (n <= KVX_INLINE_COPIES) {
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

}  // namespace

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

namespace {

void plan_free(kv_attn_plan *p)
{
    for (int i = 0; i < 2; ++i) {
        if (p->sent[i]) (void)hipEventDestroy(p->sent[i]);
        if (p->host[i]) (void)hipHostFree(p->host[i]);
    }
    if (p->dev) (void)hipFree(p->dev);
    if (p->part) (void)hipFree(p->part);
    delete p;
}

// The arguments common to append and attention; the plan's and the layer's part.
int launch_base(kv_attn_plan *p, int32_t layer, kvx::AttnLaunch *a)
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
    a->block_stride = d.block_stride;
    const uint32_t row = (uint32_t)(d.head_dim * d.elem_bytes);
    const bool hm = d.page_layout == KV_PAGE_HEAD_MAJOR;
    a->tok_stride = hm ? row : row * (uint32_t)d.num_heads;
    a->head_stride = hm ? row * (uint32_t)d.block_size : row;
    a->num_blocks = (uint32_t)d.num_blocks;
    a->block_size = (uint32_t)d.block_size;
    kvx::set_div(a->block_size, &a->bs_magic, &a->bs_shift);
    a->dim = d.head_dim;
    a->heads = d.num_heads;
    a->group = p->lim.group;
    kvx::set_div((uint32_t)a->group, &a->group_magic, &a->group_shift);
    a->window = p->desc.window;
    a->full = p->lim.full ? 1 : 0;
    a->part_o = p->part;
    a->part_ml = p->part + p->lim.cap_prows * kvx::padded_dim(d.head_dim);
    a->err = p->pool->d_err;
    return KV_OK;
}

// A strided [n][heads][dim] array of 2-byte elements: alignment, strides, extent.
int check_rows(kv_attn_plan *p, const void *q, int64_t n, int32_t heads, int64_t token, int64_t head)
{
    if (!q) return KV_ERR_ARG;
    if (!aligned(q, 16) || token % 8 || head % 8) return KV_ERR_ALIGN;
    if (token < 0 || head < 0) return KV_ERR_ARG;
    const int64_t lim = INT64_MAX / 16;
    if (token > lim / std::max<int64_t>(1, n) || head > lim / heads) return KV_ERR_ARG;
    const int64_t bytes = 2 * ((n - 1) * token + (heads - 1) * head + p->pool->desc.head_dim);
    return kvx::check_extent(p->extents, q, bytes);
}

// Whether no two elements of the array share memory (an output must not).
bool apart(int64_t n, int32_t heads, int64_t token, int64_t head, int32_t dim)
{
    if (n <= 1 || heads <= 1) return (n <= 1 || token >= dim) && (heads <= 1 || head >= dim);
    return token >= head ? head >= dim && token >= (heads - 1) * head + dim
                         : token >= dim && head >= (n - 1) * token + dim;
}

bool scale_ok(const kv_attn_plan *p, float s)
{
    return p->desc.kv_type != KV_TYPE_E4M3 || (std::isfinite(s) && s > 0);
}

}  // namespace

extern "C" {

int kv_pool_share_blocks(kv_pool *p, int32_t n, const int32_t *ids)
{
    if (!p || n < 0 || (n > 0 && !ids)) return KV_ERR_ARG;
    return p->blocks.share(n, ids);
}

int kv_pool_block_refs(const kv_pool *p, int32_t id, int32_t *out)
{
    if (!p || !out) return KV_ERR_ARG;
    if (id < 0 || id >= p->desc.num_blocks) return KV_ERR_RANGE;
    *out = (int32_t)p->blocks.refs(id);
    return KV_OK;
}

int kv_pool_fork_blocks(kv_pool *p, int64_t n_tokens, const int32_t *ids, int32_t *child_ids, kv_page_copy *tail)
{
    if (!p || n_tokens < 0 || !tail || (n_tokens > 0 && (!ids || !child_ids))) return KV_ERR_ARG;
    const int64_t bs = p->desc.block_size, whole = n_tokens / bs, pages = whole + (n_tokens % bs != 0);
    if (pages > p->desc.num_blocks) return KV_ERR_RANGE;
    try {
        std::vector<int32_t> own(ids, ids + pages);
        for (int32_t id : own)
            if (!p->blocks.allocated(id)) return KV_ERR_RANGE;
        std::sort(own.begin(), own.end());
        if (std::adjacent_find(own.begin(), own.end()) != own.end()) return KV_ERR_DUP;
    } catch (...) {
        return KV_ERR_OOM;
    }
    if (pages > whole && p->blocks.n_free < 1) return KV_ERR_OOM;
    if (int rc = p->blocks.share((int32_t)whole, ids)) return rc;
    const int32_t last = pages > whole ? ids[whole] : -1;  // child_ids may be ids
    if (whole > 0) std::memmove(child_ids, ids, (size_t)whole * sizeof(int32_t));
    *tail = kv_page_copy{0, 0, 0};
    if (pages > whole) {
        int32_t fresh = -1;
        (void)p->blocks.alloc(1, &fresh);
        child_ids[whole] = fresh;
        *tail = kv_page_copy{last, fresh, (int32_t)(n_tokens - whole * bs)};
    }
    return KV_OK;
}

int kv_pool_plan_compact(kv_pool *p, int32_t max_moves, kv_page_copy *moves, int32_t *n_moves)
{
    if (!p || !n_moves || max_moves < 0 || max_moves > KV_MAX_PAGE_COPIES || (max_moves > 0 && !moves))
        return KV_ERR_ARG;
    *n_moves = p->blocks.compact(max_moves, p->desc.block_size, moves);
    return KV_OK;
}

int kv_copy_pages(kv_pool *p, const kv_page_copy *copies, int32_t n, int32_t layer_begin, int32_t layer_end,
                  hipStream_t stream)
{
    if (!p || n < 0 || n > KV_MAX_PAGE_COPIES || (n > 0 && !copies)) return KV_ERR_ARG;
    const kv_pool_desc &d = p->desc;
    if (layer_begin < 0 || layer_end > d.num_layers || layer_end <= layer_begin) return KV_ERR_ARG;
    int32_t most = 0;
    for (int32_t i = 0; i < n; ++i) {
        const kv_page_copy &c = copies[i];
        if (c.n_tokens < 1 || c.n_tokens > d.block_size) return KV_ERR_ARG;
        if (c.src < 0 || c.src >= d.num_blocks || c.dst < 0 || c.dst >= d.num_blocks) return KV_ERR_RANGE;
        most = std::max(most, c.n_tokens);
    }
    if (n == 0) return KV_OK;
    try {
        std::vector<int32_t> src(n), dst(n);
        for (int32_t i = 0; i < n; ++i) src[i] = copies[i].src, dst[i] = copies[i].dst;
        std::sort(dst.begin(), dst.end());
        if (std::adjacent_find(dst.begin(), dst.end()) != dst.end()) return KV_ERR_DUP;
        for (int32_t s : src)
            if (std::binary_search(dst.begin(), dst.end(), s)) return KV_ERR_DUP;
    } catch (...) {
        return KV_ERR_OOM;
    }
    kvx::CopyLaunch a{};
    const int64_t row = (int64_t)d.head_dim * d.elem_bytes, tok = row * d.num_heads;
    a.block_stride = d.block_stride;
    a.n_copies = (uint32_t)n;
    a.n_regions = (uint32_t)((layer_end - layer_begin) * d.num_kv);
    a.parts = (uint32_t)cdiv(most * tok, KVX_COPY_PART);
    a.items = (int64_t)n * a.n_regions * a.parts;
    a.tok = (uint32_t)tok;
    a.block_size = (uint32_t)d.block_size;
    a.hm_heads = d.page_layout == KV_PAGE_HEAD_MAJOR ? (uint32_t)d.num_heads : 0;
    a.hm_row = (uint32_t)row;
    a.word = row % 16 ? 4 : 16;
    return launch_with_records(p, copies, n, a, &kvx::CopyLaunch::copies, stream, [&] {
        a.regions = p->d_regions + (int64_t)layer_begin * d.num_kv;
        return kvx::launch_copy_pages(a, stream);
    });
}

int kv_remap_tables(kv_pool *p, const kv_page_copy *moves, int32_t n, const int32_t *in, int32_t *out, int64_t count,
                    hipStream_t stream)
{
    if (!p || n < 0 || n > KV_MAX_PAGE_COPIES || (n > 0 && !moves) || count < 0) return KV_ERR_ARG;
    if (count > 0 && (!in || !out)) return KV_ERR_ARG;
    if (!aligned(in, 4) || !aligned(out, 4)) return KV_ERR_ALIGN;
    if (count > INT64_MAX / 8) return KV_ERR_RANGE;
    std::vector<kvx::Move> m;
    try {
        m.resize((size_t)n);
    } catch (...) {
        return KV_ERR_OOM;
    }
    for (int32_t i = 0; i < n; ++i) {
        const kv_page_copy &c = moves[i];
        if (c.src < 0 || c.src >= p->desc.num_blocks || c.dst < 0 || c.dst >= p->desc.num_blocks) return KV_ERR_RANGE;
        m[i] = kvx::Move{c.src, c.dst};
    }
    std::sort(m.begin(), m.end(), [](const kvx::Move &a, const kvx::Move &b) { return a.src < b.src; });
    for (int32_t i = 0; i + 1 < n; ++i)
        if (m[i].src == m[i + 1].src) return KV_ERR_DUP;
    if (count == 0 || (n == 0 && in == out)) return KV_OK;
    const uintptr_t x = reinterpret_cast<uintptr_t>(in), y = reinterpret_cast<uintptr_t>(out);
    const uintptr_t len = (uintptr_t)count * sizeof(int32_t);
    if (x != y && x < y + len && y < x + len) return KV_ERR_ARG;
    if (kvx::check_extent(p->extents, in, (int64_t)len) || kvx::check_extent(p->extents, out, (int64_t)len))
        return KV_ERR_RANGE;
    kvx::RemapLaunch a{};
    a.in = in;
    a.out = out;
    a.count = count;
    a.n = n;
    return launch_with_records(p, m.data(), n, a, &kvx::RemapLaunch::moves, stream,
                               [&] { return kvx::launch_remap(a, stream); });
}

int kv_attn_plan_create(kv_pool *pool, const kv_attn_desc *desc, kv_attn_plan **out)
{
    if (!out) return KV_ERR_ARG;
    *out = nullptr;
    if (!pool || !desc) return KV_ERR_ARG;
    const kv_pool_desc &d = pool->desc;
    const bool e4m3 = desc->kv_type == KV_TYPE_E4M3;
    if (desc->q_type != KV_TYPE_F16 && desc->q_type != KV_TYPE_BF16) return KV_ERR_ARG;
    if (!e4m3 && desc->kv_type != desc->q_type) return KV_ERR_ARG;
    if (d.num_kv != 2 || d.elem_bytes != (e4m3 ? 1 : 2) || d.head_dim > KV_MAX_ATTN_DIM) return KV_ERR_ARG;
    if (desc->num_q_heads < 1 || desc->num_q_heads % d.num_heads) return KV_ERR_ARG;
    if (desc->flags & ~KV_ATTN_FULL || desc->window < 0 || (desc->window && (desc->flags & KV_ATTN_FULL)))
        return KV_ERR_ARG;
    if (desc->max_seqs < 1 || desc->max_seqs > KV_MAX_SEQS) return KV_ERR_ARG;
    if (desc->max_tokens < 1 || desc->max_tokens > kMaxAttnTokens) return KV_ERR_ARG;
    if (desc->max_tokens > 0x7fffffffLL / desc->num_q_heads) return KV_ERR_ARG;
    if ((d.head_dim * d.elem_bytes) % 16) return KV_ERR_ALIGN;
    if (int rc = kvx::check_regions(pool)) return rc;
    kv_attn_plan *p = new (std::nothrow) kv_attn_plan();
    if (!p) return KV_ERR_OOM;
    p->pool = pool;
    p->desc = *desc;
    p->lim = kvx::plan_limits(d, *desc);
    try {
        p->plan.reserve(p->lim);
        p->next.reserve(p->lim);
        p->rows.reserve(desc->max_seqs);
    } catch (...) {
        delete p;
        return KV_ERR_OOM;
    }
    auto section = [p](int64_t n, int64_t size) {
        const int64_t at = p->bytes;
        p->bytes += (n * size + 255) & ~255LL;
        return at;
    };
    (void)section(1, sizeof(kvx::PlanHead));
    p->off_append = section(p->lim.cap_append, sizeof(kvx::AppendItem));
    p->off_groups = section(p->lim.cap_groups, sizeof(kvx::AttnGroup));
    p->off_few = section(p->lim.cap_few, sizeof(kvx::AttnItem));
    p->off_many = section(p->lim.cap_many, sizeof(kvx::AttnItem));
    const int64_t part = p->lim.cap_prows * (kvx::padded_dim(d.head_dim) + 2) * (int64_t)sizeof(float);
    int rc = kvx::device_setup(pool);
    if (!rc) {
        p->device = pool->device;
        bool ok = HIP_OK(hipMalloc((void **)&p->dev, p->bytes)) && HIP_OK(hipMemset(p->dev, 0, 256)) &&
                  HIP_OK(hipMalloc((void **)&p->part, part));
        for (int i = 0; ok && i < 2; ++i)
            ok = HIP_OK(hipHostMalloc((void **)&p->host[i], p->bytes, hipHostMallocDefault)) &&
                 HIP_OK(hipEventCreateWithFlags(&p->sent[i], hipEventDisableTiming));
        // the zeros are on the null stream: a plan set on another must not run before them
        ok = ok && HIP_OK(hipDeviceSynchronize());
        if (!ok) rc = KV_ERR_HIP;
    }
    if (rc) {
        plan_free(p);
        return rc;
    }
    *out = p;
    return KV_OK;
}

int kv_attn_plan_destroy(kv_attn_plan *p)
{
    if (!p) return KV_OK;
    if (int rc = kvx::device_wait(p->device)) return rc;  // its launches may still run
    plan_free(p);
    return KV_OK;
}

int kv_attn_plan_set(kv_attn_plan *p, const kv_seq *seqs, int32_t n, hipStream_t stream)
{
    if (!p || n < 0 || n > p->desc.max_seqs || (n > 0 && !seqs)) return KV_ERR_ARG;
    const kv_pool_desc &d = p->pool->desc;
    p->rows.clear();
    int64_t tokens = 0;
    for (int32_t i = 0; i < n; ++i) {
        const kv_seq &s = seqs[i];
        if (s.kv_len < 0 || s.q_begin < 0 || s.q_len < 0 || s.prefix_len < 0) return KV_ERR_ARG;
        if (s.kv_len > kMaxKv || s.q_begin > 0x7fffffffLL - s.q_len) return KV_ERR_RANGE;
        tokens += s.q_len;
        if (tokens > p->desc.max_tokens) return KV_ERR_ARG;
        if (s.q_len) p->rows.push_back({s.q_begin, s.q_begin + s.q_len});
        if (s.kv_len == 0) continue;
        if (!s.block_table) return KV_ERR_ARG;
        if (!aligned(s.block_table, 4)) return KV_ERR_ALIGN;
        if (s.table_len < cdiv(s.kv_len, d.block_size) || s.table_len > 0x7fffffffLL) return KV_ERR_RANGE;
    }
    std::sort(p->rows.begin(), p->rows.end());
    for (size_t i = 1; i < p->rows.size(); ++i)
        if (p->rows[i].first < p->rows[i - 1].second) return KV_ERR_DUP;
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (cap) return KV_ERR_CAPTURE;
    int dev = -1;
    if (!HIP_OK(hipGetDevice(&dev))) return KV_ERR_HIP;
    if (dev != p->device) return KV_ERR_ARG;
    for (int32_t i = 0; i < n; ++i)
        if (seqs[i].kv_len &&
            kvx::check_extent(p->extents, seqs[i].block_table, seqs[i].table_len * (int64_t)sizeof(int32_t)))
            return KV_ERR_RANGE;
    if (!HIP_OK(hipEventSynchronize(p->sent[p->turn]))) return KV_ERR_HIP;  // its last upload has left
    kvx::Plan &plan = p->next;
    try {
        kvx::build_plan(plan, p->lim, seqs, n);  // within the vectors' capacities
    } catch (...) {
        return KV_ERR_OOM;
    }
    uint8_t *h = p->host[p->turn];
    int64_t end = sizeof(kvx::PlanHead);
    std::memcpy(h, &plan.head, sizeof(kvx::PlanHead));
    auto put = [&](int64_t off, const auto &v) {
        if (v.empty()) return;
        std::memcpy(h + off, v.data(), v.size() * sizeof(v[0]));
        end = off + (int64_t)(v.size() * sizeof(v[0]));
    };
    put(p->off_append, plan.append);
    put(p->off_groups, plan.groups);
    put(p->off_few, plan.few);
    put(p->off_many, plan.many);
    if (!HIP_OK(hipMemcpyAsync(p->dev, h, (size_t)end, hipMemcpyHostToDevice, stream))) return KV_ERR_HIP;
    std::swap(p->plan, p->next);
    if (!HIP_OK(hipEventRecord(p->sent[p->turn], stream))) {
        (void)hipStreamSynchronize(stream);  // no fence: the image is free again once the stream has passed
        return KV_ERR_HIP;
    }
    p->turn ^= 1;
    return KV_OK;
}

int kv_append_tokens(kv_attn_plan *p, int32_t layer, const kv_append_args *x, hipStream_t stream)
{
    if (!p || !x || x->n_tokens < 0) return KV_ERR_ARG;
    kvx::AttnLaunch a{};
    if (int rc = launch_base(p, layer, &a)) return rc;
    if (!p->plan.appendable || !scale_ok(p, x->k_scale) || !scale_ok(p, x->v_scale)) return KV_ERR_ARG;
    if (x->n_tokens < p->plan.tokens_end) return KV_ERR_RANGE;
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (x->n_tokens == 0 || (!cap && p->plan.append.empty())) return KV_OK;
    const int32_t H = p->pool->desc.num_heads;
    if (int rc = check_rows(p, x->k, x->n_tokens, H, x->k_token_stride, x->k_head_stride)) return rc;
    if (int rc = check_rows(p, x->v, x->n_tokens, H, x->v_token_stride, x->v_head_stride)) return rc;
    a.n_tokens = x->n_tokens;
    a.k_new = x->k;
    a.v_new = x->v;
    a.k_token = x->k_token_stride;
    a.k_head = x->k_head_stride;
    a.v_token = x->v_token_stride;
    a.v_head = x->v_head_stride;
    a.k_scale = x->k_scale;
    a.v_scale = x->v_scale;
    const uint32_t grid = (uint32_t)(cap ? p->lim.cap_append : (int64_t)p->plan.append.size());
    return kvx::hip_ok((hipError_t)kvx::launch_append(a, p->desc.q_type, p->desc.kv_type, grid, stream),
                       "hipLaunchKernel(append_tokens)")
               ? KV_OK
               : KV_ERR_HIP;
}

int kv_attend(kv_attn_plan *p, int32_t layer, const kv_attend_args *x, hipStream_t stream)
{
    if (!p || !x || x->n_tokens < 0) return KV_ERR_ARG;
    kvx::AttnLaunch a{};
    if (int rc = launch_base(p, layer, &a)) return rc;
    if (!std::isfinite(x->scale) || !std::isfinite(x->softcap) || x->softcap < 0) return KV_ERR_ARG;
    if (!scale_ok(p, x->k_scale) || !scale_ok(p, x->v_scale)) return KV_ERR_ARG;
    if (x->n_tokens < p->plan.tokens_end) return KV_ERR_RANGE;
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (x->n_tokens == 0 || (!cap && p->plan.few.empty() && p->plan.many.empty())) return KV_OK;
    const int32_t Hq = p->desc.num_q_heads;
    if (int rc = check_rows(p, x->q, x->n_tokens, Hq, x->q_token_stride, x->q_head_stride)) return rc;
    if (int rc = check_rows(p, x->out, x->n_tokens, Hq, x->out_token_stride, x->out_head_stride)) return rc;
    if (!apart(x->n_tokens, Hq, x->out_token_stride, x->out_head_stride, p->pool->desc.head_dim)) return KV_ERR_ARG;
    if (!aligned(x->lse, 4) || !aligned(x->alibi_slopes, 4)) return KV_ERR_ALIGN;
    if (x->lse && kvx::check_extent(p->extents, x->lse, x->n_tokens * Hq * (int64_t)sizeof(float)))
        return KV_ERR_RANGE;
    if (x->alibi_slopes && kvx::check_extent(p->extents, x->alibi_slopes, Hq * (int64_t)sizeof(float)))
        return KV_ERR_RANGE;
    const bool e4m3 = p->desc.kv_type == KV_TYPE_E4M3;
    const double log2e = 1.4426950408889634, scale = (double)x->scale * (e4m3 ? (double)x->k_scale : 1.0);
    a.n_tokens = x->n_tokens;
    a.q = x->q;
    a.out = x->out;
    a.lse = x->lse;
    a.slopes = x->alibi_slopes;
    a.q_token = x->q_token_stride;
    a.q_head = x->q_head_stride;
    a.out_token = x->out_token_stride;
    a.out_head = x->out_head_stride;
    const bool small = x->softcap > 0 && x->softcap <= KVX_CAP_SMALL;
    a.scale_log2 = (float)((small ? 2 / (double)x->softcap : 1.0) * scale * log2e);
    a.cap_log2 = (float)(x->softcap * log2e);
    if (!std::isfinite(a.scale_log2) || !std::isfinite(a.cap_log2)) return KV_ERR_ARG;
    if (x->softcap > KVX_CAP_SMALL) {
        const double cap = x->softcap * log2e;
        a.cap_inv = (float)(1 / cap);
        a.cap_edge = (float)std::min(KVX_CAP_EDGE * cap, (double)std::numeric_limits<float>::max());
    }
    a.v_scale = e4m3 ? x->v_scale : 1.f;
    // a captured call holds every kernel that a plan within the limits may need
    for (int which = 0; which < 2; ++which) {
        const int64_t cap_n = which ? p->lim.cap_many : p->lim.cap_few;
        const int64_t n = cap ? cap_n : (int64_t)(which ? p->plan.many : p->plan.few).size();
        if (!n) continue;
        a.items = reinterpret_cast<const kvx::AttnItem *>(p->dev + (which ? p->off_many : p->off_few));
        if (!kvx::hip_ok((hipError_t)kvx::launch_attend(a, which, p->desc.q_type, p->desc.kv_type, (uint32_t)n, stream),
                         "hipLaunchKernel(attend)"))
            return KV_ERR_HIP;
    }
    const int64_t groups = cap ? p->lim.cap_groups : (int64_t)p->plan.groups.size();
    if (groups && !kvx::hip_ok((hipError_t)kvx::launch_join(a, p->desc.q_type, (uint32_t)groups, stream),
                               "hipLaunchKernel(join)"))
        return KV_ERR_HIP;
    return KV_OK;
}

}  // extern "C"

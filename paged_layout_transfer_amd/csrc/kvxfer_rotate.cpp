// kvxfer_rotate.cpp -- host side of rotations: their handles, appends with a rotation on the way, cached keys moved
// to other positions, cached tokens read back.  The exported functions are declared and documented in include/kvxfer.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <functional>
#include <new>
#include <vector>

#include "kvxfer_opshost.h"

using namespace kvx;

struct kv_rotation {
    uint64_t *turns = nullptr;  // device, [pairs]
    int32_t pairs = 0, adjacent = 0;
    float amplitude = 1.f;
    int device = -1;
};

namespace {

// 2^64 f / (2 pi) modulo 2^64, to the nearest: the 53 bits of f times 192 bits of 1 / (2 pi), exactly.
uint64_t turns_of(double f)
{
    static const uint64_t inv[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};  // low first
    if (f == 0) return 0;
    int e = 0;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(f, &e), 53);  // f = m 2^(e - 53)
    uint64_t prod[4];
    unsigned __int128 carry = 0;
    for (int i = 0; i < 3; ++i) {
        carry += (unsigned __int128)m * inv[i];
        prod[i] = (uint64_t)carry;
        carry >>= 64;
    }
    prod[3] = (uint64_t)carry;
    // the product counts 2^(e - 53 - 192) turns; bits from `low` on are wanted, in 2^-64 turns
    const int low = 192 + 53 - 64 - e;  // f < 2^20: at least 161
    auto bits = [&](int at) -> uint64_t {  // 64 bits from bit `at` >= 0 on
        const int w = at / 64, s = at % 64;
        const uint64_t x = w < 4 ? prod[w] >> s : 0;
        return s && w + 1 < 4 ? x | prod[w + 1] << (64 - s) : x;
    };
    return bits(low) + (bits(low - 1) & 1);
}

int rotation_of(const kv_rotation *r, int device, int32_t dim, Rotation *out)
{
    if (!r || r->device != device || 2 * r->pairs > dim) return KV_ERR_ARG;
    *out = Rotation{r->turns, (uint32_t)r->pairs, r->adjacent, r->amplitude};
    return KV_OK;
}

}  // namespace

extern "C" {

int kv_mx4_row_bytes(int32_t head_dim, int32_t num_heads, int32_t *out)
{
    if (!out || num_heads < 1 || head_dim < KVX_MX4_GROUP || head_dim > KV_MAX_ATTN_DIM || head_dim % KVX_MX4_GROUP)
        return KV_ERR_ARG;
    int64_t row = (head_dim / KVX_MX4_GROUP * KVX_MX4_BYTES + 3) / 4 * 4;
    while (row * num_heads % 16) row += 4;  // a multiple of 16 is never 17 away
    *out = (int32_t)row;
    return KV_OK;
}

int kv_rotation_create(const kv_rotation_desc *d, kv_rotation **out)
{
    if (!out) return KV_ERR_ARG;
    *out = nullptr;
    if (!d || d->pairs < 1 || d->pairs > KV_MAX_ATTN_DIM / 2 || !d->inv_freq) return KV_ERR_ARG;
    if (d->pairing != KV_ROT_HALVES && d->pairing != KV_ROT_ADJACENT) return KV_ERR_ARG;
    if (!std::isfinite(d->amplitude) || !(d->amplitude > 0)) return KV_ERR_ARG;
    uint64_t turns[KV_MAX_ATTN_DIM / 2];
    for (int32_t i = 0; i < d->pairs; ++i) {
        if (!(d->inv_freq[i] >= 0) || d->inv_freq[i] > 1048576.0) return KV_ERR_ARG;
        turns[i] = turns_of(d->inv_freq[i]);
    }
    if (d->pairs % 4) return KV_ERR_ALIGN;
    kv_rotation *r = new (std::nothrow) kv_rotation();
    if (!r) return KV_ERR_OOM;
    r->pairs = d->pairs;
    r->adjacent = d->pairing == KV_ROT_ADJACENT;
    r->amplitude = d->amplitude;
    const size_t bytes = (size_t)d->pairs * sizeof(uint64_t);
    // a copy that the host waits for, as for the pool's own state
    if (!HIP_OK(hipGetDevice(&r->device)) || !HIP_OK(hipMalloc((void **)&r->turns, bytes)) ||
        !HIP_OK(hipMemcpy(r->turns, turns, bytes, hipMemcpyHostToDevice))) {
        if (r->turns) (void)hipFree(r->turns);
        delete r;
        return KV_ERR_HIP;
    }
    *out = r;
    return KV_OK;
}

int kv_rotation_destroy(kv_rotation *r)
{
    if (!r) return KV_OK;
    if (int rc = device_wait(r->device)) return rc;  // launches that read it may still run
    (void)hipFree(r->turns);
    delete r;
    return KV_OK;
}

int kv_append_rotated(kv_attn_plan *p, int32_t layer, const kv_rotation *rotation, const kv_rotate_args *rot,
                      const kv_append_args *x, hipStream_t stream)
{
    if (!p || !rotation || !rot || !x || x->n_tokens < 0) return KV_ERR_ARG;
    AppendRotated r{};
    AttnLaunch &a = r.attn;
    if (int rc = launch_base(p, layer, &a)) return rc;
    if (int rc = rotation_of(rotation, p->device, a.dim, &r.rot)) return rc;
    if (!countable(p->pool->desc, rot->q ? p->desc.num_q_heads : 0, a.dim)) return KV_ERR_ARG;
    if (!p->plan.appendable || !scale_ok(p, x->k_scale) || !scale_ok(p, x->v_scale)) return KV_ERR_ARG;
    if (x->n_tokens < p->plan.tokens_end) return KV_ERR_RANGE;
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (x->n_tokens == 0 || (!cap && p->plan.append.empty())) return KV_OK;
    const int32_t Hq = p->desc.num_q_heads;
    if (int rc = append_rows(p, x, &a)) return rc;
    if (rot->q) {
        if (int rc = check_rows(p, rot->q, x->n_tokens, Hq, rot->q_token_stride, rot->q_head_stride)) return rc;
        if (int rc = check_rows(p, rot->q_out, x->n_tokens, Hq, rot->out_token_stride, rot->out_head_stride)) return rc;
        if (!apart(x->n_tokens, Hq, rot->out_token_stride, rot->out_head_stride, a.dim)) return KV_ERR_ARG;
    }
    if (!aligned(rot->positions, 4)) return KV_ERR_ALIGN;
    if (rot->positions && check_extent(p->extents, rot->positions, x->n_tokens * (int64_t)sizeof(int32_t)))
        return KV_ERR_RANGE;
    a.q = rot->q;
    a.out = rot->q_out;
    a.q_token = rot->q_token_stride;
    a.q_head = rot->q_head_stride;
    a.out_token = rot->out_token_stride;
    a.out_head = rot->out_head_stride;
    r.positions = rot->positions;
    const uint32_t grid = (uint32_t)(cap ? p->lim.cap_append : (int64_t)p->plan.append.size());
    return hip_ok((hipError_t)launch_append_rotated(r, p->desc.q_type, p->desc.kv_type, grid, stream),
                  "hipLaunchKernel(append_rotated)")
               ? KV_OK
               : KV_ERR_HIP;
}

int kv_read_tokens(kv_attn_plan *p, int32_t layer_begin, int32_t layer_end, const kv_read_args *x, hipStream_t stream)
{
    if (!p || !x || x->n_tokens < 0 || (!x->k && !x->v)) return KV_ERR_ARG;
    const kv_pool_desc &d = p->pool->desc;
    if (layer_begin < 0 || layer_end > d.num_layers || layer_end <= layer_begin) return KV_ERR_ARG;
    ReadLaunch r{};
    AttnLaunch &a = r.attn;
    if (int rc = launch_base(p, layer_begin, &a)) return rc;
    if (!countable(d, 0, a.dim)) return KV_ERR_ARG;
    if (!p->plan.appendable || !scale_ok(p, x->k_scale) || !scale_ok(p, x->v_scale)) return KV_ERR_ARG;
    if (x->n_tokens < p->plan.tokens_end) return KV_ERR_RANGE;
    bool cap = false;
    if (int rc = capturing(stream, &cap)) return rc;
    if (x->n_tokens == 0 || (!cap && p->plan.append.empty())) return KV_OK;
    r.layers = layer_end - layer_begin;
    const struct {
        void *rows;
        int64_t layer, token, head;
    } to[2] = {{x->k, x->k_layer_stride, x->k_token_stride, x->k_head_stride},
               {x->v, x->v_layer_stride, x->v_token_stride, x->v_head_stride}};
    for (const auto &t : to) {
        if (!t.rows) continue;
        if (int rc = check_rows(p, t.rows, x->n_tokens, d.num_heads, t.token, t.head)) return rc;
        if (r.layers > 1) {
            if (t.layer % 8) return KV_ERR_ALIGN;
            if (t.layer < 0 || t.layer > INT64_MAX / 16 / r.layers) return KV_ERR_ARG;
        }
        if (!apart(x->n_tokens, d.num_heads, t.token, t.head, a.dim, r.layers, t.layer)) return KV_ERR_ARG;
        if (r.layers == 1) continue;
        const int64_t span = (x->n_tokens - 1) * t.token + (d.num_heads - 1) * t.head + a.dim;
        if (check_extent(p->extents, t.rows, 2 * ((r.layers - 1) * t.layer + span))) return KV_ERR_RANGE;
    }
    r.regions = p->pool->d_regions + 2 * (int64_t)layer_begin;
    r.k = x->k;
    r.v = x->v;
    r.k_layer = x->k_layer_stride;
    r.v_layer = x->v_layer_stride;
    a.n_tokens = x->n_tokens;
    a.k_token = x->k_token_stride;
    a.k_head = x->k_head_stride;
    a.v_token = x->v_token_stride;
    a.v_head = x->v_head_stride;
    a.k_scale = x->k_scale;
    a.v_scale = x->v_scale;
    const uint32_t grid = (uint32_t)(cap ? p->lim.cap_append : (int64_t)p->plan.append.size());
    return hip_ok((hipError_t)launch_read(r, p->desc.q_type, p->desc.kv_type, grid, stream), "hipLaunchKernel(read_tokens)")
               ? KV_OK
               : KV_ERR_HIP;
}

int kv_rotate_cached(kv_pool *p, const kv_rotation *rotation, int32_t kv_type, const kv_shift *shifts, int32_t n,
                     int32_t layer_begin, int32_t layer_end, hipStream_t stream)
{
    if (!p || !rotation || n < 0 || n > KV_MAX_SHIFTS || (n > 0 && !shifts)) return KV_ERR_ARG;
    const kv_pool_desc &d = p->desc;
    if (layer_begin < 0 || layer_end > d.num_layers || layer_end <= layer_begin) return KV_ERR_ARG;
    ShiftLaunch a{};
    if (int rc = check_cache(d, kv_type, &a.dim)) return rc;
    if (2 * rotation->pairs > a.dim || !countable(d, 0, a.dim)) return KV_ERR_ARG;
    std::vector<ShiftRec> recs;
    int64_t items = 0;
    try {
        for (int32_t i = 0; i < n; ++i) {
            const kv_shift &s = shifts[i];
            if (s.t_begin < 0 || s.t_end < s.t_begin) return KV_ERR_ARG;
            if (s.t_end > kMaxKv) return KV_ERR_RANGE;
            if (s.t_begin == s.t_end) continue;
            if (!s.block_table) return KV_ERR_ARG;
            if (!aligned(s.block_table, 4)) return KV_ERR_ALIGN;
            if (s.table_len < cdiv(s.t_end, d.block_size) || s.table_len > 0x7fffffffLL) return KV_ERR_RANGE;
            recs.push_back(ShiftRec{s.block_table, (int32_t)s.t_begin, (int32_t)s.t_end, s.delta, (int32_t)items});
            items += cdiv(s.t_end - s.t_begin, KVX_SHIFT_TOKENS);
            if (items > 0x7fffffffLL) return KV_ERR_ARG;
        }
        std::vector<ShiftRec> by_place = recs;
        std::sort(by_place.begin(), by_place.end(), [](const ShiftRec &a, const ShiftRec &b) {
            return a.table != b.table ? std::less<const int32_t *>()(a.table, b.table) : a.begin < b.begin;
        });
        for (size_t i = 1; i < by_place.size(); ++i)
            if (by_place[i].table == by_place[i - 1].table && by_place[i].begin < by_place[i - 1].end) return KV_ERR_DUP;
    } catch (...) {
        return KV_ERR_OOM;
    }
    if (recs.empty()) return KV_OK;
    int dev = -1;
    if (!HIP_OK(hipGetDevice(&dev))) return KV_ERR_HIP;
    if (int rc = rotation_of(rotation, dev, a.dim, &a.rot)) return rc;
    for (int32_t i = 0; i < n; ++i)
        if (shifts[i].t_begin < shifts[i].t_end &&
            check_extent(p->extents, shifts[i].block_table, shifts[i].table_len * (int64_t)sizeof(int32_t)))
            return KV_ERR_RANGE;
    set_pages(d, &a);
    a.heads = d.num_heads;
    a.n = (int32_t)recs.size();
    a.layers = layer_end - layer_begin;
    a.items = (int32_t)items;
    return launch_with_records(p, recs.data(), a.n, a, &ShiftLaunch::recs, stream, [&] {
        a.regions = p->d_regions + 2 * (int64_t)layer_begin;
        a.err = p->d_err;
        return launch_shift(a, kv_type, stream);
    });
}

}  // extern "C"

// kvxfer_ops.h -- what the page, append and attention kernels share with the host code
// that launches them: launch arguments, the records of an attention plan, and the index
// arithmetic of a query's visible keys (not part of the public ABI).
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "kvxfer.h"

#ifdef __HIPCC__
#define KVX_HD __host__ __device__ __forceinline__
#else
#define KVX_HD inline
#endif

namespace kvx {

// ---- pages -------------------------------------------------------------------

#define KVX_INLINE_COPIES 256  // records that ride in the kernel arguments (3 KiB)
#define KVX_COPY_PART 4096     // bytes of a page one wave copies

struct CopyLaunch {
    uint8_t *const *regions;     // of the first layer copied
    const kv_page_copy *copies;  // device array, or null: inl
    int64_t block_stride;
    int64_t items;               // copies * regions * parts
    uint32_t n_copies, n_regions, parts;
    uint32_t tok, block_size;
    uint32_t hm_heads, hm_row;   // head-major pages: heads and row bytes; 0 heads: token-major
    uint32_t word;               // 16, or 4 where a head-major row is not whole 16-byte vectors
    kv_page_copy inl[KVX_INLINE_COPIES];
};
static_assert(sizeof(CopyLaunch) <= 4096, "kernel arguments");
int launch_copy_pages(const CopyLaunch &a, hipStream_t stream);

#define KVX_REMAP_LDS 4096  // moves searched in shared memory (32 KiB); more are searched in place

struct Move {
    int32_t src, dst;
};
struct RemapLaunch {
    const int32_t *in;
    int32_t *out;
    const Move *moves;  // sorted by src; device array, or null: inl
    int64_t count;
    int32_t n;
    Move inl[KVX_INLINE_COPIES];
};
int launch_remap(const RemapLaunch &a, hipStream_t stream);

// ---- attention plan ----------------------------------------------------------

#define KVX_TILE_KEYS 64      // keys of one tile: the unit in which work is counted and split
#define KVX_ROWS_FEW 16       // rows of a piece of the few-rows kernel
// Tiles, all heads counted, to each workgroup that runs at once from which a workgroup's waves take a head
// each (token-major pages).  A wave's 256-byte rows of one head lie heads * 256 bytes apart; four waves on
// neighbouring heads read 1 KiB runs: 64 sequences of 8 K tokens 392 -> 364 us, as head-major pages
// (356 us).  Below it there are more parts to join than this gains: one sequence of 32 K (8
// tiles) 35 -> 42 us, sixteen of 200 to 5015 (10 tiles) 222 -> 213 us for four layers.
#define KVX_ACROSS 10
#define KVX_APPEND_TOKENS 8   // new tokens of one append item
#define KVX_APPEND_SPLIT 4    // workgroups of one append item
// Rows joined by one workgroup.  Eight: cut prompts and turns 2 to 6 % less (91 -> 89 us), one token on 32 K
// 34.5 -> 37 us, four layers of sixteen sequences 207.5 -> 210.7.
#define KVX_JOIN_ROWS 4

// Rows of a piece of the many-rows kernel: 32 to a wave; at the widest heads a wave's
// registers leave room for four waves only.
KVX_HD int32_t rows_many(int dim) { return dim > 128 ? 128 : 256; }
// With fewer rows, waves 4 to 7 only help loading (chosen by build_plan).
#define KVX_ROWS_HALF 128

// One workgroup's piece of attention: rows [row0, row0 + rows) of one
// sequence and cache head, over key tiles [tile0, tile1) of the tiles any of its rows sees.
// Row r is query token r / G with head `head` * G + r % G, G query heads to a cache head.
struct AttnItem {
    const int32_t *table;
    int32_t kv_len, q_begin, q_len, prefix;
    int32_t head, row0, tile0, tile1;
    int32_t prow;    // first row in the workspace of partial results, or -1: the result is whole
    int16_t rows;    // rows of the piece, unless the sequence's end first
    int16_t across;  // few rows: the four waves take the cache heads head .. head + 3 instead of
                     // every fourth step of one head; wave w's partial rows lie 16 w behind prow
};
static_assert(sizeof(AttnItem) == 48, "");

// Partial results to join: n_parts pieces of `rows` rows (at most KVX_JOIN_ROWS), part i at
// prow + i * stride.
struct AttnGroup {
    int32_t prow, n_parts, stride, rows;
    int32_t q_begin, q_len, head, row0;
};
static_assert(sizeof(AttnGroup) == 32, "");

struct AppendItem {
    const int32_t *table;
    int32_t pos, row, count, pad;  // first token's position and row; tokens, at most KVX_APPEND_TOKENS
};
static_assert(sizeof(AppendItem) == 24, "");

// Counts of the plan that is set, read by every launch, so that a captured launch works
// on whatever plan is set when it runs.
struct PlanHead {
    int32_t n_few, n_many, n_groups, n_append;
};

// The tiles a span of rows walks: tiles [0, n_prefix) hold the prefix, the rest start at
// key `low` rounded down to a tile; keys in [prefix, low) and from `high` on are seen by
// no row.  Tile i of the walk starts at key start(i).
struct KeyWalk {
    int32_t prefix, low, high;  // visible keys: [0, prefix) and [low, high)
    int32_t n_prefix, skip, n_tiles;
    KVX_HD int32_t start(int32_t i) const { return (i < n_prefix ? i : i + skip) * KVX_TILE_KEYS; }
};

// Visible keys of the query tokens at positions p0 .. p1 of a sequence.
KVX_HD KeyWalk key_walk(int32_t kv_len, int32_t prefix, int32_t window, bool full, int32_t p0, int32_t p1)
{
    KeyWalk w;
    if (full) {
        w.prefix = 0;
        w.low = 0;
        w.high = kv_len;
    } else {
        w.prefix = prefix < kv_len ? prefix : kv_len;
        w.high = p1 + 1 < 0 ? 0 : p1 + 1;
        w.low = window > 0 && p0 >= window ? p0 - window + 1 : 0;
        if (w.low > w.high) w.low = w.high;
        if (w.prefix >= w.low) {  // one stretch
            if (w.prefix > w.high) w.high = w.prefix;
            w.low = 0;
            w.prefix = 0;
        }
    }
    w.n_prefix = (w.prefix + KVX_TILE_KEYS - 1) / KVX_TILE_KEYS;
    int32_t first = w.low / KVX_TILE_KEYS;
    const int32_t last = w.high > w.low ? (w.high + KVX_TILE_KEYS - 1) / KVX_TILE_KEYS : first;
    if (first < w.n_prefix) first = w.n_prefix;  // the stretches share a tile: walked once
    w.skip = first - w.n_prefix;
    w.n_tiles = w.n_prefix + (last > first ? last - first : 0);
    return w;
}

// Caps up to this take the form with an exponential, whose error is 2^-21 of the cap at most: 3e-5 of a score, a
// sixteenth of the half step to which a half weight is rounded.  Larger ones take a quotient of polynomials, good to the
// score's last places, at a cost: a capped 8192-token prompt of 128-wide heads 736 and 943 us, eight short
// turns of 64-wide ones 95 and 109.
#define KVX_CAP_SMALL 64.f
// Scores beyond this many caps are at the cap: 2 e^(-2 x) < 2^-23.
#define KVX_CAP_EDGE 8.6

// Launch arguments of append and attention.
struct AttnLaunch {
    const PlanHead *head;
    const AttnItem *items;
    const AttnGroup *groups;
    const AppendItem *append;
    uint8_t *k_base, *v_base;  // the layer's regions
    int64_t block_stride;
    uint32_t tok_stride, head_stride;  // bytes between tokens and heads of one page
    uint32_t num_blocks, block_size, bs_magic, bs_shift;
    int32_t dim, heads, group;  // head_dim, cache heads, query heads to a cache head
    uint32_t group_magic, group_shift;
    int32_t window, full;
    int64_t n_tokens;
    const void *q;
    void *out;
    float *lse;
    const float *slopes;
    int64_t q_token, q_head, out_token, out_head;  // elements
    float scale_log2;     // scale * k_scale * log2(e), times 2 / softcap with a small cap
    float cap_log2;       // softcap * log2(e), or 0
    float cap_inv, cap_edge;  // a cap over KVX_CAP_SMALL: 1 / cap_log2 and KVX_CAP_EDGE * cap_log2; else 0
    float k_scale, v_scale;
    const void *k_new, *v_new;
    int64_t k_token, k_head, v_token, v_head;
    float *part_o;   // [partial row][padded dim]
    float *part_ml;  // [partial row][2]: maximum (base 2) and sum
    int32_t *err;
};

// floor(x / d) of 0 <= x < 2^31 as a high product and a shift; d a power of two: magic 0.
KVX_HD uint32_t div_by(uint32_t x, uint32_t magic, uint32_t shift)
{
#if defined(__HIP_DEVICE_COMPILE__)
    return magic ? __umulhi(x, magic) >> shift : x >> shift;
#else
    return magic ? (uint32_t)(((uint64_t)x * magic) >> 32) >> shift : x >> shift;
#endif
}
inline void set_div(uint32_t d, uint32_t *magic, uint32_t *shift)
{
    uint32_t s = 31 - (uint32_t)__builtin_clz(d);
    *shift = s;
    // ceil(2^(32+s) / d) < 2^32 for d no power of two; its excess e < d < 2^(s+1) keeps
    // x * e below 2^(32+s) for x < 2^31, so the floor is exact
    *magic = (d & (d - 1)) ? (uint32_t)((((uint64_t)1 << (32 + s)) + d - 1) / d) : 0;
}

int padded_dim(int dim);  // 64, 128 or 256
// which: 0 the few-rows kernel, 1 the many-rows kernel; grid workgroups
int launch_attend(const AttnLaunch &a, int which, int q_type, int kv_type, uint32_t grid, hipStream_t stream);
int launch_join(const AttnLaunch &a, int q_type, uint32_t grid, hipStream_t stream);
int launch_append(const AttnLaunch &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream);

}  // namespace kvx

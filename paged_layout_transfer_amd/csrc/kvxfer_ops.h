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
#define KVX_MX4_GROUP 32      // elements that share a scale
#define KVX_MX4_BYTES 17      // of one group: its elements and its scale
// The elements of a row of `bytes` bytes, as the operators see them.
inline int64_t mx4_dim(int64_t bytes) { return bytes / KVX_MX4_BYTES * KVX_MX4_GROUP; }
inline int32_t attn_dim(const kv_pool_desc &d, int kv_type)
{
    return kv_type == KV_TYPE_MX4 ? (int32_t)mx4_dim(d.head_dim) : d.head_dim;
}

// Few rows over mx4 pools, for a width padded to `dp`: the 1 KiB pieces of a wave's 32 keys that its lanes read, and their
// space in shared memory, where the rows of each head take the place of one more.
KVX_HD constexpr int32_t mx4_pieces(int32_t dp) { return dp == 64 ? 12 : dp == 128 ? 10 : 9; }
KVX_HD constexpr int32_t mx4_raw(int32_t dp) { return dp == 64 ? 13312 : dp == 128 ? 10752 : 9728; }
// The cache heads whose rows share a product's 16 columns: as many as those hold (a row of values takes whole 16-byte
// pieces), at most most_heads, dividing the heads.
inline int32_t mx4_pack(int32_t heads, int64_t rows, int32_t row_bytes, int32_t dp, int64_t most_heads)
{
    const int64_t per = (row_bytes + 15) / 16;
    int64_t most = 2 * mx4_pieces(dp) / per;
    if (most > mx4_raw(dp) / (33 * 16 * per)) most = mx4_raw(dp) / (33 * 16 * per);
    if (most > KVX_ROWS_FEW / rows) most = KVX_ROWS_FEW / rows;
    if (most > most_heads) most = most_heads;
    int32_t n = most < heads ? (int32_t)most : heads;
    while (n > 1 && heads % n) --n;
    return n < 1 ? 1 : n;
}
// Tiles of a workgroup below which packs are made smaller, so that more workgroups work: one sequence of 128 K tokens (8
// tiles to each of 512 workgroups with four heads) 42.4 -> 40.3 us, four layers of sixteen of 200 to 5015 (2.6) 148 -> 140.
#define KVX_PACK_TILES 12

#define KVX_APPEND_TOKENS 8   // new tokens of one append item
#define KVX_APPEND_SPLIT 4    // workgroups of one append item
#define KVX_FEW_UNITS 128     // a token's units up to which one workgroup takes a whole item (rotated appends, reads)
// Rows joined by one workgroup.  Eight: cut prompts and turns 2 to 6 % less (91 -> 89 us), one token on 32 K
// 34.5 -> 37 us, four layers of sixteen sequences 207.5 -> 210.7.
#define KVX_JOIN_ROWS 4
#define KVX_JOIN_MANY 16  // parts beyond which a workgroup joins one row of a 4-bit pool's results

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
                     // every fourth step of one head; wave w's partial rows lie 16 w behind prow.  mx4 pools:
                     // the cache heads, from `head` on, whose rows are worked on together (mx4_pack); the
                     // partial rows of the h-th of them lie h * (rows of one head) behind prow
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
    uint32_t row;                      // bytes of one row
    uint32_t num_blocks, block_size, bs_magic, bs_shift;
    int32_t dim, heads, group;  // head_dim, cache heads, query heads to a cache head
    uint32_t group_magic, group_shift;
    int32_t window, full, mx4;
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

// A rotation, on the device: what turns pair i by one position, in 2^-64 turns.
struct Rotation {
    const uint64_t *turns;
    uint32_t pairs;
    int32_t adjacent;
    float amplitude;
};

// Append with a rotation on the way: q and out of `attn` are the queries and where they go (null: no queries).
struct AppendRotated {
    AttnLaunch attn;
    Rotation rot;
    const int32_t *positions;  // or null: the tokens' places
    uint32_t lg_split;         // 2^lg_split workgroups to an item
    // divisions by the units of a row, of a token, by the pairs, and by the eights of an mx4 row and of a token's k and v
    uint32_t unit_magic, unit_shift, all_magic, all_shift, pair_magic, pair_shift, eight_magic, eight_shift, each_magic, each_shift;
};

// The new tokens' places of layers that lie one after another in `regions`, to rows.
struct ReadLaunch {
    AttnLaunch attn;
    uint8_t *const *regions;  // of the first layer
    int32_t layers;
    void *k, *v;  // or null
    int64_t k_layer, v_layer;  // elements; tokens' and heads' strides in attn
    uint32_t lg_split, unit_magic, unit_shift, all_magic, all_shift;
    int32_t deep;  // layers of a workgroup
};

#define KVX_INLINE_SHIFTS 64  // records that ride in the kernel arguments
#define KVX_READ_DEEP 4       // layers that a workgroup reads (32 of 2860 tokens of 2 heads: 13.9 us with 1, 11.7, 12.9 with 16)
#define KVX_SHIFT_TOKENS 16   // tokens of one workgroup's item
// Units of work of a thread for which a workgroup takes more layers of mx4 rows: of 2 heads, two units to a thread and layer,
// four layers (30.1 us with one, 25.0 with two, 23.2 with four or eight).  Of other rows it takes one: 8 heads' 16-bit rows
// 232 us, 234 with two, 238 with four, 256 with eight.
#define KVX_SHIFT_UNITS 8
#define KVX_DEEP_GROUPS 1024  // workgroups that remain where one takes more than a layer
#define KVX_SHIFT_GRID (1 << 20)  // workgroups along a shift's items at most

// The items of one of a shift's workgroups: its own number, then every `step`-th below `end`.  Counted without a sign: an
// item below 2^31 and a step of up to KVX_SHIFT_GRID may pass 31 bits together.
struct ItemWalk {
    uint32_t at, step, end;
    KVX_HD bool there() const { return at < end; }
    KVX_HD void next() { at += step; }
};

struct ShiftRec {
    const int32_t *table;
    int32_t begin, end;  // tokens
    int32_t delta;
    int32_t item;  // its first item
};
struct ShiftLaunch {
    uint8_t *const *regions;  // of the first layer
    const ShiftRec *recs;     // device array, or null: inl
    Rotation rot;
    int64_t block_stride;
    uint32_t tok_stride, head_stride, num_blocks, block_size, bs_magic, bs_shift;
    int32_t dim, heads, n, layers, items;  // items of one layer
    int32_t deep;                          // layers of a workgroup
    uint32_t unit_magic, unit_shift, head_magic, head_shift;
    int32_t *err;
    ShiftRec inl[KVX_INLINE_SHIFTS];
};
static_assert(sizeof(ShiftLaunch) <= 4096, "kernel arguments");

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
int launch_append_mx4(const AttnLaunch &a, int q_type, uint32_t grid, hipStream_t stream);
int launch_append_rotated(const AppendRotated &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream);
int launch_read(const ReadLaunch &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream);
int launch_shift(const ShiftLaunch &a, int kv_type, hipStream_t stream);

}  // namespace kvx

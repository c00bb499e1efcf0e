// kvxfer_attn.h -- attention of new tokens over a paged cache: device code, instantiated
// for one query type by kvxfer_attn_f16.hip and kvxfer_attn_bf16.hip, over mx4 pools by
// kvxfer_attn_mx4_f16.hip and kvxfer_attn_mx4_bf16.hip.
//
// Mathematics.  For a query row and keys taken tile by tile, with x_j the score in base 2
// (score * log2 e) and m the running maximum, the kernel keeps l = sum 2^(x_j - m) and
// o = sum 2^(x_j - m) v_j; where m grows by d both are scaled by 2^-d.  The result is o / l,
// and (m + log2 l) ln 2 the log-sum-exp.  Pieces over disjoint keys join the same way.
//
// Both products run transposed on the matrix cores: S^T = K Q^T and O^T = V^T P^T.  A
// lane then owns one query row (the matrix column) in both, so maxima, sums, masks and
// scalings stay in the lane (with one exchange between the lanes that share a row), and the
// weights leave the first product in the order in which the second takes them: its
// contraction runs over keys, whose order is free as long as V^T is read in the same one.
// V^T comes from row-major tiles in shared memory by transposing reads.
//
// Rows are the (token, query head) pairs of one cache head, so every key row that is
// loaded serves all query heads that share it.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kvxfer_device.h"

namespace kvx {

__device__ __forceinline__ f32x4 mfma16(Vec<_Float16>::x8 a, Vec<_Float16>::x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(Vec<__bf16>::x8 a, Vec<__bf16>::x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(Vec<_Float16>::x8 a, Vec<_Float16>::x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(Vec<__bf16>::x8 a, Vec<__bf16>::x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Whether a 16-bit value is an infinity or NaN.
template <class T>
__device__ __forceinline__ bool not_finite(uint16_t x)
{
    constexpr uint16_t e = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
    return (x & e) == e;
}
template <class T>
__device__ __forceinline__ bool any_not_finite(typename Vec<T>::x8 v)
{
    constexpr uint32_t e = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= ((w[i] & e) == e) | ((w[i] & (e << 16)) == (e << 16));
    return bad;
}
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
// The values with zeros for infinities and NaN.
template <class T>
__device__ __forceinline__ typename Vec<T>::x8 only_finite(typename Vec<T>::x8 v)
{
    u16x8 w = __builtin_bit_cast(u16x8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = not_finite<T>(w[i]) ? 0 : w[i];
    return __builtin_bit_cast(typename Vec<T>::x8, w);
}
// Ones where the values are of one kind: 0 NaN, 1 +infinity, 2 -infinity.
template <class T>
__device__ __forceinline__ typename Vec<T>::x8 ones_at(typename Vec<T>::x8 v, int kind)
{
    constexpr uint16_t inf = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u, one = __is_same(T, __bf16) ? 0x3f80u : 0x3c00u;
    u16x8 w = __builtin_bit_cast(u16x8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool is = kind == 0 ? (w[i] & 0x7fff) > inf : w[i] == (kind == 1 ? inf : inf | 0x8000u);
        w[i] = is ? one : 0;
    }
    return __builtin_bit_cast(typename Vec<T>::x8, w);
}
__device__ __forceinline__ float special(int kind) { return kind == 0 ? __builtin_nanf("") : kind == 1 ? INFINITY : -INFINITY; }

// A seen infinity whose weight is zero (2^-149 of the largest, 2^-32 in half) has made NaN of a result that is
// infinite.  Such results are set to zero, what they see of infinities and NaN is added, and those to which
// nothing was added stay NaN: they are none of ours.
template <class V, int N>
struct Lost {
    static constexpr int kEach = sizeof(V) / 4;
    uint32_t bits[(N * kEach + 31) / 32] = {};
    __device__ __forceinline__ void clear(V (&o)[N])
    {
#pragma unroll
        for (int i = 0; i < N * kEach; ++i) {
            const float x = o[i / kEach][i % kEach];
            bits[i / 32] |= (x != x ? 1u : 0u) << (i % 32);
            o[i / kEach][i % kEach] = x != x ? 0.f : x;
        }
    }
    __device__ __forceinline__ void restore(V (&o)[N])
    {
#pragma unroll
        for (int i = 0; i < N * kEach; ++i) {
            const float x = o[i / kEach][i % kEach];
            o[i / kEach][i % kEach] = (bits[i / 32] >> (i % 32) & 1u) && x == 0.f ? __builtin_nanf("") : x;
        }
    }
    // Whether any result is infinite or NaN.
    static __device__ __forceinline__ bool any(const V (&o)[N])
    {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < N * kEach; ++i) x = __builtin_fmaf(o[i / kEach][i % kEach], 0.f, x);
        return x != x;
    }
};

// How pool rows are read: the values of one load of the few-rows kernel (a lane in four shares a row, so an mx4 load is
// at most a quarter of it: 32 values, or 16 of a 64-wide row), their bytes, and eight of them as T.
template <int CACHE, int DP>
constexpr int cache_values() { return CACHE == kHalves ? 8 : CACHE == kE4m3 ? 16 : DP == 64 ? 16 : 32; }
template <int CACHE>
constexpr int cache_bytes(int values) { return CACHE == kHalves ? 2 * values : CACHE == kE4m3 ? values : values / 2; }
template <int BYTES>
struct Words;
template <>
struct Words<4> {
    typedef uint32_t type;
};
// mx4 rows start at multiples of four bytes
template <>
struct Words<8> {
    typedef u32x2 type __attribute__((aligned(4)));
};
template <>
struct Words<16> {
    typedef u32x4 type __attribute__((aligned(4)));
};
template <class T, int CACHE, class R>
__device__ __forceinline__ typename Vec<T>::x8 widen8(const R &r, int u)
{
    if constexpr (CACHE == kE4m3)
        return __builtin_shufflevector(from_e4m3<T>(r[2 * u]), from_e4m3<T>(r[2 * u + 1]), 0, 1, 2, 3, 4, 5, 6, 7);
    else
        return __builtin_bit_cast(typename Vec<T>::x8, r);
}

// Rows of a tile in shared memory, in values.  Key rows are one 16-byte chunk longer than
// their values, so that the 16 lanes that read one chunk of 16 rows meet all banks; value rows 64
// bytes, so that the transposing reads' 64-byte stretches of four rows do.  (Exchanging chunks
// instead saves the space, but takes an address register for each chunk.)
template <int DP>
constexpr int key_row() { return DP + 8; }
template <int DP>
constexpr int value_row() { return DP + 32; }

// Four consecutive rows of one column, transposed: the 16 lanes of a group read 4 rows of
// 16 values, lane i giving the address of values 4 (i mod 4) .. +3 of row i / 4, and lane i
// receives column i of the four rows.
template <class T>
__device__ __forceinline__ typename Vec<T>::x4 read_column(const T *p)
{
    const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KVX_LDS i16x4 *)(KVX_LDS void *)p);
    return __builtin_bit_cast(typename Vec<T>::x4, v);
}

// The larger of a lane's value and that of the lane 32 away, on the vector pipe.
__device__ __forceinline__ float max_of_halves(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// And of the lane 16 away.
__device__ __forceinline__ float max_of_quarters(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// The keys one query sees, as two stretches: [0, prefix) and [low, high].  Compared without
// branches: a mask is three compares and a select.  (With short-circuit branches beside the capped score's code
// one of four fully masked scores was kept; the cause was not found.)
struct RowMask {
    int32_t low, high, prefix;
    __device__ __forceinline__ bool sees(int32_t j) const { return ((j >= low) & (j <= high)) | (j < prefix); }
};

// A piece's place in its sequence, the same for the whole workgroup.
struct Piece {
    const int32_t *table;
    int32_t kv_len, q_begin, q_len, prefix, head, row0, tile0, tile1, prow;
    int32_t rows;   // rows of the sequence and cache head from row0 on
    int32_t first;  // position of query token 0
    int32_t p0, p1; // positions of the piece's first and last query token
    KeyWalk walk;
};

__device__ __forceinline__ Piece piece_of(const AttnLaunch &a, const AttnItem &it)
{
    Piece s;
    s.table = it.table;
    s.kv_len = it.kv_len;
    s.q_begin = it.q_begin;
    s.q_len = it.q_len;
    s.prefix = it.prefix;
    s.head = it.head;
    s.row0 = it.row0;
    s.tile0 = it.tile0;
    s.tile1 = it.tile1;
    s.prow = it.prow;
    s.rows = s.q_len * a.group - s.row0;
    if (s.rows > it.rows) s.rows = it.rows;
    s.first = s.kv_len - s.q_len;
    s.p0 = s.first + (int32_t)div_by(s.row0, a.group_magic, a.group_shift);
    s.p1 = s.first + (int32_t)div_by(s.row0 + s.rows - 1, a.group_magic, a.group_shift);
    s.walk = key_walk(s.kv_len, s.prefix, a.window, a.full != 0, s.p0, s.p1);
    return s;
}

__device__ __forceinline__ RowMask row_mask(const AttnLaunch &a, const Piece &s, int32_t p)
{
    RowMask m;
    m.low = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    m.high = a.full || p >= s.kv_len ? s.kv_len - 1 : p;
    m.prefix = s.prefix < s.kv_len ? s.prefix : s.kv_len;
    return m;
}

// The key to read in j's place: j itself if some row sees it, else a neighbour that some row
// sees, so that no page is read, and no table entry followed, that nothing sees.
__device__ __forceinline__ int32_t seen_key(const Piece &s, int32_t j)
{
    const int32_t k = min(max(j, s.walk.low), s.walk.high - 1);
    return j < s.walk.prefix ? j : s.walk.high > s.walk.low ? k : s.walk.prefix - 1;
}

// Whether every row of the piece sees the n keys from j on: the scores need no mask.
__device__ __forceinline__ bool all_see(const AttnLaunch &a, const Piece &s, int32_t j, int32_t n)
{
    if (j + n > s.kv_len) return false;
    if (a.full || j + n <= s.prefix) return true;
    return j + n - 1 <= s.p0 && (a.window == 0 || s.p1 < a.window || j > s.p1 - a.window);
}

// The block that holds key j, and where key j's row (of the piece's head) starts in a region.  A
// block id out of range is reported, and block 0 read.
__device__ __forceinline__ int32_t block_of(const AttnLaunch &a, const Piece &s, int32_t j)
{
    return s.table[div_by((uint32_t)j, a.bs_magic, a.bs_shift)];
}
__device__ __forceinline__ int64_t key_offset(const AttnLaunch &a, const Piece &s, int32_t j, int32_t blk)
{
    const uint32_t slot = (uint32_t)j - div_by((uint32_t)j, a.bs_magic, a.bs_shift) * a.block_size;
    if ((uint32_t)blk >= a.num_blocks) {
        atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
        blk = 0;
    }
    return (int64_t)blk * a.block_stride + ((int64_t)slot * a.tok_stride + (int64_t)s.head * a.head_stride);
}

// Score transforms other than one positive scale, by the kernels' SHAPED: 1 the tanh cap, the distance slopes and
// scales that are not positive; 2 a cap over KVX_CAP_SMALL, with slopes or without; 0 none of them, nothing to
// do here.  Base-2 scores out.  key(i) is the key of score i.
template <int SHAPED, int N, class X, class Key>
__device__ __forceinline__ void shape(const AttnLaunch &a, X &x, float slope_log2, int32_t p, Key key)
{
    if (SHAPED == 2) {
        // c tanh(s / c) = s R((s / c)^2), R(u) = tanh(sqrt u) / sqrt u, relative to the score itself however
        // large the cap is.  R is a minimax quotient of two polynomials on |s / c| <= KVX_CAP_EDGE, good to
        // 2^-26.2; beyond, tanh is 1 - 2^-23.8 or more.  Coefficients and u are positive, so nothing
        // cancels: 24 roundings of 2^-24 at most, 2^-21.4 of the score the worst of 4 million.  The bounds
        // let NaN pass.
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float w = __builtin_elementwise_maximum(
                __builtin_elementwise_minimum(x[i] * a.scale_log2, a.cap_edge), -a.cap_edge);
            const float y = w * a.cap_inv, u = y * y;
            float num = __builtin_fmaf(u, 1.40824019e-08f, 2.11223269e-05f);
            float den = __builtin_fmaf(u, 8.07060701e-07f, 3.33626464e-04f);
            num = __builtin_fmaf(u, num, 3.52639798e-03f);
            den = __builtin_fmaf(u, den, 2.59938873e-02f);
            num = __builtin_fmaf(u, num, 1.34068727e-01f);
            den = __builtin_fmaf(u, den, 4.67401952e-01f);
            num = __builtin_fmaf(u, num, 1.f);
            den = __builtin_fmaf(u, den, 1.f);
            x[i] = w * num * __builtin_amdgcn_rcpf(den);
        }
    } else if (a.cap_log2 != 0.f) {
        // c tanh y = c - 2 c / (e^2y + 1); the scale makes 2^x of it e^2y.  A difference of numbers near the
        // cap, good to 2^-21 of it: 3e-5 of a score at KVX_CAP_SMALL.
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = __builtin_fmaf(-2.f * a.cap_log2, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x[i] * a.scale_log2) + 1.f),
                                  a.cap_log2);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= a.scale_log2;
    }
    if (a.slopes) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] -= slope_log2 * fabsf((float)(p - key(i)));
    }
}

template <int N, class X, class Key>
__device__ __forceinline__ void hide(X &x, const RowMask &mask, Key key)
{
    asm volatile("");  // a tile that all rows see whole branches past the compares
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = mask.sees(key(i)) ? x[i] : -INFINITY;
}

// A factor for a row's sums, never zero: an infinity among them stays one however far the
// maximum grows (zero times it would be NaN), and 2^-149 of anything else is nothing.
__device__ __forceinline__ float keep(float by) { return fmaxf(by, 1.401298464e-45f); }

// Half weights are scaled by 2^7.  They reach 2^8 (a maximum that grows by less is not followed), so they stay
// below 2^15, and the smallest that is not rounded to zero is 2^-32 of the largest instead of 2^-25: the sum of
// the weights, in 32 bits, keeps what the product would lose (a first key 17.5 above 32 K others in one
// accumulator: 0.08 % of their result was lost, 2.6 % of a million's).  bfloat16 has the exponents of 32 bits.
template <class T>
constexpr float weight_shift() { return __is_same(T, __bf16) ? 0.f : 7.f; }

// One query row's eight consecutive values, zero past the row's width.
template <class T>
__device__ __forceinline__ typename Vec<T>::x8 load_q(const AttnLaunch &a, const T *row, int d)
{
    if (d >= a.dim) return typename Vec<T>::x8{};
    return *(const typename Vec<T>::x8 *)(row + d);
}

template <class T>
__device__ __forceinline__ const T *q_row(const AttnLaunch &a, const Piece &s, int r)
{
    const uint32_t R = (uint32_t)(s.row0 + (r < s.rows ? r : s.rows - 1));
    const uint32_t t = div_by(R, a.group_magic, a.group_shift);
    int64_t row = (int64_t)s.q_begin + t;
    if (row >= a.n_tokens) row = a.n_tokens - 1;  // replays of a call with shorter arrays: not stored
    return (const T *)a.q + row * a.q_token + (int64_t)(s.head * a.group + (int32_t)(R - t * a.group)) * a.q_head;
}

// Eight result values of one row, from columns d .. d + 7.
template <class T>
__device__ __forceinline__ void store_out(const AttnLaunch &a, int64_t row, int32_t head, int d, const float *o,
                                          float by)
{
    if (d >= a.dim || row >= a.n_tokens) return;
    typename Vec<T>::x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)(o[i] * by);
    *(typename Vec<T>::x8 *)((T *)a.out + row * a.out_token + (int64_t)head * a.out_head + d) = v;
}

__device__ __forceinline__ void store_lse(const AttnLaunch &a, int64_t row, int32_t head, float m, float l)
{
    if (!a.lse || row >= a.n_tokens) return;
    // the natural logarithm of sum 2^(x - m) 2^m
    a.lse[row * (a.heads * a.group) + head] =
        l == 0.f ? -INFINITY : 0.6931471805599453f * (m + __builtin_amdgcn_logf(l));
}

// ---- few rows: single tokens and drafts ----------------------------------------

struct RowPlace {
    int32_t token, head;
};

// The end of a few-rows kernel: the waves' maxima (m, and `mine` with the scale in base 2), sums and results, joined in
// shared memory and stored.
// row_of(r) is the token of the piece and the query head of row r of n_rows.
template <class T, int DP, int SLICE, class RowOf>
__device__ __forceinline__ void finish_few(const AttnLaunch &a, const Piece &s, bool across, int n_rows, RowOf row_of, char *shared,
                                           float (&join_m)[4][16], float (&join_l)[4][16], float m, float mine, float l,
                                           const f32x4 (&o)[DP / 16])
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    float *const slice = (float *)(shared + wave * SLICE);
    // join the four waves: their slices hold 16 rows of 32-bit results.  With a head to each wave
    // there is nothing to join, and a wave reads its own slice back, a row at a time.
    if (g == 0) join_m[wave][n] = mine, join_l[wave][n] = l;
    __syncthreads();  // the slices' values are no longer needed
    float top = mine;
    if (!across) {
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, join_m[w][n]);
    }
    const float by = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mine - top);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) *(f32x4 *)(slice + n * DP + d * 16 + 4 * g) = o[d] * keep(by);
    __syncthreads();
    const int at = across ? lane : (int)threadIdx.x, wide = across ? 4 : 16;  // threads of a row
    const int row = at / wide, w0 = across ? wave : 0, w1 = across ? wave + 1 : 4;
    if (row >= n_rows) return;
    const auto [t_r, head] = row_of(row);
    const int64_t to_row = (int64_t)s.q_begin + t_r;
    float sum = 0.f;
    top = -INFINITY;
    for (int w = w0; w < w1; ++w) top = fmaxf(top, join_m[w][row]);
    for (int w = w0; w < w1; ++w)
        sum += join_l[w][row] * (join_m[w][row] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(join_m[w][row] - top));
    for (int d = at % wide * 8; d < DP; d += wide * 8) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int w = w0; w < w1; ++w)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += ((float *)(shared + w * SLICE))[row * DP + d + k];
        if (s.prow >= 0) {
            float *to = a.part_o + ((int64_t)s.prow + row) * DP + d;
            *(f32x4 *)to = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4 *)(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            store_out<T>(a, to_row, head, d, v, sum == 0.f ? 0.f : a.v_scale / sum);
        }
    }
    if (at % wide == 0) {
        if (s.prow >= 0) {
            a.part_ml[2 * ((int64_t)s.prow + row)] = top;
            a.part_ml[2 * ((int64_t)s.prow + row) + 1] = sum;
        } else {
            store_lse(a, to_row, head, top, sum);
        }
    }
}

// At most 16 rows (16x16x32 products).  Four waves take the piece's 32-key steps in turn, each
// with its own running maximum, and join at the end in shared memory; or each takes a cache head
// (AttnItem::across).  Bound by the cache's bytes: keys go from memory to the first product's
// registers directly, values through a slice of shared memory of the wave's own, both loaded a
// step ahead and their block ids two, with no barrier in the loop.  At most 256 registers, so
// that two workgroups share a compute unit and 128 KiB are on their way to it.  Measured, 128-wide
// bf16 heads, 4 query heads to a cache head: 32 sequences of 1 K to 64 K tokens 306 us, 5.7 TB/s;
// one of 32 K 28 us and 6 us to join; a context that one step of each wave covers 7 us, the latency of
// record, block id, rows and the way out.
// 64-wide e4m3 heads keep four waves a SIMD, 128 registers, in all forms: 128 sequences of 4 K to 5.4 K, head-major, a cap of
// 30 117 us (three waves, with 131 registers: 154), of 300 120 us (151).
template <class T, int CACHE, int DP, int SHAPED>
__global__ __launch_bounds__(256, DP == 256 ? 1 : CACHE == kE4m3 && DP == 64 ? 4 : 2) void attend_few(const AttnLaunch a)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    constexpr int kStep = 32;                         // keys of one wave's step
    constexpr int kS = DP / 32;                       // contraction steps of the first product
    constexpr int kVals = cache_values<CACHE, DP>();  // values of a lane's load: 16 bytes, or 8
    constexpr int kLoads = DP / (4 * kVals);          // loads of a lane for one key row
    constexpr int kBytes = cache_bytes<CACHE>(kVals);
    typedef typename Words<kBytes>::type Load;
    constexpr int kRow = value_row<DP>();
    // each wave's values, then its 16 rows of 32-bit results
    constexpr int kSlice = kStep * kRow * 2 > 16 * DP * 4 ? kStep * kRow * 2 : 16 * DP * 4;
    __shared__ __attribute__((aligned(16))) char shared[4 * kSlice];
    __shared__ float join_m[4][16], join_l[4][16];

    // the record is read before the count is known: the array holds one for every workgroup
    const AttnItem it = plan_record(a.items + blockIdx.x);
    const int32_t n_few = plan_record(a.head).n_few;
    asm volatile("" : : "s"(it.kv_len), "s"(n_few));  // both on their way before either is waited for
    if ((int32_t)blockIdx.x >= n_few) return;
    Piece s = piece_of(a, it);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const bool across = it.across != 0;
    if (across) {
        s.head += wave;
        if (s.prow >= 0) s.prow += 16 * wave;
    }
    const int32_t first = across ? 0 : wave, apart = across ? 1 : 4;  // the wave's steps
    const int n = lane & 15, g = lane >> 4;
    T *tile = (T *)(shared + wave * kSlice);

    // The lane's row, and its query as the first product's right operand.  One load of a key row
    // serves kVals / 8 contraction steps: lane group g holds, for step u of load c, columns (4 c + g) kVals + 8 u.
    const uint32_t R = (uint32_t)(s.row0 + (n < s.rows ? n : s.rows - 1));
    const int32_t tok = (int32_t)div_by(R, a.group_magic, a.group_shift);
    const int32_t pos = s.first + tok;
    const RowMask mask = row_mask(a, s, pos);
    float slope = 0.f;
    if (SHAPED && a.slopes) slope = a.slopes[s.head * a.group + (int32_t)R - tok * a.group] * 1.4426950408889634f;

    struct Rows {
        Load r[2][kLoads];
    };
    Rows kr, vr;
    const int32_t i1 = s.tile1 * 2;
    int32_t i = s.tile0 * 2 + first;
    auto start = [&](int32_t i) { return s.walk.start(i >> 1) + (i & 1) * kStep; };
    auto key = [&](int32_t i, int t) { return seen_key(s, start(i) + 16 * t + n); };
    const bool whole_rows = a.dim == DP;
    auto load = [&](Rows &to, const uint8_t *base, const int64_t(&off)[2]) __attribute__((always_inline)) {
        auto one = [&](int t, int c) __attribute__((always_inline)) {
            to.r[t][c] = *(const KVX_GLOBAL Load *)(base + off[t] + (4 * c + g) * kBytes);
        };
        if (whole_rows) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < kLoads; ++c) one(t, c);
        } else {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < kLoads; ++c) {
                    to.r[t][c] = Load{};
                    if ((4 * c + g) * kVals < a.dim) one(t, c);
                }
        }
    };
    // values 8 u .. 8 u + 7 of a load
    auto widen = [&](const Rows &from, int t, int c, int u) __attribute__((always_inline)) {
        return widen8<T, CACHE>(from.r[t][c], u);
    };
    auto put_values = [&]() __attribute__((always_inline)) {  // to shared memory, row-major
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < kLoads; ++c)
#pragma unroll
                for (int u = 0; u < kVals / 8; ++u)
                    *(T8 *)(tile + (16 * t + n) * kRow + (4 * c + g) * kVals + 8 * u) = widen(vr, t, c, u);
    };
    // O^T: column d of keys 16 t + 4 g + r
    const T *const col = tile + (4 * g + (n >> 2)) * kRow + (n & 3) * 4;
    auto value = [&](int d) __attribute__((always_inline)) {
        const T4 lo = read_column<T>(col + 16 * d), hi = read_column<T>(col + 16 * kRow + 16 * d);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    // Infinities and NaN among the values of the step from key j0 on, added where they are seen: where a product
    // of ones, for seen keys and such values, is not zero.
    auto seen_ones = [&](int32_t j0) __attribute__((always_inline)) {
        T8 seen;
#pragma unroll
        for (int k = 0; k < 8; ++k) seen[k] = (T)(mask.sees(j0 + 16 * (k >> 2) + 4 * g + (k & 3)) ? 1.f : 0.f);
        return seen;
    };
    auto add_specials = [&](f32x4 &to, T8 v, T8 seen) __attribute__((always_inline)) {
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {
            const f32x4 c = mfma16(ones_at<T>(v, kind), seen, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int r = 0; r < 4; ++r) to[r] += c[r] != 0.f ? special(kind) : 0.f;
        }
    };
    int64_t off[2] = {0, 0};
    int32_t blk[2] = {0, 0};
    if (i < i1) {
#pragma unroll
        for (int t = 0; t < 2; ++t) blk[t] = block_of(a, s, key(i, t));
#pragma unroll
        for (int t = 0; t < 2; ++t) off[t] = key_offset(a, s, key(i, t), blk[t]);
        load(kr, a.k_base, off);
        load(vr, a.v_base, off);
    }
    if (i + apart < i1) {
#pragma unroll
        for (int t = 0; t < 2; ++t) blk[t] = block_of(a, s, key(i + apart, t));
    }
    T8 q[kS];
    const T *qr = q_row<T>(a, s, n);
#pragma unroll
    for (int c = 0; c < kS; ++c) q[c] = load_q<T>(a, qr, (4 * (8 * c / kVals) + g) * kVals + 8 * c % kVals);

    f32x4 o[DP / 16];
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.f;
    const float sc = SHAPED ? 1.f : a.scale_log2;
    const float slack = 8.f / sc;  // a maximum that grows by less than 2^8 is not worth a rescaling

    for (; i < i1; i += apart) {
        const int32_t j0 = start(i);
        const bool more = i + apart < i1;
        if (more) {
#pragma unroll
            for (int t = 0; t < 2; ++t) off[t] = key_offset(a, s, key(i + apart, t), blk[t]);
        }
        // S^T: keys 16 t + 4 g + r of the step against row n
        f32x4 x[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            x[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < kLoads; ++c)
#pragma unroll
                for (int u = 0; u < kVals / 8; ++u) x[t] = mfma16(widen(kr, t, c, u), q[c * (kVals / 8) + u], x[t]);
        }
        if (more) load(kr, a.k_base, off);
        put_values();
        if (more) load(vr, a.v_base, off);
        if (i + 2 * apart < i1) {
#pragma unroll
            for (int t = 0; t < 2; ++t) blk[t] = block_of(a, s, key(i + 2 * apart, t));
        }
        // the slice is the wave's own and its accesses stay in order: no barrier, but the
        // compiler must not move the reads below above the writes of other lanes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

        const bool masked = !all_see(a, s, j0, kStep);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            auto at = [&](int r) { return j0 + 16 * t + 4 * g + r; };
            if (SHAPED) shape<SHAPED, 4>(a, x[t], slope, pos, at);
            if (masked) hide<4>(x[t], mask, at);
        }
        float mx = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                         fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__any(mx > m + slack || (m == -INFINITY && mx > m))) {
            const float up = fmaxf(m, mx);
            const float by = up == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - up) * sc);
            m = up;
            l *= by;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) o[d] *= keep(by);
        }
        const float mm = m == -INFINITY ? 0.f : m * sc - weight_shift<T>();
        T8 w;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r], sc, -mm));
                l += e;
                w[4 * t + r] = (T)e;
            }
        bool odd = false;
        if (masked) {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) odd |= any_not_finite<T>(value(d));
        }
        if (masked && __any(odd)) {
            // An infinity or NaN among the values: a zero weight would turn it into NaN in rows
            // that do not see it.  So it is left out of the product, and added where it is seen.
            const T8 seen = seen_ones(j0);
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                const T8 v = value(d);
                o[d] = mfma16(only_finite<T>(v), w, o[d]);
                add_specials(o[d], v, seen);
            }
        } else {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) o[d] = mfma16(value(d), w, o[d]);
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    typedef Lost<f32x4, DP / 16> Results;
    if (__builtin_expect(__any(Results::any(o) && l == l), 0)) {
        Results lost;
        lost.clear(o);
        for (i = s.tile0 * 2 + first; i < i1; i += apart) {
#pragma unroll
            for (int t = 0; t < 2; ++t) off[t] = key_offset(a, s, key(i, t), block_of(a, s, key(i, t)));
            load(vr, a.v_base, off);
            put_values();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const T8 seen = seen_ones(start(i));
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) add_specials(o[d], value(d), seen);
        }
        lost.restore(o);
    }

    auto row_of = [&](int row) __attribute__((always_inline)) {
        const uint32_t Rr = (uint32_t)(s.row0 + row);
        const int32_t t_r = (int32_t)div_by(Rr, a.group_magic, a.group_shift);
        return RowPlace{t_r, s.head * a.group + (int32_t)Rr - t_r * a.group};
    };
    finish_few<T, DP, kSlice>(a, s, across, s.rows, row_of, shared, join_m, join_l, m,
                              m == -INFINITY ? m : m * sc - weight_shift<T>(), l, o);
}

// ---- many rows: chunks and prompts ----------------------------------------------

template <int DP>
constexpr int many_waves() { return DP == 256 ? 4 : 8; }

// Shared memory: two tiles of keys and of values, and the row offsets of four tiles.
template <int DP>
constexpr int many_lds() { return KVX_TILE_KEYS * (2 * (key_row<DP>() + value_row<DP>()) * 2 + 4 * 8); }

// 32 rows a wave (32x32x16 products); the workgroup's waves share 64-key tiles of K and V in
// shared memory, two deep.  While tile i is worked on, tile i + 1, which has arrived in
// registers, goes to shared memory, tile i + 2 is sent for, the places of its rows having been
// worked out an iteration before by one wave for all (a lane a key), and the block ids of tile
// i + 4 are fetched by another.  One barrier a tile.
// Bound by the matrix pipe and the vector pipe together (one exponential and four other
// operations for each score): of the cycles a compute unit is busy the matrix pipe works 46 %, the
// vector pipe 42 %, and the two of one SIMD overlap only in part (56 vector operations beside 8
// products take 375 cycles, alone 156 and 292).  Eight waves share a tile so that shared memory is read
// for 256 rows at a time, with no bank conflict; two workgroups of four waves took 15 % longer,
// and half of the waves half a tile behind the others gained nothing.  Measured, bf16, 32 query heads on 8 of
// 128: 8192 tokens 565-585 us, 940-973 TFLOP/s; 2048 tokens on 34816 cached 1120-1157 us,
// 980-1012; the clock falls to 2.0-2.2 GHz meanwhile.  Direct loads to shared memory make the
// compiler wait for all of them before each read, and lost to the way through registers.
// 64-wide heads keep four waves a SIMD, 128 registers: the forms with a cap, slopes or another scale then
// spill 16 to 18 of them (5 to 8 with a large cap), a few scratch accesses a tile.  Measured with four waves
// and spills, an 8192-token prompt: 345 us plain, 575 capped, 530 with slopes.
template <class T, int CACHE, int DP, int SHAPED>
__global__ __launch_bounds__(64 * many_waves<DP>(), DP == 64 ? 4 : DP == 128 ? 2 : 1) void attend_many(const AttnLaunch a)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    constexpr int kWaves = many_waves<DP>();
    constexpr int N = KVX_TILE_KEYS;
    constexpr int kRow = DP / 8;                      // pieces of one key row: eight values each
    constexpr int kLoads = N * kRow / (64 * kWaves);  // loads of a thread for one tile of K or V
    static_assert(kLoads * 64 * kWaves == N * kRow, "whole loads");
    constexpr int kK = key_row<DP>(), kV = value_row<DP>();
    extern __shared__ __attribute__((aligned(16))) char shared[];
    T *const keys = (T *)shared, *const values = keys + 2 * N * kK;  // [2][N][kK], [2][N][kV]
    int64_t *const offs = (int64_t *)(values + 2 * N * kV);          // [4][N]
    __shared__ int32_t odd[2];  // one past the last tile (of either parity) with infinities or NaN in V

    const AttnItem it = plan_record(a.items + blockIdx.x);
    if ((int32_t)blockIdx.x >= plan_record(a.head).n_many) return;
    const Piece s = piece_of(a, it);
    const int32_t n_tiles = s.tile1 - s.tile0;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 31, g = lane >> 5;
    const int rw = wave * 32 + n;  // the lane's row of the piece

    const uint32_t R = (uint32_t)(s.row0 + (rw < s.rows ? rw : s.rows - 1));
    const int32_t tok = (int32_t)div_by(R, a.group_magic, a.group_shift);
    const int32_t head = s.head * a.group + (int32_t)R - tok * a.group;
    const int32_t pos = s.first + tok;
    const RowMask mask = row_mask(a, s, pos);
    float slope = 0.f;
    if (SHAPED && a.slopes) slope = a.slopes[head] * 1.4426950408889634f;
    T8 q[DP / 16];
    const T *qr = q_row<T>(a, s, rw);
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) q[c] = load_q<T>(a, qr, 16 * c + 8 * g);

    f32x16 o[DP / 32];
#pragma unroll
    for (int i = 0; i < DP / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float sc = SHAPED ? 1.f : a.scale_log2;
    const float slack = 8.f / sc;  // a maximum that grows by less than 2^8 is not worth a rescaling

    // The thread's pieces of a tile: eight values of key rows krow + c * kApart.
    struct Piece8 {
        typename Words<cache_bytes<CACHE>(8)>::type r;
        uint32_t e;  // mx4: the scale byte
    };
    constexpr int kApart = 64 * kWaves / kRow;
    const int krow = threadIdx.x / kRow, chunk = threadIdx.x % kRow;
    const bool inside = chunk * 8 < a.dim;  // columns past the rows' width are zeros
    Piece8 kr[kLoads], vr[kLoads];
#pragma unroll
    for (int c = 0; c < kLoads; ++c) kr[c] = vr[c] = Piece8{};
    auto load = [&](Piece8(&r)[kLoads], const uint8_t *base, int32_t i) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            const int64_t off = offs[(i & 3) * N + krow + c * kApart] + chunk * cache_bytes<CACHE>(8);
            if (inside) {
                r[c].r = *(const KVX_GLOBAL decltype(r[c].r) *)(base + off);
                if constexpr (CACHE == kMx4)
                    r[c].e = *(const KVX_GLOBAL uint8_t *)(base + off + (a.dim / 2 + chunk / 4 - chunk * 4));
            }
        }
    };
    auto widen = [&](const Piece8 &r) __attribute__((always_inline)) {
        if constexpr (CACHE == kMx4) return from_mx4<T>(r.r, mx4_scale(r.e));
        else return widen8<T, CACHE>(r.r, 0);
    };
    auto start = [&](int32_t i) __attribute__((always_inline)) { return s.walk.start(s.tile0 + i); };
    auto partly = [&](int32_t i) __attribute__((always_inline)) { return !all_see(a, s, start(i), N); };
    // rows' places: the lane's key of tile i
    auto find = [&](int32_t i) __attribute__((always_inline)) { return block_of(a, s, seen_key(s, start(i) + lane)); };
    auto place = [&](int32_t i, int32_t blk) __attribute__((always_inline)) {
        offs[(i & 3) * N + lane] = key_offset(a, s, seen_key(s, start(i) + lane), blk);
    };
    auto put_keys = [&](int32_t i) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < kLoads; ++c)
            *(T8 *)(keys + ((i & 1) * N + krow + c * kApart) * kK + chunk * 8) = widen(kr[c]);
    };
    auto put_values = [&](int32_t i) __attribute__((always_inline)) {
        T *V = values + (i & 1) * N * kV;
#pragma unroll
        for (int c = 0; c < kLoads; ++c) *(T8 *)(V + (krow + c * kApart) * kV + chunk * 8) = widen(vr[c]);
        if (partly(i)) {
            bool any = false;
#pragma unroll
            for (int c = 0; c < kLoads; ++c) any |= any_not_finite<T>(widen(vr[c]));
            if (any) odd[i & 1] = i + 1;
        }
    };
    int32_t blk = 0;
    // Before tile i is worked on.
    auto stage = [&](int32_t i) __attribute__((always_inline)) {
        if (i + 1 < n_tiles) {
            put_keys(i + 1);
            put_values(i + 1);
        }
        if (i + 2 < n_tiles) {
            load(kr, a.k_base, i + 2);
            load(vr, a.v_base, i + 2);
        }
        if ((i + 3) % kWaves == wave && i + 3 < n_tiles) place(i + 3, blk);
        if ((i + 4) % kWaves == wave && i + 4 < n_tiles) blk = find(i + 4);
    };

    f32x16 x[2];
    T8 w[4];  // the weights of 16 keys each
    // register r of x[t]: key 32 t + 8 (r / 4) + 4 g + r mod 4
    auto scores = [&](int32_t i) __attribute__((always_inline)) {
        const T *K = keys + ((i & 1) * N + n) * kK + 8 * g;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[t][r] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t) x[t] = mfma32(*(const T8 *)(K + 32 * t * kK + 16 * c), q[c], x[t]);
        // reads run kAhead ahead of the products that use them; left to itself the compiler waits
        // for each one
        constexpr int kReads = DP / 8, kAhead = kReads < 8 ? kReads : 8;
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int c = 0; c < kReads - kAhead; ++c) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
    };
    auto weights = [&](int32_t j0, bool masked) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            auto key = [&](int r) { return j0 + 32 * t + 8 * (r >> 2) + 4 * g + (r & 3); };
            if (SHAPED) shape<SHAPED, 16>(a, x[t], slope, pos, key);
            if (masked) hide<16>(x[t], mask, key);
        }
        float mx = x[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, x[t][r]);
        mx = max_of_halves(mx);
        if (__any(mx > m + slack || (m == -INFINITY && mx > m))) {
            const float up = fmaxf(m, mx);
            const float by = up == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - up) * sc);
            m = up;
            l *= by;
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) o[d] *= keep(by);
        }
        const float mm = m == -INFINITY ? 0.f : m * sc - weight_shift<T>();
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r], sc, -mm));
                const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r + 1], sc, -mm));
                sum[0] += e0;
                sum[1] += e1;
                w[2 * t + (r >> 3)][r & 7] = (T)e0;
                w[2 * t + (r >> 3)][(r & 7) + 1] = (T)e1;
            }
        l += sum[0] + sum[1];
    };
    // V^T of 16 keys: slots 0-3 are keys 4 g + 0..3, slots 4-7 keys 8 + 4 g + 0..3
    auto add_values = [&](int32_t i) __attribute__((always_inline)) {
        const T *V = values + ((i & 1) * N + 4 * g + ((lane & 15) >> 2)) * kV + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) {
                const T4 lo = read_column<T>(V + 16 * u * kV + 32 * d), hi = read_column<T>(V + (16 * u + 8) * kV + 32 * d);
                o[d] = mfma32(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), w[u], o[d]);
            }
    };
    // Infinities and NaN among the values of the tile `was` from key j0 on, added where they are seen.
    auto add_specials = [&](const T *was, int32_t j0) __attribute__((always_inline)) {
#pragma unroll 1
        for (int k = 0; k < N; ++k) {
            const bool seen = mask.sees(j0 + k);
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const T4 v = *(const T4 *)(was + k * kV + 32 * d + 8 * b + 4 * g);
                    // the whole vector: a bit cast of one element reads element 0
                    const u16x4 bits = __builtin_bit_cast(u16x4, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[d][4 * b + e] += seen && not_finite<T>(bits[e]) ? (float)v[e] : 0.f;
                }
        }
    };
    // Infinities and NaN among the values of a tile that some rows see in part: a zero weight would
    // turn them into NaN in rows that do not see them.  Before tile i is worked on it is read
    // again; its copy for the product gets zeros in their place, and each row adds those it sees from
    // a copy as it was, in the space of tile i + 1, which is put there afterwards.
    auto specials = [&](int32_t i, auto rows) __attribute__((always_inline)) {
        Piece8 r[kLoads];
#pragma unroll
        for (int c = 0; c < kLoads; ++c) r[c] = Piece8{};
        load(r, a.v_base, i);
        T *V = values + (i & 1) * N * kV, *was = values + ((i + 1) & 1) * N * kV;
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            const T8 v = widen(r[c]);
            *(T8 *)(was + (krow + c * kApart) * kV + chunk * 8) = v;
            *(T8 *)(V + (krow + c * kApart) * kV + chunk * 8) = only_finite<T>(v);
        }
        __syncthreads();
        if (decltype(rows)::value) add_specials(was, start(i));
        __syncthreads();
    };

    if (threadIdx.x < 2) odd[threadIdx.x] = 0;
    for (int32_t i = 0; i < 3 && i < n_tiles; ++i)
        if (i % kWaves == wave) place(i, find(i));
    if (3 % kWaves == wave && 3 < n_tiles) blk = find(3);
    __syncthreads();
    if (n_tiles > 0) {
        load(kr, a.k_base, 0);
        load(vr, a.v_base, 0);
        put_keys(0);
        put_values(0);
        if (1 < n_tiles) {
            load(kr, a.k_base, 1);
            load(vr, a.v_base, 1);
        }
    }
    __syncthreads();
    const bool works = wave * 32 < s.rows;  // a wave without rows only helps loading
    if (!works) {
        for (int32_t i = 0; i < n_tiles; ++i) {
            if (__builtin_expect(odd[i & 1] == i + 1, 0)) specials(i, std::false_type{});
            stage(i);
            __syncthreads();
        }
    } else {
        for (int32_t i = 0; i < n_tiles; ++i) {
            if (__builtin_expect(odd[i & 1] == i + 1, 0)) specials(i, std::true_type{});
            stage(i);
            scores(i);
            weights(start(i), partly(i));
            add_values(i);
            __syncthreads();
        }
    }
    l += __shfl_xor(l, 32);
    typedef Lost<f32x16, DP / 32> Results;
    if (works && __any(Results::any(o) && l == l)) odd[0] = -1;
    __syncthreads();
    if (__builtin_expect(odd[0] == -1, 0)) {
        Results lost;
        if (works) lost.clear(o);
        for (int32_t i = 0; i < n_tiles; ++i) {
            if (wave == 0) place(i, find(i));
            __syncthreads();
            load(vr, a.v_base, i);
#pragma unroll
            for (int c = 0; c < kLoads; ++c) *(T8 *)(values + (krow + c * kApart) * kV + chunk * 8) = widen(vr[c]);
            __syncthreads();
            if (works) add_specials(values, start(i));
        }
        if (works) lost.restore(o);
    }
    if (rw >= s.rows) return;
    const int64_t to_row = (int64_t)s.q_begin + tok;
    const float top = m == -INFINITY ? m : m * sc - weight_shift<T>();
    if (s.prow >= 0) {
        const int64_t pr = (int64_t)s.prow + rw;
        if (g == 0) {
            a.part_ml[2 * pr] = top;
            a.part_ml[2 * pr + 1] = l;
        }
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(f32x4 *)(a.part_o + pr * DP + 32 * d + 8 * r + 4 * g) =
                    f32x4{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
        return;
    }
    if (g == 0) store_lse(a, to_row, head, top, l);
    if (to_row >= a.n_tokens) return;
    const float by = l == 0.f ? 0.f : a.v_scale / l;
    T *to = (T *)a.out + to_row * a.out_token + (int64_t)head * a.out_head;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int at = 32 * d + 8 * r + 4 * g;
            if (at >= a.dim) continue;
            T4 v;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = (T)(o[d][4 * r + k] * by);
            *(T4 *)(to + at) = v;
        }
}

// ---- joining split pieces ---------------------------------------------------------

// One workgroup joins up to KVX_JOIN_ROWS rows of a group.  A thread takes eight columns of a
// row over every kLanes-th part, in one pass with its own running maximum; the threads of a row then
// add up in a fixed order, so the result does not depend on which part ended first.
template <class T, int DP, int ROWS>
__device__ __forceinline__ void join_rows(const AttnLaunch &a, const AttnGroup &gr, int row0)
{
    constexpr int kCols = DP / 8, kLanes = 256 / (ROWS * kCols);
    static_assert(kLanes >= 1, "");
    __shared__ float share_m[kLanes][ROWS], share_l[kLanes][ROWS];
    __shared__ __attribute__((aligned(16))) float share_v[kLanes][ROWS][DP];
    const int d = threadIdx.x % kCols * 8, row = row0 + threadIdx.x / kCols % ROWS;
    const int k0 = threadIdx.x / (kCols * ROWS);
    const bool live = row < gr.rows;
    if (ROWS == 1 && !live) return;
    const int64_t first = (int64_t)gr.prow + (live ? row : 0);
    float m = -INFINITY, l = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int k = k0; k < gr.n_parts; k += kLanes) {
        const int64_t at = first + (int64_t)k * gr.stride;
        const float pm = a.part_ml[2 * at], pl = a.part_ml[2 * at + 1];
        const f32x4 x = *(const f32x4 *)(a.part_o + at * DP + d), y = *(const f32x4 *)(a.part_o + at * DP + d + 4);
        const float up = fmaxf(m, pm);
        // a part that saw nothing holds zeros and no maximum (or NaN, from a score that is none)
        const float was = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - up);
        const float by = pm == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(pm - up);
        m = up;
        l = l * was + pl * by;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = v[i] * keep(was) + x[i] * keep(by);
            v[4 + i] = v[4 + i] * keep(was) + y[i] * keep(by);
        }
    }
    if (kLanes > 1) {
        const int at = row - row0;
        if (d == 0) share_m[k0][at] = m, share_l[k0][at] = l;
        *(f32x4 *)&share_v[k0][at][d] = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4 *)&share_v[k0][at][d + 4] = f32x4{v[4], v[5], v[6], v[7]};
        __syncthreads();
        if (k0 > 0) return;
        constexpr int kUnroll = kLanes < 8 ? kLanes : 8;
        m = -INFINITY;
#pragma unroll
        for (int k = 0; k < kLanes; ++k) m = fmaxf(m, share_m[k][at]);
        l = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll kUnroll
        for (int k = 0; k < kLanes; ++k) {
            const float by = share_m[k][at] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(share_m[k][at] - m);
            l += share_l[k][at] * by;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += share_v[k][at][d + i] * keep(by);
        }
    }
    if (!live) return;
    const uint32_t R = (uint32_t)(gr.row0 + row);
    const int32_t tok = (int32_t)div_by(R, a.group_magic, a.group_shift);
    const int32_t head = gr.head * a.group + (int32_t)R - tok * a.group;
    store_out<T>(a, (int64_t)gr.q_begin + tok, head, d, v, l == 0.f ? 0.f : a.v_scale / l);
    if (d == 0) store_lse(a, (int64_t)gr.q_begin + tok, head, m, l);
}

template <class T, int DP>
__global__ __launch_bounds__(256) void join(const AttnLaunch a)
{
    const AttnGroup gr = plan_record(a.groups + blockIdx.x);
    if ((int32_t)blockIdx.x >= plan_record(a.head).n_groups) return;
    join_rows<T, DP, KVX_JOIN_ROWS>(a, gr, 0);
}

// The same for 4-bit pools, whose long contexts have as many parts as other pools' but took a quarter of the time: where
// there are more than KVX_JOIN_MANY, a record holds one row and all of a workgroup's threads take it.  256 parts of 32 rows: 6.5
// us, 16 to 22 with four rows to a workgroup; up to 31 parts (16 sequences of a decode step) 4.7 either way.
template <class T, int DP>
__global__ __launch_bounds__(256) void join_mx4(const AttnLaunch a)
{
    const AttnGroup gr = plan_record(a.groups + blockIdx.x);
    if ((int32_t)blockIdx.x >= plan_record(a.head).n_groups) return;
    if (gr.n_parts > KVX_JOIN_MANY && gr.rows == 1) join_rows<T, DP, 1>(a, gr, 0);
    else join_rows<T, DP, KVX_JOIN_ROWS>(a, gr, 0);
}

// ---- launches ---------------------------------------------------------------------

template <class T, int DP, int SHAPED>
__global__ void attend_few_mx4(const AttnLaunch a);  // kvxfer_attn_mx4.h

template <class T, int CACHE, int DP>
int launch_attend_dim(const AttnLaunch &a, int which, uint32_t grid, hipStream_t stream)
{
    // one positive scale is folded into the exponential; anything else is shaped first
    const bool plain = a.cap_log2 == 0.f && !a.slopes && a.scale_log2 > 0.f, large = a.cap_inv != 0.f;
    const void *fn;
    size_t lds = 0;
    uint32_t threads = 256;
    if (which == 0) {
        if constexpr (CACHE == kMx4)
            fn = plain   ? (const void *)&attend_few_mx4<T, DP, 0>
             : large ? (const void *)&attend_few_mx4<T, DP, 2>
                     : (const void *)&attend_few_mx4<T, DP, 1>;
        else
            fn = plain   ? (const void *)&attend_few<T, CACHE, DP, 0>
                 : large ? (const void *)&attend_few<T, CACHE, DP, 2>
                         : (const void *)&attend_few<T, CACHE, DP, 1>;
    } else {
        fn = plain   ? (const void *)&attend_many<T, CACHE, DP, 0>
             : large ? (const void *)&attend_many<T, CACHE, DP, 2>
                     : (const void *)&attend_many<T, CACHE, DP, 1>;
        lds = many_lds<DP>();
        threads = 64 * many_waves<DP>();
        const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return (int)e;
    }
    AttnLaunch arg = a;
    void *args[] = {&arg};
    return (int)hipLaunchKernel(fn, dim3(grid), dim3(threads), args, lds, stream);
}

template <class T, int CACHE>
int launch_attend_cache(const AttnLaunch &a, int which, uint32_t grid, hipStream_t stream)
{
    switch (padded_dim(a.dim)) {
    case 64: return launch_attend_dim<T, CACHE, 64>(a, which, grid, stream);
    case 128: return launch_attend_dim<T, CACHE, 128>(a, which, grid, stream);
    default: return launch_attend_dim<T, CACHE, 256>(a, which, grid, stream);
    }
}

template <class T>
int launch_join_type(const AttnLaunch &a, uint32_t grid, hipStream_t stream)
{
    AttnLaunch arg = a;
    void *args[] = {&arg};
    const int dp = padded_dim(a.dim);
    const void *fn = dp == 64    ? (a.mx4 ? (const void *)&join_mx4<T, 64> : (const void *)&join<T, 64>)
                     : dp == 128 ? (a.mx4 ? (const void *)&join_mx4<T, 128> : (const void *)&join<T, 128>)
                                 : (a.mx4 ? (const void *)&join_mx4<T, 256> : (const void *)&join<T, 256>);
    return (int)hipLaunchKernel(fn, dim3(grid), dim3(256), args, 0, stream);
}

}  // namespace kvx

// kvxfer_attn.h -- attention of new tokens over a paged cache: device code, instantiated
// for one query type by kvxfer_attn_f16.hip and kvxfer_attn_bf16.hip.
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

#include "kvxfer_ops.h"

namespace kvx {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define KVX_GLOBAL __attribute__((address_space(1)))
#define KVX_LDS __attribute__((address_space(3)))

template <class T>
struct Vec {
    typedef T x2 __attribute__((ext_vector_type(2)));
    typedef T x4 __attribute__((ext_vector_type(4)));
    typedef T x8 __attribute__((ext_vector_type(8)));
};

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

// Four e4m3 values (one word) as T: every one is a value of both 16-bit types.
template <class T>
__device__ __forceinline__ typename Vec<T>::x4 from_e4m3(uint32_t w)
{
    typedef typename Vec<T>::x2 T2;
    T2 a, b;
    if constexpr (__is_same(T, __bf16)) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true);
    }
    return typename Vec<T>::x4{a[0], a[1], b[0], b[1]};
}

// Whether any of eight 16-bit values is an infinity or a NaN.
template <class T>
__device__ __forceinline__ bool not_finite(typename Vec<T>::x8 v)
{
    constexpr uint32_t e = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & e) == e || (w[i] & (e << 16)) == (e << 16);
    return bad;
}

// 16-bit storage of one tile in shared memory: rows of DP values in 16-byte chunks, chunk c
// of row r at c ^ (r mod chunks), so that reads down a column meet different banks.
template <int DP>
__device__ __forceinline__ int lds_at(int row, int chunk)
{
    constexpr int C = DP / 8, M = C < 16 ? C : 16;
    return row * DP + ((chunk ^ (row & (M - 1))) << 3);
}

// Four consecutive rows of one column, transposed: the 16 lanes of a group read 4 rows of
// 16 values, lane i giving the address of values 4 (i mod 4) .. +3 of row i / 4, and lane i
// receives column i of the four rows.
template <class T>
__device__ __forceinline__ typename Vec<T>::x4 read_column(const T *p)
{
    const i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KVX_LDS i16x4 *)(KVX_LDS void *)p);
    return __builtin_bit_cast(typename Vec<T>::x4, v);
}

// The keys one query sees, as two stretches: [0, prefix) and [low, high].  Compared without
// branches: a mask is three compares and a select.
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

template <int ROWS>
__device__ __forceinline__ Piece load_piece(const AttnLaunch &a)
{
    const AttnItem it = a.items[blockIdx.x];
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
    if (s.rows > ROWS) s.rows = ROWS;
    s.first = s.kv_len - s.q_len;
    s.p0 = s.first + (int32_t)div_by(s.row0, a.group_magic, a.group_shift);
    s.p1 = s.first + (int32_t)div_by(s.row0 + s.rows - 1, a.group_magic, a.group_shift);
    s.walk = key_walk(s.kv_len, s.prefix, a.window, a.full != 0, s.p0, s.p1);
    return s;
}

__device__ __forceinline__ RowMask row_mask(const AttnLaunch &a, const Piece &s, int32_t p)
{
    RowMask m;
    m.low = a.window > 0 ? p - a.window + 1 : 0;
    m.high = a.full || p >= s.kv_len ? s.kv_len - 1 : p;
    m.prefix = s.prefix < s.kv_len ? s.prefix : s.kv_len;
    return m;
}

// Whether any row of the piece sees key j.
__device__ __forceinline__ bool any_sees(const Piece &s, int32_t j)
{
    return j < s.walk.prefix || (j >= s.walk.low && j < s.walk.high);
}

// Whether every row of the piece sees the n keys from j on: the scores need no mask.
__device__ __forceinline__ bool all_see(const AttnLaunch &a, const Piece &s, int32_t j, int32_t n)
{
    if (j + n > s.kv_len) return false;
    if (a.full || j + n <= s.prefix) return true;
    return j + n - 1 <= s.p0 && (a.window == 0 || j > s.p1 - a.window);
}

// Byte offset in a region of key j's row (of the piece's head).  A key that no row sees is
// not looked up: offset -1.  A block id out of range is reported, and block 0 read.
__device__ __forceinline__ int64_t key_offset(const AttnLaunch &a, const Piece &s, int32_t j)
{
    if (!any_sees(s, j)) return -1;
    const uint32_t page = div_by((uint32_t)j, a.bs_magic, a.bs_shift);
    int32_t blk = s.table[page];
    if ((uint32_t)blk >= a.num_blocks) {
        atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
        blk = 0;
    }
    return (int64_t)blk * a.block_stride + (int64_t)((uint32_t)j - page * a.block_size) * a.tok_stride +
           (int64_t)s.head * a.head_stride;
}

// Score transforms other than one positive scale: the tanh cap, the distance slopes, and
// scales that are not positive.  Base-2 scores out.  key(i) is the key of score i.
template <int N, class X, class Key>
__device__ __forceinline__ void shape(const AttnLaunch &a, X &x, float slope_log2, int32_t p, Key key)
{
    if (a.cap_log2 != 0.f) {
#pragma unroll
        for (int i = 0; i < N; ++i)  // tanh y = 1 - 2 / (e^2y + 1)
            x[i] = a.cap_log2 *
                   (1.f - 2.f / (__builtin_amdgcn_exp2f(x[i] * a.scale_log2 * 2.8853900817779268f) + 1.f));
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
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = mask.sees(key(i)) ? x[i] : -INFINITY;
}

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

// At most 16 rows (16x16x32 products).  Four waves take the piece's 32-key steps in turn,
// each with its own running maximum, and join at the end in shared memory.  Bound by the
// cache's bytes: keys go from memory to the first product's registers directly, values through a
// slice of shared memory of the wave's own, both loaded a step ahead, with no barrier in the
// loop.
template <class T, bool E4M3, int DP, bool SHAPED>
__global__ __launch_bounds__(256) void attend_few(const AttnLaunch a)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    constexpr int kStep = 32;                  // keys of one wave's step
    constexpr int kS = DP / 32;                // contraction steps of the first product
    constexpr int kLoads = E4M3 ? DP / 64 : DP / 32;  // 16-byte loads of a lane for one key row
    constexpr int kVals = E4M3 ? 16 : 8;       // values of one load
    __shared__ __attribute__((aligned(16))) char shared[4 * kStep * DP * 2];
    __shared__ float join_m[4][16], join_l[4][16];

    if ((int32_t)blockIdx.x >= a.head->n_few) return;
    const Piece s = load_piece<16>(a);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    T *tile = (T *)(shared + wave * kStep * DP * 2);

    // The lane's row, and its query as the first product's right operand.  Lane group g
    // holds, for contraction step c, columns 32 c + 8 g (16-bit pools) or, so that one
    // 16-byte load of an 8-bit key row serves two steps, 64 (c / 2) + 16 g + 8 (c mod 2).
    const uint32_t R = (uint32_t)(s.row0 + (n < s.rows ? n : s.rows - 1));
    const int32_t tok = (int32_t)div_by(R, a.group_magic, a.group_shift);
    const int32_t pos = s.first + tok;
    const RowMask mask = row_mask(a, s, pos);
    float slope = 0.f;
    if (SHAPED && a.slopes) slope = a.slopes[s.head * a.group + (int32_t)R - tok * a.group] * 1.4426950408889634f;
    T8 q[kS];
    const T *qr = q_row<T>(a, s, n);
#pragma unroll
    for (int c = 0; c < kS; ++c) q[c] = load_q<T>(a, qr, E4M3 ? 64 * (c / 2) + 16 * g + 8 * (c & 1) : 32 * c + 8 * g);

    f32x4 o[DP / 16];
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) o[i] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.f;
    const float sc = SHAPED ? 1.f : a.scale_log2;
    const float slack = 8.f / sc;  // a maximum that grows by less than 2^8 is not worth a rescaling

    u32x4 kr[2][kLoads], vr[2][kLoads];
    const int32_t i1 = s.tile1 * 2;
    int32_t i = s.tile0 * 2 + wave;
    auto start = [&](int32_t i) { return s.walk.start(i >> 1) + (i & 1) * kStep; };
    auto load = [&](u32x4(&r)[2][kLoads], const uint8_t *base, const int64_t(&off)[2]) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < kLoads; ++c) {
                const int d = c * 4 * kVals + g * kVals;
                r[t][c] = u32x4{0, 0, 0, 0};
                if (off[t] >= 0 && d < a.dim) r[t][c] = *(const KVX_GLOBAL u32x4 *)(base + off[t] + c * 64 + g * 16);
            }
    };
    int64_t off[2] = {-1, -1};
    if (i < i1) {
#pragma unroll
        for (int t = 0; t < 2; ++t) off[t] = key_offset(a, s, start(i) + 16 * t + n);
        load(kr, a.k_base, off);
        load(vr, a.v_base, off);
    }
    for (; i < i1; i += 4) {
        const int32_t j0 = start(i);
        const bool more = i + 4 < i1;
        int64_t next[2] = {-1, -1};
        if (more) {
#pragma unroll
            for (int t = 0; t < 2; ++t) next[t] = key_offset(a, s, start(i + 4) + 16 * t + n);
        }
        // S^T: keys 16 t + 4 g + r of the step against row n
        f32x4 x[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            x[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < kLoads; ++c) {
                if constexpr (E4M3) {
                    const T4 w0 = from_e4m3<T>(kr[t][c][0]), w1 = from_e4m3<T>(kr[t][c][1]);
                    const T4 w2 = from_e4m3<T>(kr[t][c][2]), w3 = from_e4m3<T>(kr[t][c][3]);
                    x[t] = mfma16(__builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7), q[2 * c], x[t]);
                    x[t] = mfma16(__builtin_shufflevector(w2, w3, 0, 1, 2, 3, 4, 5, 6, 7), q[2 * c + 1], x[t]);
                } else {
                    x[t] = mfma16(__builtin_bit_cast(T8, kr[t][c]), q[c], x[t]);
                }
            }
        }
        if (more) load(kr, a.k_base, next);
        // V to shared memory, row-major
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < kLoads; ++c) {
                const int row = 16 * t + n;
                if constexpr (E4M3) {
                    const T4 w0 = from_e4m3<T>(vr[t][c][0]), w1 = from_e4m3<T>(vr[t][c][1]);
                    const T4 w2 = from_e4m3<T>(vr[t][c][2]), w3 = from_e4m3<T>(vr[t][c][3]);
                    *(T8 *)(tile + lds_at<DP>(row, 8 * c + 2 * g)) = __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
                    *(T8 *)(tile + lds_at<DP>(row, 8 * c + 2 * g + 1)) =
                        __builtin_shufflevector(w2, w3, 0, 1, 2, 3, 4, 5, 6, 7);
                } else {
                    *(u32x4 *)(tile + lds_at<DP>(row, 4 * c + g)) = vr[t][c];
                }
            }
        if (more) load(vr, a.v_base, next);
        // the slice is the wave's own and its accesses stay in order: no barrier, but the
        // compiler must not move the reads below above the writes of other lanes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

        const bool masked = !all_see(a, s, j0, kStep);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            auto key = [&](int r) { return j0 + 16 * t + 4 * g + r; };
            if (SHAPED) shape<4>(a, x[t], slope, pos, key);
            if (masked) hide<4>(x[t], mask, key);
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
            for (int d = 0; d < DP / 16; ++d) o[d] *= by;
        }
        const float mm = m == -INFINITY ? 0.f : m * sc;
        T8 w;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = __builtin_amdgcn_exp2f(x[t][r] * sc - mm);
                l += e;
                w[4 * t + r] = (T)e;
            }
        // O^T: column d of keys 16 t + 4 g + r
        const T *col = tile + 0;
        auto value = [&](int d) {
            const int row = 4 * g + (n >> 2), c = 2 * d + ((n & 3) >> 1), half = (n & 1) * 4;
            const T4 lo = read_column<T>(col + lds_at<DP>(row, c) + half);
            const T4 hi = read_column<T>(col + lds_at<DP>(row + 16, c) + half);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        bool odd = false;
        if (masked) {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) odd |= not_finite<T>(value(d));
        }
        if (masked && __any(odd)) {
            // An infinity or NaN among the values: a zero weight would turn it into NaN in rows that do not
            // see it, so the keys go one at a time and such rows leave the product out.
            for (int key = 0; key < kStep; ++key) {
                const int slot = (key >> 4) * 4 + (key & 3);
                const bool here = ((key >> 2) & 3) == g, seen = mask.sees(j0 + key);
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    const T8 v = value(d);
                    T8 vk{}, wk{};
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (here && k == slot) vk[k] = v[k], wk[k] = w[k];
                    const f32x4 one = mfma16(vk, wk, f32x4{0, 0, 0, 0});
                    if (seen) o[d] += one;
                }
            }
        } else {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) o[d] = mfma16(value(d), w, o[d]);
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the four waves: their slices hold 16 rows of 32-bit results
    __syncthreads();
    float *part = (float *)shared + wave * 16 * DP;
    if (g == 0) join_m[wave][n] = m == -INFINITY ? m : m * sc, join_l[wave][n] = l;
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, join_m[w][n]);
    const float by = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m * sc - top);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) *(f32x4 *)(part + n * DP + d * 16 + 4 * g) = o[d] * by;
    __syncthreads();
    const int row = threadIdx.x >> 4;
    if (row >= s.rows) return;
    const uint32_t Rr = (uint32_t)(s.row0 + row);
    const int32_t t_r = (int32_t)div_by(Rr, a.group_magic, a.group_shift);
    const int32_t head = s.head * a.group + (int32_t)Rr - t_r * a.group;
    const int64_t to_row = (int64_t)s.q_begin + t_r;
    float sum = 0.f;
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, join_m[w][row]);
#pragma unroll
    for (int w = 0; w < 4; ++w)
        if (join_m[w][row] != -INFINITY) sum += join_l[w][row] * __builtin_amdgcn_exp2f(join_m[w][row] - top);
    for (int d = (threadIdx.x & 15) * 8; d < DP; d += 128) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += ((float *)shared)[(w * 16 + row) * DP + d + k];
        if (s.prow >= 0) {
            float *to = a.part_o + ((int64_t)s.prow + row) * DP + d;
            *(f32x4 *)to = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4 *)(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            store_out<T>(a, to_row, head, d, v, sum == 0.f ? 0.f : a.v_scale / sum);
        }
    }
    if ((threadIdx.x & 15) == 0) {
        if (s.prow >= 0) {
            a.part_ml[2 * ((int64_t)s.prow + row)] = top;
            a.part_ml[2 * ((int64_t)s.prow + row) + 1] = sum;
        } else {
            store_lse(a, to_row, head, top, sum);
        }
    }
}

// ---- many rows: chunks and prompts ----------------------------------------------

// 128 rows, 32 a wave (32x32x16 products); the four waves share 64-key tiles of K and V in
// shared memory, two deep, the next one loaded while the last one is worked on.
template <class T, bool E4M3, int DP, bool SHAPED>
__global__ __launch_bounds__(256) void attend_many(const AttnLaunch a)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    constexpr int N = KVX_TILE_KEYS;
    constexpr int kVals = E4M3 ? 16 : 8;             // values of one 16-byte load
    constexpr int kRow = DP / kVals;                 // loads of one key row
    constexpr int kLoads = N * kRow / 256;           // loads of a thread for one tile
    constexpr int kRows = 256 / kRow;                // key rows between a thread's loads
    extern __shared__ __attribute__((aligned(16))) char shared[];
    T *kt = (T *)shared, *vt = kt + 2 * N * DP;      // [2][N][DP] each

    if ((int32_t)blockIdx.x >= a.head->n_many) return;
    const Piece s = load_piece<KVX_ROWS_MANY>(a);
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
    const float slack = 8.f / sc;

    const int lr = threadIdx.x / kRow, lc = threadIdx.x % kRow;
    u32x4 kr[kLoads], vr[kLoads];
    auto load = [&](int32_t i) {
        const int32_t j0 = s.walk.start(i);
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            const int64_t off = key_offset(a, s, j0 + lr + c * kRows);
            kr[c] = vr[c] = u32x4{0, 0, 0, 0};
            if (off >= 0 && lc * kVals < a.dim) {
                kr[c] = *(const KVX_GLOBAL u32x4 *)(a.k_base + off + lc * 16);
                vr[c] = *(const KVX_GLOBAL u32x4 *)(a.v_base + off + lc * 16);
            }
        }
    };
    auto put = [&](T *tile, const u32x4(&r)[kLoads]) {
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            const int row = lr + c * kRows;
            if constexpr (E4M3) {
                const T4 w0 = from_e4m3<T>(r[c][0]), w1 = from_e4m3<T>(r[c][1]);
                const T4 w2 = from_e4m3<T>(r[c][2]), w3 = from_e4m3<T>(r[c][3]);
                *(T8 *)(tile + lds_at<DP>(row, 2 * lc)) = __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
                *(T8 *)(tile + lds_at<DP>(row, 2 * lc + 1)) = __builtin_shufflevector(w2, w3, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
                *(u32x4 *)(tile + lds_at<DP>(row, lc)) = r[c];
            }
        }
    };
    if (s.tile0 < s.tile1) load(s.tile0);
    for (int32_t i = s.tile0; i < s.tile1; ++i) {
        const int buf = (i - s.tile0) & 1;
        T *K = kt + buf * N * DP, *V = vt + buf * N * DP;
        put(K, kr);
        put(V, vr);
        __syncthreads();
        if (i + 1 < s.tile1) load(i + 1);

        const int32_t j0 = s.walk.start(i);
        f32x16 x[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int r = 0; r < 16; ++r) x[t][r] = 0.f;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c)
                x[t] = mfma32(*(const T8 *)(K + lds_at<DP>(32 * t + n, 2 * c + g)), q[c], x[t]);
        }
        // register r of tile t: key 32 t + 8 (r / 4) + 4 g + r mod 4
        const bool masked = !all_see(a, s, j0, N);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            auto key = [&](int r) { return j0 + 32 * t + 8 * (r >> 2) + 4 * g + (r & 3); };
            if (SHAPED) shape<16>(a, x[t], slope, pos, key);
            if (masked) hide<16>(x[t], mask, key);
        }
        float mx = x[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, x[t][r]);
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__any(mx > m + slack || (m == -INFINITY && mx > m))) {
            const float up = fmaxf(m, mx);
            const float by = up == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - up) * sc);
            m = up;
            l *= by;
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) o[d] *= by;
        }
        const float mm = m == -INFINITY ? 0.f : m * sc;
        T8 w[4];  // the weights of 16 keys each
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = __builtin_amdgcn_exp2f(x[t][r] * sc - mm);
                l += e;
                w[2 * t + (r >> 3)][r & 7] = (T)e;
            }
        // V^T of 16 keys: slots 0-3 are keys 4 g + 0..3, slots 4-7 keys 8 + 4 g + 0..3
        auto value = [&](int d, int u) {
            const int row = 16 * u + 4 * g + ((lane & 15) >> 2);
            const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), half = (lane & 1) * 4;
            const T4 lo = read_column<T>(V + lds_at<DP>(row, c) + half);
            const T4 hi = read_column<T>(V + lds_at<DP>(row + 8, c) + half);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        bool odd = false;
        if (masked) {
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                for (int u = 0; u < 4; ++u) odd |= not_finite<T>(value(d, u));
        }
        if (masked && __any(odd)) {
            // as in attend_few: one key at a time, left out by the rows that do not see it
#pragma unroll
            for (int u = 0; u < 4; ++u)
                for (int key = 0; key < 16; ++key) {
                    const int slot = (key >> 3) * 4 + (key & 3);
                    const bool here = ((key >> 2) & 1) == g, seen = mask.sees(j0 + 16 * u + key);
#pragma unroll
                    for (int d = 0; d < DP / 32; ++d) {
                        const T8 v = value(d, u);
                        T8 vk{}, wk{};
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (here && k == slot) vk[k] = v[k], wk[k] = w[u][k];
                        f32x16 one;
#pragma unroll
                        for (int r = 0; r < 16; ++r) one[r] = 0.f;
                        one = mfma32(vk, wk, one);
                        if (seen) o[d] += one;
                    }
                }
        } else {
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[d] = mfma32(value(d, u), w[u], o[d]);
        }
    }
    l += __shfl_xor(l, 32);
    if (rw >= s.rows) return;
    const int64_t row = (int64_t)s.q_begin + tok;
    if (s.prow >= 0) {
        const int64_t pr = (int64_t)s.prow + rw;
        if (g == 0) {
            a.part_ml[2 * pr] = m == -INFINITY ? m : m * sc;
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
    if (g == 0) store_lse(a, row, head, m == -INFINITY ? m : m * sc, l);
    if (row >= a.n_tokens) return;
    const float by = l == 0.f ? 0.f : a.v_scale / l;
    T *to = (T *)a.out + row * a.out_token + (int64_t)head * a.out_head;
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

// One workgroup joins one group: a thread takes eight columns of a row, over all parts in
// order, so the result does not depend on which part ended first.
template <class T, int DP>
__global__ __launch_bounds__(256) void join(const AttnLaunch a)
{
    if ((int32_t)blockIdx.x >= a.head->n_groups) return;
    const AttnGroup gr = a.groups[blockIdx.x];
    for (int c = threadIdx.x; c < gr.rows * (DP / 8); c += 256) {
        const int row = c / (DP / 8), d = c % (DP / 8) * 8;
        float top = -INFINITY;
        for (int k = 0; k < gr.n_parts; ++k)
            top = fmaxf(top, a.part_ml[2 * ((int64_t)gr.prow + (int64_t)k * gr.stride + row)]);
        float l = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int k = 0; k < gr.n_parts; ++k) {
            const int64_t pr = (int64_t)gr.prow + (int64_t)k * gr.stride + row;
            const float m = a.part_ml[2 * pr];
            if (m == -INFINITY) continue;  // this part saw nothing
            const float by = __builtin_amdgcn_exp2f(m - top);
            l += a.part_ml[2 * pr + 1] * by;
            const f32x4 x = *(const f32x4 *)(a.part_o + pr * DP + d), y = *(const f32x4 *)(a.part_o + pr * DP + d + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += x[i] * by, v[4 + i] += y[i] * by;
        }
        const uint32_t R = (uint32_t)(gr.row0 + row);
        const int32_t tok = (int32_t)div_by(R, a.group_magic, a.group_shift);
        const int32_t head = gr.head * a.group + (int32_t)R - tok * a.group;
        store_out<T>(a, (int64_t)gr.q_begin + tok, head, d, v, l == 0.f ? 0.f : a.v_scale / l);
        if (d == 0) store_lse(a, (int64_t)gr.q_begin + tok, head, top, l);
    }
}

// ---- launches ---------------------------------------------------------------------

template <class T, bool E4M3, int DP>
int launch_attend_dim(const AttnLaunch &a, int which, uint32_t grid, hipStream_t stream)
{
    // one positive scale is folded into the exponential; anything else is shaped first
    const bool plain = a.cap_log2 == 0.f && !a.slopes && a.scale_log2 > 0.f;
    const void *fn;
    size_t lds = 0;
    if (which == 0) {
        fn = plain ? (const void *)&attend_few<T, E4M3, DP, false> : (const void *)&attend_few<T, E4M3, DP, true>;
    } else {
        fn = plain ? (const void *)&attend_many<T, E4M3, DP, false> : (const void *)&attend_many<T, E4M3, DP, true>;
        lds = 4 * KVX_TILE_KEYS * DP * sizeof(T);
        const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return (int)e;
    }
    AttnLaunch arg = a;
    void *args[] = {&arg};
    return (int)hipLaunchKernel(fn, dim3(grid), dim3(256), args, lds, stream);
}

template <class T>
int launch_attend_type(const AttnLaunch &a, int which, bool e4m3, uint32_t grid, hipStream_t stream)
{
    switch (padded_dim(a.dim)) {
    case 64:
        return e4m3 ? launch_attend_dim<T, true, 64>(a, which, grid, stream)
                    : launch_attend_dim<T, false, 64>(a, which, grid, stream);
    case 128:
        return e4m3 ? launch_attend_dim<T, true, 128>(a, which, grid, stream)
                    : launch_attend_dim<T, false, 128>(a, which, grid, stream);
    default:
        return e4m3 ? launch_attend_dim<T, true, 256>(a, which, grid, stream)
                    : launch_attend_dim<T, false, 256>(a, which, grid, stream);
    }
}

template <class T>
int launch_join_type(const AttnLaunch &a, uint32_t grid, hipStream_t stream)
{
    AttnLaunch arg = a;
    void *args[] = {&arg};
    const int dp = padded_dim(a.dim);
    const void *fn = dp == 64    ? (const void *)&join<T, 64>
                     : dp == 128 ? (const void *)&join<T, 128>
                                 : (const void *)&join<T, 256>;
    return (int)hipLaunchKernel(fn, dim3(grid), dim3(256), args, 0, stream);
}

}  // namespace kvx

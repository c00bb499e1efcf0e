// kvxfer_rotate.hip -- kernels that turn heads to their positions: new tokens appended with their rotation, cached
// keys moved to other positions; appends to mx4 pools, and cached tokens read back as 16-bit rows.
//
// Mathematics.  Pair (x, y) of a head at position p becomes (x c - y s, x s + y c) with c + i s = amplitude
// e^(2 pi i p f), f the turns of a pair in one position.  f is a fraction of 64 bits, so p f is an exact
// product modulo one turn: position 2^31 is as good as position 1 to 2^-33 turns.  The fraction's two top
// bits choose the quarter, and what is left of it, all 62 bits, within an eighth of a turn of zero, goes through the power series of
// sine and cosine: to x^9 and x^10 in 32 bits (2^-29 and 2^-32 beyond them), to x^15 and x^16 in 64.  The sine is good relative to
// itself, so that pairs of the slowest frequencies turn by what they should.
//
// Keys on their way into an mx4 pool turn in 64 bits and are then rounded to 32 bits towards the odd neighbour, from which
// the rounding to 4 bits gives the same as from all 64: so a stored value is that of the formula, with the amplitude's 32
// bits, except where the formula lies within 2^-45 or so of a border between two values (2^-22 or so below 2^-126, where 32 bits
// hold fewer digits).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kvxfer_device.h"

namespace kvx {

static constexpr int kThreads = 256;
static constexpr int kMaxPairs = KV_MAX_ATTN_DIM / 2;

// ---- angles ------------------------------------------------------------------

// The quarter a fraction of a turn lies nearest to, and the turn's cosine and sine from those of the rest.
template <class F>
__device__ __forceinline__ void of_quarter(uint32_t quarter, F c, F s, F amplitude, F &cos, F &sin)
{
    const F x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    cos = ((quarter + 1) & 2 ? -x : x) * amplitude;
    sin = (quarter & 2 ? -y : y) * amplitude;
}

__device__ __forceinline__ float2 turn32(uint64_t turns, float amplitude)
{
    // two words with signs of their own, the upper one rounded: small angles of either sign lie in the lower one whole
    const uint32_t t = (uint32_t)((turns + 0x80000000u) >> 32), quarter = (t + 0x20000000u) >> 30;
    const float rest = __builtin_fmaf((float)(int32_t)(uint32_t)turns, 0x1p-32f, (float)(int32_t)(t - (quarter << 30)));
    const float x = rest * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = x * x;
    float s = __builtin_fmaf(z, 1.f / 362880, -1.f / 5040);
    s = __builtin_fmaf(z, s, 1.f / 120);
    s = __builtin_fmaf(z, s, -1.f / 6);
    s = __builtin_fmaf(z * x, s, x);
    float c = __builtin_fmaf(z, -1.f / 3628800, 1.f / 40320);
    c = __builtin_fmaf(z, c, -1.f / 720);
    c = __builtin_fmaf(z, c, 1.f / 24);
    c = __builtin_fmaf(z, c, -1.f / 2);
    c = __builtin_fmaf(z, c, 1.f);
    float2 r;
    of_quarter(quarter & 3, c, s, amplitude, r.x, r.y);
    return r;
}

__device__ __forceinline__ double2 turn64(uint64_t turns, float amplitude)
{
    const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
    const double x = (double)(int64_t)(turns - ((uint64_t)quarter << 62)) * 3.4061215800304446e-19;  // 2 pi / 2^64
    const double z = x * x;
    double s = -1.0 / 1307674368000.0;
    s = __builtin_fma(z, s, 1.0 / 6227020800.0);
    s = __builtin_fma(z, s, -1.0 / 39916800.0);
    s = __builtin_fma(z, s, 1.0 / 362880.0);
    s = __builtin_fma(z, s, -1.0 / 5040.0);
    s = __builtin_fma(z, s, 1.0 / 120.0);
    s = __builtin_fma(z, s, -1.0 / 6.0);
    s = __builtin_fma(z * x, s, x);
    double c = 1.0 / 20922789888000.0;
    c = __builtin_fma(z, c, -1.0 / 87178291200.0);
    c = __builtin_fma(z, c, 1.0 / 479001600.0);
    c = __builtin_fma(z, c, -1.0 / 3628800.0);
    c = __builtin_fma(z, c, 1.0 / 40320.0);
    c = __builtin_fma(z, c, -1.0 / 720.0);
    c = __builtin_fma(z, c, 1.0 / 24.0);
    c = __builtin_fma(z, c, -1.0 / 2.0);
    c = __builtin_fma(z, c, 1.0);
    double2 r;
    of_quarter(quarter & 3, c, s, (double)amplitude, r.x, r.y);
    return r;
}

__device__ __forceinline__ uint64_t turns_of(const Rotation &r, int32_t pos, uint32_t pair)
{
    return (uint64_t)(int64_t)pos * r.turns[pair];
}

// ---- heads -------------------------------------------------------------------

// A row is worked on in units of two runs of VEC elements, so that a unit holds whole pairs: 8, 16 bytes of a 16-bit row
// each, where the pairs are a multiple of 8 and the row one of 16, else 4.  Unit j of paired halves holds elements VEC j ..
// and their partners pairs + VEC j ..; behind the pairs, and of neighbours paired, 2 VEC j .. 2 VEC j + 2 VEC - 1.
template <bool ADJACENT, int VEC>
struct Unit {
    uint32_t a, b;  // first element of either run
    bool turns;
    __device__ __forceinline__ Unit(uint32_t j, uint32_t pairs)
    {
        turns = j < pairs / VEC;
        a = !ADJACENT && turns ? VEC * j : 2 * VEC * j;
        b = !ADJACENT && turns ? pairs + VEC * j : 2 * VEC * j + VEC;
    }
};
inline int unit_vec(uint32_t pairs, int32_t dim) { return pairs % 8 == 0 && dim % 16 == 0 ? 8 : 4; }

// The values of a unit turned; cs holds its pairs.
template <bool ADJACENT, int VEC>
__device__ __forceinline__ void turn_unit(float (&x)[2 * VEC], const float2 *cs)
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float &u = x[ADJACENT ? 2 * i : i], &v = x[ADJACENT ? 2 * i + 1 : i + VEC];
        const float c = cs[i].x, s = cs[i].y, y = u;
        u = __builtin_fmaf(y, c, -(v * s));
        v = __builtin_fmaf(y, s, v * c);
    }
}

// 64 bits to 32, to the neighbour with an odd last bit unless exact: what is rounded again to fewer bits than 23 is as if
// rounded once.
__device__ __forceinline__ float to_odd(double x)
{
    uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint64_t rest = b & 0x1fffffffull;
    b = (b & ~0x1fffffffull) | (rest ? 0x20000000ull : 0);
    return (float)__builtin_bit_cast(double, b);
}

// Turned values may pass the range of 32 bits, where a group's scale need not: such a group (its scale came out as that of an
// infinity) is turned again at 2^-kDown of its size, values past what the largest scale holds cut to that, 7 * 2^127.
// Infinities and NaN pass.
static constexpr int kDown = 8;
__device__ __forceinline__ float to_odd_cut(double x)
{
    constexpr double kMost = 7 * 0x1p119;
    return to_odd(__builtin_fabs(x) < __builtin_inf() ? __builtin_fmin(__builtin_fmax(x, -kMost), kMost) : x);
}

// Eight consecutive values from element e on, turned in 64 bits: `x` themselves, `other` those that
// are `pairs` away (only where halves are paired).
template <bool ADJACENT, class Round>
__device__ __forceinline__ void turn_wide(float (&x)[8], const float (&other)[8], uint32_t e, uint32_t pairs, const double2 *cs,
                                          Round round)
{
    if (ADJACENT) {
        if (e >= 2 * pairs) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double2 t = cs[e / 2 + i];
            const double u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = round(__builtin_fma(u, t.x, -(v * t.y)));
            x[2 * i + 1] = round(__builtin_fma(u, t.y, v * t.x));
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t at = e + 4 * h;
        if (at >= 2 * pairs) continue;
        const bool low = at < pairs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double2 t = cs[(low ? at : at - pairs) + i];
            const double u = x[4 * h + i], v = other[4 * h + i];
            // the same products and sums as for the pair's other element's unit: x c - y s, x s + y c
            x[4 * h + i] = round(low ? __builtin_fma(u, t.x, -(v * t.y)) : __builtin_fma(v, t.y, u * t.x));
        }
    }
}
// The element that pairs with e, for a run of four (pairs is a multiple of four).
__device__ __forceinline__ uint32_t partner(uint32_t e, uint32_t pairs)
{
    return e < pairs ? e + pairs : e < 2 * pairs ? e - pairs : e;
}

// A run of elements: as it lies in memory, as values, and back.
template <class E, int N>
struct Run {
    typedef E type __attribute__((ext_vector_type(N)));
};
template <class T, int N>
__device__ __forceinline__ void values_of(float *x, typename Run<T, N>::type v)
{
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)v[i];
}
template <class T, int N>
__device__ __forceinline__ typename Run<T, N>::type run_of(const float *x)
{
    typename Run<T, N>::type v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (T)x[i];
    return v;
}

// A store past the caches, of turned queries and of rows that were read: what lies in the caches stays there, and nothing is
// written back when the kernel ends.  With whoever reads it next in the same measurement: a layer's append and attention of
// 2048, 8192 and 16384 new tokens 89, 630 and 2293 us, queries through the caches 88, 630 and 2298; of 64 decode
// steps 105.0 and 105.2; reads of 7874 tokens of a 4-bit pool with copies of them 95.4 and 94.3, of 32 layers of 4000 262
// and 284.  New keys and values go through the caches, where the attention finds them: past them those layers take 92, 637 and
// 2311 us, a decode step 104.9.
template <class E, class V>
__device__ __forceinline__ void store_past(E *to, V v)
{
    __builtin_nontemporal_store(v, (V *)to);
}

// x / scale in 32 bits (correctly rounded), clamped to +-448; NaN passes by the bounds.
__device__ __forceinline__ float e4m3_of(float x, float scale)
{
    const float y = x / scale;
    return y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
}
__device__ __forceinline__ uint32_t to_e4m3_word(const float *x, float scale)
{
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_of(x[0], scale), e4m3_of(x[1], scale), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_of(x[2], scale), e4m3_of(x[3], scale), p, true);
}

template <int N>
__device__ __forceinline__ typename Run<uint8_t, N>::type to_e4m3(const float *x, float scale)
{
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = to_e4m3_word(x + 4 * i, scale);
    return __builtin_bit_cast(typename Run<uint8_t, N>::type, w);
}
template <int N>
__device__ __forceinline__ void values_of_e4m3(float *x, typename Run<uint8_t, N>::type v)
{
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) w |= (uint32_t)v[4 * i + k] << (8 * k);
        const Vec<__bf16>::x4 y = from_e4m3<__bf16>(w);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[4 * i + k] = (float)y[k];
    }
}

// ---- append with a rotation on the way --------------------------------------------

// A workgroup's tokens, of an item's: 2^lg_split workgroups to an item.
struct Part {
    int32_t item, begin;
    int32_t count;  // below 1: none
    __device__ __forceinline__ Part(const AttnLaunch &a, uint32_t lg_split, AppendItem *it)
    {
        item = (int32_t)(blockIdx.x >> lg_split);
        begin = (int32_t)(blockIdx.x & ((1u << lg_split) - 1)) * (KVX_APPEND_TOKENS >> lg_split);
        count = 0;
        if (item >= plan_record(a.head).n_append) return;
        *it = plan_record(a.append + item);
        count = min(it->count - begin, KVX_APPEND_TOKENS >> lg_split);
    }
};
// Layers to a workgroup: `most` where KVX_DEEP_GROUPS workgroups remain (a decode step of 16 tokens with its four layers
// read: 141.0 us with a layer each, 142.4 with all in one), and no more than 65535 along y.
inline int32_t layers_of(int64_t most, int64_t groups, int32_t layers)
{
    return (int32_t)std::max<int64_t>({1, std::min(most, groups * layers / KVX_DEEP_GROUPS), (layers + 65534) / 65535});
}
// Two tokens to a workgroup; all eight where a token's units are few (32 layers of 2860 tokens of 2 heads read: 12.9 us,
// 11.7; of 8 heads, one layer: 10.8, 13.2).
inline uint32_t lg_split(uint32_t units) { return units <= KVX_FEW_UNITS ? 0 : 2; }
static_assert(KVX_APPEND_SPLIT == 4, "lg_split");

// One new token's place in its region, from the region's row of head 0 on; its block id has been read.
__device__ __forceinline__ int64_t place_of(const AttnLaunch &a, uint32_t pos, int32_t blk)
{
    return (int64_t)blk * a.block_stride + (int64_t)(pos - div_by(pos, a.bs_magic, a.bs_shift) * a.block_size) * a.tok_stride;
}

// A workgroup's units of a token: keys, values and queries, or, in mx4 pools, queries alone, in one sequence over all tokens.
template <class T, int CACHE, bool ADJACENT, int VEC>
struct AppendUnit {
    uint32_t u, c, h, j, units;
    bool there, key, query;
    __device__ __forceinline__ AppendUnit(const AppendRotated &x, uint32_t i, uint32_t count, int64_t row0)
    {
        const AttnLaunch &a = x.attn;
        units = (uint32_t)a.dim / (2 * VEC);
        const uint32_t kv = CACHE == kMx4 ? 0 : units * (uint32_t)a.heads;
        const uint32_t all = 2 * kv + (a.q ? units * (uint32_t)(a.heads * a.group) : 0);
        u = div_by(i, x.all_magic, x.all_shift);
        c = i - u * all;
        there = i < count * all && row0 + u < a.n_tokens;
        key = c < kv;
        query = c >= 2 * kv;
        const uint32_t hc = key ? c : query ? c - 2 * kv : c - kv;
        h = div_by(hc, x.unit_magic, x.unit_shift);
        j = hc - h * units;
    }
};
// The same of an mx4 pool's keys and values: eight consecutive elements to a thread, a group to four of them.
struct AppendEight {
    uint32_t u, c, h, e;
    bool there, key;
    __device__ __forceinline__ AppendEight(const AppendRotated &x, uint32_t i, uint32_t count, int64_t row0)
    {
        const AttnLaunch &a = x.attn;
        const uint32_t eights = (uint32_t)a.dim / 8, each = eights * (uint32_t)a.heads;
        u = div_by(i, x.each_magic, x.each_shift);
        c = i - u * 2 * each;
        there = i < count * 2 * each && row0 + u < a.n_tokens;
        key = c < each;
        const uint32_t hc = key ? c : c - each;
        h = div_by(hc, x.eight_magic, x.eight_shift);
        e = 8 * (hc - h * eights);
    }
};

// A workgroup works out the angles of its tokens once, for all heads, and then streams their units through, kAhead (of mx4
// keys and values kAhead8) of them loaded by a thread before the first is turned.  An mx4 pool's keys and values, with angles
// and sums of 64 bits, and the queries have workgroups of their own (blockIdx.y): the first loads of the former are on their
// way while the angles are worked out.
// Bound by HBM: 8192 new tokens of 32 heads on 8, 128 wide, 201 MB, in 34.7 us (5.8 TB/s); queries too through the caches 45 us.
// Into an e4m3 pool the quotients' instructions count: 4326 tokens, 97 MB, 20.8 us.  Into an mx4 pool 7874 tokens, 169 MB, in
// 31.6 us (5.3 TB/s); keys, values and queries in one workgroup after another: 36 us, and 5.7 us instead of 4.3 for the 16
// tokens of a decode step.  Loads ahead of the angles of 32 bits cost registers and give nothing (33.6 -> 35.0 us, all stores
// past the caches).
template <class T, int CACHE, bool ADJACENT, int VEC>
__global__ __launch_bounds__(kThreads) void append_rotated(const AppendRotated x)
{
    typedef typename Run<T, VEC>::type TV;
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    typedef AppendUnit<T, CACHE, ADJACENT, VEC> At;
    constexpr bool MX4 = CACHE == kMx4;
    constexpr int kAhead = 3, kAhead8 = 2;
    __shared__ float2 cs[KVX_APPEND_TOKENS][kMaxPairs];
    __shared__ double2 cs64[MX4 ? KVX_APPEND_TOKENS : 1][MX4 ? kMaxPairs : 1];
    const AttnLaunch &a = x.attn;
    AppendItem it;
    const Part part(a, x.lg_split, &it);
    if (part.count < 1) return;
    const uint32_t begin = part.begin, count = part.count, pairs = x.rot.pairs;
    const int64_t row0 = (int64_t)it.row + begin;
    const uint32_t pos0 = (uint32_t)it.pos + begin;
    const uint32_t units = (uint32_t)a.dim / (2 * VEC);
    const bool wide = MX4 && blockIdx.y == 0;
    const uint32_t all = wide ? 0 : units * (uint32_t)a.heads * ((MX4 ? 0 : 2) + (a.q ? (uint32_t)a.group : 0));
    const uint32_t eights = wide ? 2 * ((uint32_t)a.dim / 8) * (uint32_t)a.heads : 0;
    auto row_of = [&](const auto &at, bool key, bool query) __attribute__((always_inline)) -> const T * {
        const int64_t row = row0 + at.u;
        return query ? (const T *)a.q + row * a.q_token + (int64_t)at.h * a.q_head
               : key ? (const T *)a.k_new + row * a.k_token + (int64_t)at.h * a.k_head
                     : (const T *)a.v_new + row * a.v_token + (int64_t)at.h * a.v_head;
    };
    auto block_of = [&](uint32_t u) __attribute__((always_inline)) { return it.table[div_by(pos0 + u, a.bs_magic, a.bs_shift)]; };

    TV va[kAhead], vb[kAhead];
    int32_t blk[kAhead];
    auto ask = [&](uint32_t i0) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
            const At at(x, i0 + m * kThreads, count, row0);
            if (!at.there) continue;
            const Unit<ADJACENT, VEC> unit(at.j, at.key || at.query ? pairs : 0);
            const T *from = row_of(at, at.key, at.query);
            va[m] = *(const TV *)(from + unit.a);
            vb[m] = *(const TV *)(from + unit.b);
            blk[m] = 0;
            if (!at.query) blk[m] = block_of(at.u);
        }
    };
    T8 v8[kAhead8];
    T4 o4[kAhead8][2];
    int32_t blk8[kAhead8];
    auto ask8 = [&](uint32_t i0) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < kAhead8; ++m) {
            const AppendEight at(x, i0 + m * kThreads, count, row0);
            if (!at.there) continue;
            const T *from = row_of(at, at.key, false);
            v8[m] = *(const T8 *)(from + at.e);
            if (at.key && !ADJACENT) {
                o4[m][0] = *(const T4 *)(from + partner(at.e, pairs));
                o4[m][1] = *(const T4 *)(from + partner(at.e + 4, pairs));
            }
            blk8[m] = block_of(at.u);
        }
    };
    if (wide) ask8(threadIdx.x);
    for (uint32_t i = threadIdx.x; i < count * pairs; i += kThreads) {
        const uint32_t u = div_by(i, x.pair_magic, x.pair_shift), pair = i - u * pairs;
        if (row0 + u >= a.n_tokens) continue;
        const int32_t pos = x.positions ? x.positions[row0 + u] : (int32_t)(pos0 + u);
        const uint64_t t = turns_of(x.rot, pos, pair);
        if (!wide) cs[u][pair] = turn32(t, x.rot.amplitude);
        else if constexpr (MX4) cs64[u][pair] = turn64(t, x.rot.amplitude);
    }
    __syncthreads();

    if constexpr (MX4) {
        for (uint32_t i0 = threadIdx.x; i0 < count * eights;) {
#pragma unroll
            for (int m = 0; m < kAhead8; ++m) {
                const AppendEight at(x, i0 + m * kThreads, count, row0);
                if (!at.there) continue;
                if ((uint32_t)blk8[m] >= a.num_blocks) {
                    if (at.c == 0) atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
                    continue;
                }
                float v[8], other[8] = {};
                values_of<T, 8>(v, v8[m]);
                if (at.key && !ADJACENT) {
                    values_of<T, 4>(other, o4[m][0]);
                    values_of<T, 4>(other + 4, o4[m][1]);
                }
                if (at.key) turn_wide<ADJACENT>(v, other, at.e, pairs, cs64[at.u], to_odd);
                uint8_t *to = (at.key ? a.k_base : a.v_base) + place_of(a, pos0 + at.u, blk8[m]) + (int64_t)at.h * a.head_stride;
                uint32_t s = mx4_scale_of(v), down = 0;
                if (__builtin_expect(s == 255, 0)) {  // the same of the four lanes of a group
                    const T *from = row_of(at, at.key, false);  // again: kept, it would take registers of every other group
                    values_of<T, 8>(v, *(const T8 *)(from + at.e));
                    if (at.key && !ADJACENT) {
                        values_of<T, 4>(other, *(const T4 *)(from + partner(at.e, pairs)));
                        values_of<T, 4>(other + 4, *(const T4 *)(from + partner(at.e + 4, pairs)));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= 1.f / (1 << kDown), other[i] *= 1.f / (1 << kDown);
                    if (at.key) turn_wide<ADJACENT>(v, other, at.e, pairs, cs64[at.u], to_odd_cut);
                    s = mx4_scale_of(v);
                    down = s == 255 ? 0 : kDown;
                }
                *(uint32_t *)(to + at.e / 2) = to_mx4(v, s);
                s += down;
                if (at.e % 32 == 0) to[a.dim / 2 + at.e / 32] = (uint8_t)s;
            }
            i0 += kAhead8 * kThreads;
            if (i0 < count * eights) ask8(i0);
        }
    }
    if (wide) return;
    ask(threadIdx.x);
    for (uint32_t i0 = threadIdx.x; i0 < count * all;) {
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
            const At at(x, i0 + m * kThreads, count, row0);
            if (!at.there) continue;
            const Unit<ADJACENT, VEC> unit(at.j, at.key || at.query ? pairs : 0);
            float v[2 * VEC];
            values_of<T, VEC>(v, va[m]);
            values_of<T, VEC>(v + VEC, vb[m]);
            if (unit.turns) turn_unit<ADJACENT, VEC>(v, &cs[at.u][VEC * at.j]);
            if (at.query) {
                T *to = (T *)a.out + (row0 + at.u) * a.out_token + (int64_t)at.h * a.out_head;
                store_past(to + unit.a, run_of<T, VEC>(v));
                store_past(to + unit.b, run_of<T, VEC>(v + VEC));
                continue;
            }
            if ((uint32_t)blk[m] >= a.num_blocks) {
                if (at.c == 0) atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
                continue;
            }
            uint8_t *to = (at.key ? a.k_base : a.v_base) + place_of(a, pos0 + at.u, blk[m]) + (int64_t)at.h * a.head_stride;
            if constexpr (CACHE == kE4m3) {
                const float scale = at.key ? a.k_scale : a.v_scale;
                *(typename Run<uint8_t, VEC>::type *)(to + unit.a) = to_e4m3<VEC>(v, scale);
                *(typename Run<uint8_t, VEC>::type *)(to + unit.b) = to_e4m3<VEC>(v + VEC, scale);
            } else {
                *(TV *)((T *)to + unit.a) = run_of<T, VEC>(v);
                *(TV *)((T *)to + unit.b) = run_of<T, VEC>(v + VEC);
            }
        }
        i0 += kAhead * kThreads;
        if (i0 < count * all) ask(i0);
    }
}

template <class T, bool ADJACENT, int VEC>
const void *append_kernel(int kv_type)
{
    switch (cache_of(kv_type)) {
    case kMx4: return (const void *)&append_rotated<T, kMx4, ADJACENT, VEC>;
    case kE4m3: return (const void *)&append_rotated<T, kE4m3, ADJACENT, VEC>;
    default: return (const void *)&append_rotated<T, kHalves, ADJACENT, VEC>;
    }
}
template <class T>
const void *append_kernel(int kv_type, bool adjacent, int vec)
{
    return adjacent ? (vec == 8 ? append_kernel<T, true, 8>(kv_type) : append_kernel<T, true, 4>(kv_type))
                    : (vec == 8 ? append_kernel<T, false, 8>(kv_type) : append_kernel<T, false, 4>(kv_type));
}

int launch_append_rotated(const AppendRotated &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream)
{
    AppendRotated arg = a;
    const AttnLaunch &l = a.attn;
    const int vec = unit_vec(a.rot.pairs, l.dim);
    const bool mx4 = kv_type == KV_TYPE_MX4;
    const uint32_t units = (uint32_t)l.dim / (2 * vec), eights = (uint32_t)l.dim / 8;
    const uint32_t all = units * (uint32_t)l.heads * ((mx4 ? 0 : 2) + (l.q ? (uint32_t)l.group : 0));
    const uint32_t threads = std::max(all, mx4 ? 2 * eights * (uint32_t)l.heads : 0);
    // Angles of 64 bits, and 17 bytes written for 64 read: eight tokens to a workgroup where there are many (7874 tokens of 32
    // heads on 8: 36.4 -> 31.1 us; of 16-bit pools 33.6 -> 35.4, e4m3 20.9 -> 24.0, all stores past the caches).
    arg.lg_split = mx4 && 2 * grid >= KVX_DEEP_GROUPS ? 0 : lg_split(threads);
    set_div(units, &arg.unit_magic, &arg.unit_shift);
    set_div(all ? all : 1, &arg.all_magic, &arg.all_shift);
    set_div(a.rot.pairs ? a.rot.pairs : 1, &arg.pair_magic, &arg.pair_shift);
    set_div(eights, &arg.eight_magic, &arg.eight_shift);
    set_div(2 * eights * (uint32_t)l.heads, &arg.each_magic, &arg.each_shift);
    void *args[] = {&arg};
    const void *fn = q_type == KV_TYPE_F16 ? append_kernel<_Float16>(kv_type, a.rot.adjacent != 0, vec)
                                           : append_kernel<__bf16>(kv_type, a.rot.adjacent != 0, vec);
    return (int)hipLaunchKernel(fn, dim3(grid << arg.lg_split, mx4 && l.q ? 2 : 1), dim3(kThreads), args, 0, stream);
}

// Appends to mx4 pools without a rotation: the same kernel with no pairs and no queries.
int launch_append_mx4(const AttnLaunch &a, int q_type, uint32_t grid, hipStream_t stream)
{
    AppendRotated arg{};
    arg.attn = a;
    arg.attn.q = nullptr;
    arg.rot.adjacent = 1;
    return launch_append_rotated(arg, q_type, KV_TYPE_MX4, grid, stream);
}

// ---- cached tokens as 16-bit rows ---------------------------------------------------

// The append's items the other way.  Eight elements to a thread; a unit's places are worked out once for all layers of
// a workgroup, and kAhead loads asked for before the first is written.  From mx4 rows, 7874 tokens of 8 heads, k and v, 41 MB:
// 10.8 us; 32 layers of 2860 tokens of 2 heads, k, 59 MB: 11.7 us (5.1 TB/s; with places worked out for each layer 17 us,
// bound by those instructions, 127 to each eight elements).
template <class T, int CACHE>
__global__ __launch_bounds__(kThreads) void read_tokens(const ReadLaunch x)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    typedef typename std::conditional<CACHE == kMx4, uint32_t, typename std::conditional<CACHE == kE4m3, uint2, T8>::type>::type Held;
    constexpr int kAhead = 4;
    const AttnLaunch &a = x.attn;
    AppendItem it;
    const Part part(a, x.lg_split, &it);
    if (part.count < 1) return;
    const uint32_t begin = part.begin, count = part.count;
    const uint32_t units = (uint32_t)a.dim / 8, kv = units * (uint32_t)a.heads, all = x.k && x.v ? 2 * kv : kv;
    const int32_t layer0 = (int32_t)blockIdx.y * x.deep, layer1 = min(layer0 + x.deep, x.layers);
    for (uint32_t i = threadIdx.x; i < count * all; i += kThreads) {
        const uint32_t u = div_by(i, x.all_magic, x.all_shift), c = i - u * all;
        const int64_t row = (int64_t)it.row + begin + u;
        if (row >= a.n_tokens) continue;
        const bool key = x.k && c < kv;
        const uint32_t hc = c < kv ? c : c - kv, h = div_by(hc, x.unit_magic, x.unit_shift), j = hc - h * units;
        const uint32_t pos = (uint32_t)it.pos + begin + u;
        const int32_t blk = it.table[div_by(pos, a.bs_magic, a.bs_shift)];
        if ((uint32_t)blk >= a.num_blocks) {
            if (c == 0) atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
            continue;
        }
        const int64_t off = place_of(a, pos, blk) + (int64_t)h * a.head_stride;
        T *to = key ? (T *)x.k + layer0 * x.k_layer + row * a.k_token + (int64_t)h * a.k_head + 8 * j
                    : (T *)x.v + layer0 * x.v_layer + row * a.v_token + (int64_t)h * a.v_head + 8 * j;
        const int64_t layer_step = key ? x.k_layer : x.v_layer;
        for (int32_t layer = layer0; layer < layer1; layer += kAhead) {
            uint8_t *const KVX_CONST *regions = (uint8_t *const KVX_CONST *)x.regions + 2 * (int64_t)layer;
            Held held[kAhead];
            uint32_t scale[kAhead];
#pragma unroll
            for (int m = 0; m < kAhead; ++m) {
                if (layer + m >= layer1) break;
                const uint8_t *from = (key ? regions[2 * m] : regions[2 * m + 1]) + off;
                held[m] = *(const Held *)(from + j * sizeof(Held));
                if constexpr (CACHE == kMx4) scale[m] = from[a.dim / 2 + j / 4];
            }
#pragma unroll
            for (int m = 0; m < kAhead; ++m) {
                if (layer + m >= layer1) break;
                T8 v;
                if constexpr (CACHE == kMx4) {
                    v = from_mx4<T>(held[m], mx4_scale(scale[m]));
                } else if constexpr (CACHE == kE4m3) {
                    const T4 lo = from_e4m3<T>(held[m].x), hi = from_e4m3<T>(held[m].y);
                    const float by = key ? a.k_scale : a.v_scale;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        v[k] = (T)((float)lo[k] * by);
                        v[4 + k] = (T)((float)hi[k] * by);
                    }
                } else {
                    v = held[m];
                }
                store_past(to, v);
                to += layer_step;
            }
        }
    }
}

int launch_read(const ReadLaunch &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream)
{
    ReadLaunch arg = a;
    const uint32_t units = (uint32_t)a.attn.dim / 8, all = units * (uint32_t)a.attn.heads * (a.k && a.v ? 2 : 1);
    arg.lg_split = lg_split(all);
    set_div(units, &arg.unit_magic, &arg.unit_shift);
    set_div(all, &arg.all_magic, &arg.all_shift);
    void *args[] = {&arg};
    const Cache cache = cache_of(kv_type);
    const void *fn = q_type == KV_TYPE_F16 ? (cache == kMx4    ? (const void *)&read_tokens<_Float16, kMx4>
                                              : cache == kE4m3 ? (const void *)&read_tokens<_Float16, kE4m3>
                                                               : (const void *)&read_tokens<_Float16, kHalves>)
                                           : (cache == kMx4    ? (const void *)&read_tokens<__bf16, kMx4>
                                              : cache == kE4m3 ? (const void *)&read_tokens<__bf16, kE4m3>
                                                               : (const void *)&read_tokens<__bf16, kHalves>);
    arg.deep = layers_of(KVX_READ_DEEP, (int64_t)grid << arg.lg_split, a.layers);
    return (int)hipLaunchKernel(fn, dim3(grid << arg.lg_split, (a.layers + arg.deep - 1) / arg.deep), dim3(kThreads), args, 0, stream);
}

// ---- cached keys to other positions ---------------------------------------------------

// An item is up to 16 tokens of one record, in some layers (y).  All of a record's tokens turn by the same angles, so a
// workgroup works them out once, with the places of its tokens, and then streams the rows through.
// 16-bit rows are bound by HBM: 32 layers of 9000 tokens of 8 heads, 1.18 GB in place, 232 us (5.1 TB/s), and 234 with four rows in
// flight and two layers to a workgroup (neighbours paired 232 and 241, a quarter of the pairs 117 and 126; e4m3 121 and 124); segments of
// 8 or 16 bytes, items of 4, 8 or 16 tokens, pages in order and accesses past the caches the same; a plain scale of as many bytes
// in place takes 198.  mx4 rows are bound by the vector pipe: 171 instructions to eight elements over a launch, 16
// of them sums of 64 bits and 40 the roundings behind them; 32 layers of 2860 tokens of 2 heads, 25 MB, 23.6 us.
// mx4: four waves a SIMD, as without the second turn of large groups; it costs 12 to 44 bytes of scratch, written and read once
// an item, outside the loops (35.5 us with the read behind it, 35.2 without that turn).
template <class T, int CACHE, bool ADJACENT, int VEC>
__global__ __launch_bounds__(kThreads, CACHE == kMx4 ? 4 : 1) void shift_keys(const ShiftLaunch x)
{
    constexpr bool MX4 = CACHE == kMx4;
    __shared__ float2 cs[MX4 ? 1 : kMaxPairs];
    __shared__ double2 cs64[MX4 ? kMaxPairs : 1];
    __shared__ int64_t place[KVX_SHIFT_TOKENS];  // of each token, or -1
    constexpr int kRows = 2, kLayers = MX4 ? 2 : 1;
    const KVX_CONST ShiftRec *recs =
        x.recs ? (const KVX_CONST ShiftRec *)x.recs
               : (const KVX_CONST ShiftRec *)((const KVX_CONST uint8_t *)__builtin_amdgcn_kernarg_segment_ptr() + offsetof(ShiftLaunch, inl));
    const uint32_t pairs = x.rot.pairs;
    const int32_t layer0 = (int32_t)blockIdx.y * x.deep;
    for (ItemWalk walk{blockIdx.x, gridDim.x, (uint32_t)x.items}; walk.there(); walk.next()) {
        const int32_t item = (int32_t)walk.at;
        int32_t r = 0, n = x.n;  // the last record that begins at or before the item
        while (n > 1) {
            const int32_t half = n >> 1;
            const bool right = recs[r + half].item <= item;
            r = right ? r + half : r;
            n = right ? n - half : half;
        }
        const int32_t first = recs[r].begin + (item - recs[r].item) * KVX_SHIFT_TOKENS;
        const int32_t tokens = min(recs[r].end - first, KVX_SHIFT_TOKENS), delta = recs[r].delta;
        const int32_t *table = recs[r].table;
        if (threadIdx.x < pairs) {
            const uint64_t t = turns_of(x.rot, delta, threadIdx.x);
            if constexpr (MX4) cs64[threadIdx.x] = turn64(t, 1.f);
            else cs[threadIdx.x] = turn32(t, 1.f);
        }
        if (threadIdx.x >= kThreads - KVX_SHIFT_TOKENS) {
            const int32_t t = threadIdx.x - (kThreads - KVX_SHIFT_TOKENS);
            int64_t at = -1;
            if (t < tokens) {
                const uint32_t pos = (uint32_t)(first + t), page = div_by(pos, x.bs_magic, x.bs_shift);
                const int32_t blk = table[page];
                if ((uint32_t)blk < x.num_blocks)
                    at = (int64_t)blk * x.block_stride + (int64_t)(pos - page * x.block_size) * x.tok_stride;
                else
                    atomicOr(x.err, KV_DEVERR_BLOCK_RANGE);
            }
            place[t] = at;
        }
        __syncthreads();
        // A thread keeps its place in a row, and with it its angles; kRows rows and kLayers layers are loaded before the first
        // is turned.  Rows follow each other as they lie: (token, head), or (head, token) in pages by heads.
        const uint32_t rows = KVX_SHIFT_TOKENS * (uint32_t)x.heads;
        const bool by_token = x.tok_stride > x.head_stride;
        const uint32_t units = MX4 ? (uint32_t)x.dim / 8 : pairs / VEC, span = MX4 ? 64 : kThreads;
        const uint32_t lane = threadIdx.x % span, slot = div_by(lane, x.unit_magic, x.unit_shift), j = lane - slot * units;
        const uint32_t each = span / units, step = each * (kThreads / span), slot0 = slot + threadIdx.x / span * each;
        const int32_t layer1 = min(layer0 + x.deep, x.layers);
        // of an mx4 row the unit's sums, else its turns
        double c[MX4 ? 8 : 1], sn[MX4 ? 8 : 1];
        float2 turn[MX4 ? 1 : VEC];
        const uint32_t e = 8 * j, p0 = partner(e, pairs), p1 = partner(e + 4, pairs);
        const int lane0 = (int)(lane - j + p0 / 8), lane1 = (int)(lane - j + p1 / 8);
        if constexpr (MX4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = e + i, pair = ADJACENT ? at / 2 : at < pairs ? at : at - pairs;
                const bool turns = at < 2 * pairs, first = ADJACENT ? i % 2 == 0 : at < pairs;
                const double2 t = cs64[turns ? pair : 0];
                c[i] = turns ? t.x : 1.;
                sn[i] = !turns ? 0. : first ? -t.y : t.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) turn[i] = cs[VEC * j + i];
        }
        for (uint32_t r0 = 0; r0 < rows; r0 += kRows * step) {
            int64_t off[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const uint32_t r = r0 + k * step + slot0, q = by_token ? div_by(r, x.head_magic, x.head_shift) : r / KVX_SHIFT_TOKENS;
                const uint32_t t = by_token ? q : r % KVX_SHIFT_TOKENS, h = by_token ? r - q * (uint32_t)x.heads : q;
                off[k] = slot < each && r < rows ? place[t] : -1;
                if (off[k] >= 0) off[k] += (int64_t)h * x.head_stride;
            }
            for (int32_t layer = layer0; layer < layer1; layer += kLayers) {
                uint8_t *const KVX_CONST *regions = (uint8_t *const KVX_CONST *)x.regions + 2 * (int64_t)layer;
                if constexpr (MX4) {
                    uint32_t w[kRows * kLayers], scale[kRows * kLayers];
#pragma unroll
                    for (int m = 0; m < kRows * kLayers; ++m) {
                        w[m] = scale[m] = 0;
                        if (off[m % kRows] < 0 || layer + m / kRows >= layer1) continue;
                        const uint8_t *row = regions[2 * (m / kRows)] + off[m % kRows];
                        w[m] = *(const uint32_t *)(row + e / 2);
                        scale[m] = row[x.dim / 2 + e / 32];
                    }
                    float y[8];
                    // A row's units lie in one wave, so a unit's partners come from the lanes that hold them.  WIDE: of
                    // scales whose values 32 bits may not hold by 2^-kDown, and back in 64.
                    auto turned = [&](uint32_t w, uint32_t scale, auto wide, auto round) __attribute__((always_inline)) {
                        double v[8], other[8];
                        auto values = [&](uint32_t w, uint32_t scale, double *to, int n) __attribute__((always_inline)) {
                            const bool far = decltype(wide)::value && scale > 254 - kDown && scale < 255;
                            const Vec<float>::x8 x = from_mx4<float>(w, mx4_scale(far ? scale - kDown : scale));
#pragma unroll
                            for (int i = 0; i < n; ++i) to[i] = far ? (double)x[i] * (1 << kDown) : (double)x[i];
                        };
                        values(w, scale, v, 8);
                        if (ADJACENT) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) other[i] = e < 2 * pairs ? v[i ^ 1] : v[i];  // times 0 of its own sign
                        } else {
                            const uint32_t w0 = __shfl(w, lane0), w1 = __shfl(w, lane1);
                            const uint32_t s0 = __shfl(scale, lane0), s1 = __shfl(scale, lane1);
                            values(p0 % 8 ? w0 >> 16 : w0, s0, other, 4);
                            values(p1 % 8 ? w1 >> 16 : w1, s1, other + 4, 4);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = round(__builtin_fma(v[i], c[i], other[i] * sn[i]));
                    };
                    auto store = [&](uint8_t *row, uint32_t s, uint32_t down) __attribute__((always_inline)) {
                        *(uint32_t *)(row + e / 2) = to_mx4(y, s);
                        if (j % 4 == 0) row[x.dim / 2 + j / 4] = (uint8_t)(s + down);
                    };
                    uint32_t left = 0;  // rows of this wave with a group that came out as NaN: none of theirs is stored yet
#pragma unroll
                    for (int m = 0; m < kRows * kLayers; ++m) {
                        if (off[m % kRows] < 0 || layer + m / kRows >= layer1) continue;
                        turned(w[m], scale[m], std::false_type{}, to_odd);
                        const uint32_t s = mx4_scale_of(y);
                        if (__builtin_expect(__any(s == 255), 0)) left |= 1u << m;
                        else store(regions[2 * (m / kRows)] + off[m % kRows], s, 0);
                    }
                    if (__builtin_expect(left != 0, 0)) {
#pragma unroll 1
                        for (int m = 0; m < kRows * kLayers; ++m) {
                            if (!(left >> m & 1)) continue;
                            int64_t at = off[0];
#pragma unroll
                            for (int k = 1; k < kRows; ++k) at = m % kRows == k ? off[k] : at;
                            uint8_t *row = regions[2 * (m / kRows)] + at;
                            const uint32_t again = *(const uint32_t *)(row + e / 2), scale = row[x.dim / 2 + e / 32];
                            turned(again, scale, std::true_type{}, to_odd);
                            uint32_t s = mx4_scale_of(y);
                            const bool far = s == 255;  // the same of the four lanes of a group
                            turned(again, scale, std::true_type{}, [&](double x) {
                                return far ? to_odd_cut(x * (1. / (1 << kDown))) : to_odd(x);
                            });
                            s = mx4_scale_of(y);
                            store(row, s, far && s < 255 ? kDown : 0);
                        }
                    }
                } else {
                    // only the units that turn
                    typedef typename std::conditional<CACHE == kE4m3, uint8_t, T>::type E;
                    typedef typename Run<E, VEC>::type EV;
                    const Unit<ADJACENT, VEC> unit(j, pairs);
                    EV va[kRows], vb[kRows];
#pragma unroll
                    for (int k = 0; k < kRows; ++k) {
                        if (off[k] < 0) continue;
                        const E *row = (const E *)(regions[0] + off[k]);
                        va[k] = *(const EV *)(row + unit.a);
                        vb[k] = *(const EV *)(row + unit.b);
                    }
#pragma unroll
                    for (int k = 0; k < kRows; ++k) {
                        if (off[k] < 0) continue;
                        E *row = (E *)(regions[0] + off[k]);
                        float v[2 * VEC];
                        if constexpr (CACHE == kE4m3) {
                            values_of_e4m3<VEC>(v, va[k]);
                            values_of_e4m3<VEC>(v + VEC, vb[k]);
                        } else {
                            values_of<T, VEC>(v, va[k]);
                            values_of<T, VEC>(v + VEC, vb[k]);
                        }
                        turn_unit<ADJACENT, VEC>(v, turn);
                        if constexpr (CACHE == kE4m3) {
                            *(EV *)(row + unit.a) = to_e4m3<VEC>(v, 1.f);
                            *(EV *)(row + unit.b) = to_e4m3<VEC>(v + VEC, 1.f);
                        } else {
                            *(EV *)(row + unit.a) = run_of<T, VEC>(v);
                            *(EV *)(row + unit.b) = run_of<T, VEC>(v + VEC);
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
}

template <bool ADJACENT, int VEC>
const void *shift_kernel(int kv_type)
{
    switch (kv_type) {
    case KV_TYPE_MX4: return (const void *)&shift_keys<__bf16, kMx4, ADJACENT, 4>;
    case KV_TYPE_E4M3: return (const void *)&shift_keys<__bf16, kE4m3, ADJACENT, VEC>;
    case KV_TYPE_F16: return (const void *)&shift_keys<_Float16, kHalves, ADJACENT, VEC>;
    default: return (const void *)&shift_keys<__bf16, kHalves, ADJACENT, VEC>;
    }
}

int launch_shift(const ShiftLaunch &a, int kv_type, hipStream_t stream)
{
    ShiftLaunch arg = a;
    const int vec = unit_vec(a.rot.pairs, a.dim);
    // mx4 rows go by all their units, others by those that turn
    const uint32_t units = kv_type == KV_TYPE_MX4 ? (uint32_t)a.dim / 8 : a.rot.pairs / vec;
    set_div(units, &arg.unit_magic, &arg.unit_shift);
    set_div((uint32_t)a.heads, &arg.head_magic, &arg.head_shift);
    void *args[] = {&arg};
    const uint32_t items = (uint32_t)std::min(a.items, KVX_SHIFT_GRID);
    const int64_t own = ((int64_t)KVX_SHIFT_TOKENS * a.heads * units + kThreads - 1) / kThreads;
    arg.deep = layers_of(kv_type == KV_TYPE_MX4 ? KVX_SHIFT_UNITS / own : 1, a.items, a.layers);
    const uint32_t layers = (uint32_t)((a.layers + arg.deep - 1) / arg.deep);
    const void *fn = a.rot.adjacent ? (vec == 8 ? shift_kernel<true, 8>(kv_type) : shift_kernel<true, 4>(kv_type))
                                    : (vec == 8 ? shift_kernel<false, 8>(kv_type) : shift_kernel<false, 4>(kv_type));
    return (int)hipLaunchKernel(fn, dim3(items, layers), dim3(kThreads), args, 0, stream);
}

}  // namespace kvx

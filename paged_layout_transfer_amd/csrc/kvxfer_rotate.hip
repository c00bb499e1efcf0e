// kvxfer_rotate.hip -- kernels that turn heads to their positions: new tokens appended with their rotation, cached
// keys moved to other positions; appends to mx4 pools, and cached tokens read back as 16-bit rows.
//
// Mathematics.  Pair (x, y) of a head at position p becomes (x c - y s, x s + y c) with c + i s = amplitude
// e^(2 pi i p f), f the turns of a pair in one position.  f is a fraction of 64 bits, so p f is an exact
// product modulo one turn: position 2^31 is as good as position 1 to 2^-33 turns.  The fraction's two top
// bits choose the quarter, and what is left of it, within an eighth of a turn of zero, goes through the power series of
// sine and cosine: to x^9 and x^10 in 32 bits (2^-29 and 2^-32 beyond them), to x^15 and x^16 in 64.
//
// Keys on their way into an mx4 pool turn in 64 bits and are then rounded to 32 bits towards the odd neighbour, from which
// the rounding to 4 bits gives the same as from all 64: so a stored value is that of the formula except where the formula
// lies within 2^-45 or so of a border between two values.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kvxfer_device.h"

namespace kvx {

static constexpr int kThreads = 256;
static constexpr int kWaves = kThreads / 64;
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
    const uint32_t t = (uint32_t)(turns >> 32), quarter = (t + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(t - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
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

// A row is worked on in units of eight elements: two runs of four, so that a unit holds whole pairs.  Unit j of
// paired halves holds elements 4j .. and their partners pairs + 4j ..; behind the pairs, and of neighbours paired, 8j .. 8j + 7.
template <bool ADJACENT>
struct Unit {
    uint32_t a, b;  // first element of either run
    bool turns;
    __device__ __forceinline__ Unit(uint32_t j, uint32_t pairs)
    {
        turns = j < pairs / 4;
        a = !ADJACENT && turns ? 4 * j : 8 * j;
        b = !ADJACENT && turns ? pairs + 4 * j : 8 * j + 4;
    }
};

// Eight values of a unit turned; cs holds the four pairs from the unit's first on.
template <bool ADJACENT>
__device__ __forceinline__ void turn_unit(float (&x)[8], const float2 *cs)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &u = x[ADJACENT ? 2 * i : i], &v = x[ADJACENT ? 2 * i + 1 : i + 4];
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

// Eight consecutive values from element e on, turned in 64 bits: `x` themselves, `other` those that
// are `pairs` away (only where halves are paired).
template <bool ADJACENT>
__device__ __forceinline__ void turn_wide(float (&x)[8], const float (&other)[8], uint32_t e, uint32_t pairs, const double2 *cs)
{
    if (ADJACENT) {
        if (e >= 2 * pairs) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double2 t = cs[e / 2 + i];
            const double u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = to_odd(__builtin_fma(u, t.x, -(v * t.y)));
            x[2 * i + 1] = to_odd(__builtin_fma(u, t.y, v * t.x));
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
            x[4 * h + i] = to_odd(low ? __builtin_fma(u, t.x, -(v * t.y)) : __builtin_fma(v, t.y, u * t.x));
        }
    }
}
// The element that pairs with e, for a run of four (pairs is a multiple of four).
__device__ __forceinline__ uint32_t partner(uint32_t e, uint32_t pairs)
{
    return e < pairs ? e + pairs : e < 2 * pairs ? e - pairs : e;
}

template <class T>
__device__ __forceinline__ void load4(float *x, const T *p)
{
    const typename Vec<T>::x4 v = *(const typename Vec<T>::x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)v[i];
}
template <class T>
__device__ __forceinline__ void store4(T *p, const float *x)
{
    typename Vec<T>::x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)x[i];
    *(typename Vec<T>::x4 *)p = v;
}

// x / scale in 32 bits (correctly rounded), clamped to +-448; NaN passes by the bounds.
__device__ __forceinline__ float e4m3_of(float x, float scale)
{
    const float y = x / scale;
    return y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
}
__device__ __forceinline__ uint32_t to_e4m3(const float *x, float scale)
{
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_of(x[0], scale), e4m3_of(x[1], scale), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_of(x[2], scale), e4m3_of(x[3], scale), p, true);
}

// ---- append with a rotation on the way --------------------------------------------

// Four workgroups to an item, two of its tokens each, and as many along y as a token's units (keys, values, then
// queries) take 256 threads: a thread owns one unit of both tokens.
template <class T, int CACHE, bool ADJACENT>
__global__ __launch_bounds__(kThreads) void append_rotated(const AppendRotated x)
{
    constexpr int kBatch = KVX_APPEND_TOKENS / KVX_APPEND_SPLIT;
    constexpr bool MX4 = CACHE == kMx4;
    __shared__ float2 cs[kBatch][kMaxPairs];
    __shared__ double2 cs64[MX4 ? kBatch : 1][MX4 ? kMaxPairs : 1];
    const AttnLaunch &a = x.attn;
    const AppendItem it = plan_record(a.append + blockIdx.x / KVX_APPEND_SPLIT);
    if ((int32_t)(blockIdx.x / KVX_APPEND_SPLIT) >= plan_record(a.head).n_append) return;
    const uint32_t begin = blockIdx.x % KVX_APPEND_SPLIT * kBatch;
    if (begin >= (uint32_t)it.count) return;
    const uint32_t count = min((uint32_t)it.count - begin, (uint32_t)kBatch), pairs = x.rot.pairs;
    const int64_t row0 = (int64_t)it.row + begin;
    const uint32_t pos0 = (uint32_t)it.pos + begin;
    const uint32_t units = (uint32_t)a.dim / 8, kv = units * (uint32_t)a.heads;
    const uint32_t all = 2 * kv + (a.q ? kv * (uint32_t)a.group : 0);

    const bool wide = MX4 && blockIdx.y * kThreads < kv;  // keys are among the units
    for (uint32_t i = threadIdx.x; i < count * pairs; i += kThreads) {
        const uint32_t u = i >= pairs, pair = i - u * pairs;
        if (row0 + u >= a.n_tokens) continue;
        const int32_t pos = x.positions ? x.positions[row0 + u] : (int32_t)(pos0 + u);
        const uint64_t t = turns_of(x.rot, pos, pair);
        cs[u][pair] = turn32(t, x.rot.amplitude);
        if constexpr (MX4) {
            if (wide) cs64[u][pair] = turn64(t, x.rot.amplitude);
        }
    }
    __syncthreads();

    for (uint32_t c = blockIdx.y * kThreads + threadIdx.x; c < all; c += gridDim.y * kThreads) {
        const bool key = c < kv, query = c >= 2 * kv;
        const uint32_t hc = key ? c : query ? c - 2 * kv : c - kv;
        const uint32_t h = div_by(hc, x.unit_magic, x.unit_shift), j = hc - h * units;
        if (query) {
            const Unit<ADJACENT> unit(j, pairs);
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                const int64_t row = row0 + u;
                if (u >= count || row >= a.n_tokens) continue;
                const T *from = (const T *)a.q + row * a.q_token + (int64_t)h * a.q_head;
                T *to = (T *)a.out + row * a.out_token + (int64_t)h * a.out_head;
                float v[8];
                load4(v, from + unit.a);
                load4(v + 4, from + unit.b);
                if (unit.turns) turn_unit<ADJACENT>(v, &cs[u][4 * j]);
                store4(to + unit.a, v);
                store4(to + unit.b, v + 4);
            }
            continue;
        }
        const T *src = key ? (const T *)a.k_new + (int64_t)h * a.k_head : (const T *)a.v_new + (int64_t)h * a.v_head;
        const int64_t src_tok = key ? a.k_token : a.v_token;
        uint8_t *base = (key ? a.k_base : a.v_base) + (int64_t)h * a.head_stride;
        const float scale = key ? a.k_scale : a.v_scale;
#pragma unroll
        for (uint32_t u = 0; u < kBatch; ++u) {
            const int64_t row = row0 + u;
            if (u >= count || row >= a.n_tokens) continue;
            const uint32_t pos = pos0 + u, page = div_by(pos, a.bs_magic, a.bs_shift);
            const int32_t blk = it.table[page];
            const T *from = src + row * src_tok;
            if ((uint32_t)blk >= a.num_blocks) {
                if (c == 0) atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
                continue;
            }
            uint8_t *to = base + (int64_t)blk * a.block_stride + (int64_t)(pos - page * a.block_size) * a.tok_stride;
            float v[8];
            if constexpr (MX4) {
                const uint32_t e = 8 * j;
                load4(v, from + e);
                load4(v + 4, from + e + 4);
                if (key) {
                    float other[8] = {};
                    if (!ADJACENT) {
                        load4(other, from + partner(e, pairs));
                        load4(other + 4, from + partner(e + 4, pairs));
                    }
                    turn_wide<ADJACENT>(v, other, e, pairs, cs64[u]);
                }
                const uint32_t s = mx4_scale_of(v);
                *(uint32_t *)(to + e / 2) = to_mx4(v, s);
                if (j % 4 == 0) to[a.dim / 2 + j / 4] = (uint8_t)s;
            } else {
                const Unit<ADJACENT> unit(j, key ? pairs : 0);
                load4(v, from + unit.a);
                load4(v + 4, from + unit.b);
                if (unit.turns) turn_unit<ADJACENT>(v, &cs[u][4 * j]);
                if (CACHE == kE4m3) {
                    *(uint32_t *)(to + unit.a) = to_e4m3(v, scale);
                    *(uint32_t *)(to + unit.b) = to_e4m3(v + 4, scale);
                } else {
                    store4((T *)to + unit.a, v);
                    store4((T *)to + unit.b, v + 4);
                }
            }
        }
    }
}

template <class T, bool ADJACENT>
const void *append_kernel(int kv_type)
{
    switch (cache_of(kv_type)) {
    case kMx4: return (const void *)&append_rotated<T, kMx4, ADJACENT>;
    case kE4m3: return (const void *)&append_rotated<T, kE4m3, ADJACENT>;
    default: return (const void *)&append_rotated<T, kHalves, ADJACENT>;
    }
}

int launch_append_rotated(const AppendRotated &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream)
{
    AppendRotated arg = a;
    set_div((uint32_t)a.attn.dim / 8, &arg.unit_magic, &arg.unit_shift);
    void *args[] = {&arg};
    const uint32_t all = (uint32_t)a.attn.dim / 8 * (uint32_t)a.attn.heads * (2 + (a.attn.q ? (uint32_t)a.attn.group : 0));
    const uint32_t slices = std::min((all + kThreads - 1) / kThreads, 65535u);
    const void *fn = q_type == KV_TYPE_F16
                         ? (a.rot.adjacent ? append_kernel<_Float16, true>(kv_type) : append_kernel<_Float16, false>(kv_type))
                         : (a.rot.adjacent ? append_kernel<__bf16, true>(kv_type) : append_kernel<__bf16, false>(kv_type));
    return (int)hipLaunchKernel(fn, dim3(grid * KVX_APPEND_SPLIT, slices), dim3(kThreads), args, 0, stream);
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

// The append's items the other way; layers along y.  A thread owns one unit of both tokens' keys, then values.
template <class T, int CACHE>
__global__ __launch_bounds__(kThreads) void read_tokens(const ReadLaunch x)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    constexpr int kBatch = KVX_APPEND_TOKENS / KVX_APPEND_SPLIT;
    const AttnLaunch &a = x.attn;
    const AppendItem it = plan_record(a.append + blockIdx.x / KVX_APPEND_SPLIT);
    if ((int32_t)(blockIdx.x / KVX_APPEND_SPLIT) >= plan_record(a.head).n_append) return;
    const uint32_t begin = blockIdx.x % KVX_APPEND_SPLIT * kBatch;
    const uint32_t end = min((uint32_t)it.count, begin + kBatch);
    const uint32_t units = (uint32_t)a.dim / 8, kv = units * (uint32_t)a.heads;
    for (int32_t layer = blockIdx.y; layer < x.layers; layer += gridDim.y) {
        for (uint32_t c = threadIdx.x; c < 2 * kv; c += kThreads) {
            const bool key = c < kv;
            if (!(key ? x.k : x.v)) continue;
            const uint32_t hc = key ? c : c - kv, h = div_by(hc, x.unit_magic, x.unit_shift), j = hc - h * units;
            const uint8_t *base = ((uint8_t *const KVX_CONST *)x.regions)[2 * layer + (key ? 0 : 1)] + (int64_t)h * a.head_stride;
            T *out = key ? (T *)x.k + layer * x.k_layer + (int64_t)h * a.k_head : (T *)x.v + layer * x.v_layer + (int64_t)h * a.v_head;
            const int64_t out_tok = key ? a.k_token : a.v_token;
            const float scale = key ? a.k_scale : a.v_scale;
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                const uint32_t t = begin + u;
                const int64_t row = (int64_t)it.row + t;
                if (t >= end || row >= a.n_tokens) continue;
                const uint32_t pos = (uint32_t)it.pos + t, page = div_by(pos, a.bs_magic, a.bs_shift);
                const int32_t blk = it.table[page];
                if ((uint32_t)blk >= a.num_blocks) {
                    atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
                    continue;
                }
                const uint8_t *from = base + (int64_t)blk * a.block_stride + (int64_t)(pos - page * a.block_size) * a.tok_stride;
                T8 v;
                if constexpr (CACHE == kMx4) {
                    v = from_mx4<T>(*(const uint32_t *)(from + 4 * j), mx4_scale(from[a.dim / 2 + j / 4]));
                } else if constexpr (CACHE == kE4m3) {
                    const uint2 w = *(const uint2 *)(from + 8 * j);
                    const T4 lo = from_e4m3<T>(w.x), hi = from_e4m3<T>(w.y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = (T)((float)lo[i] * scale);
                        v[4 + i] = (T)((float)hi[i] * scale);
                    }
                } else {
                    v = *(const T8 *)(from + 16 * j);
                }
                *(T8 *)(out + row * out_tok + 8 * j) = v;
            }
        }
    }
}

int launch_read(const ReadLaunch &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream)
{
    ReadLaunch arg = a;
    set_div((uint32_t)a.attn.dim / 8, &arg.unit_magic, &arg.unit_shift);
    void *args[] = {&arg};
    const Cache cache = cache_of(kv_type);
    const void *fn = q_type == KV_TYPE_F16 ? (cache == kMx4    ? (const void *)&read_tokens<_Float16, kMx4>
                                              : cache == kE4m3 ? (const void *)&read_tokens<_Float16, kE4m3>
                                                               : (const void *)&read_tokens<_Float16, kHalves>)
                                           : (cache == kMx4    ? (const void *)&read_tokens<__bf16, kMx4>
                                              : cache == kE4m3 ? (const void *)&read_tokens<__bf16, kE4m3>
                                                               : (const void *)&read_tokens<__bf16, kHalves>);
    const uint32_t layers = (uint32_t)std::min(a.layers, 65535);
    return (int)hipLaunchKernel(fn, dim3(grid * KVX_APPEND_SPLIT, layers), dim3(kThreads), args, 0, stream);
}

// ---- cached keys to other positions ---------------------------------------------------

// An item is up to 16 tokens of one record, in one layer (y).  All of a record's tokens turn by the same angles, so a
// workgroup works them out once, with the places of its tokens, and then streams the rows through.
template <class T, int CACHE, bool ADJACENT>
__global__ __launch_bounds__(kThreads) void shift_keys(const ShiftLaunch x)
{
    constexpr bool MX4 = CACHE == kMx4;
    __shared__ float2 cs[MX4 ? 1 : kMaxPairs];
    __shared__ double2 cs64[MX4 ? kMaxPairs : 1];
    __shared__ int64_t place[KVX_SHIFT_TOKENS];  // of each token, or -1
    const KVX_CONST ShiftRec *recs =
        x.recs ? (const KVX_CONST ShiftRec *)x.recs
               : (const KVX_CONST ShiftRec *)((const KVX_CONST uint8_t *)__builtin_amdgcn_kernarg_segment_ptr() + offsetof(ShiftLaunch, inl));
    const uint32_t pairs = x.rot.pairs, units = (uint32_t)x.dim / 8;
    for (int32_t item = blockIdx.x; item < x.items; item += gridDim.x) {
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
        for (int32_t layer = blockIdx.y; layer < x.layers; layer += gridDim.y) {
            uint8_t *base = ((uint8_t *const KVX_CONST *)x.regions)[2 * layer];
            // rows of the item in the order in which they lie: token, head, or head, token
            auto row_of = [&](uint32_t r) __attribute__((always_inline)) -> uint8_t * {
                const bool by_token = x.tok_stride > x.head_stride;
                const uint32_t t = by_token ? div_by(r, x.head_magic, x.head_shift) : r % KVX_SHIFT_TOKENS;
                const uint32_t h = by_token ? r - t * (uint32_t)x.heads : r / KVX_SHIFT_TOKENS;
                const int64_t at = place[t];
                return at < 0 ? nullptr : base + at + (int64_t)h * x.head_stride;
            };
            const uint32_t rows = KVX_SHIFT_TOKENS * (uint32_t)x.heads;
            if constexpr (MX4) {
                // A row's units lie in one wave: all of them have been read before the first is written, as the wave waits for
                // its loads as one.
                const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
                const uint32_t slot = div_by(lane, x.unit_magic, x.unit_shift), j = lane - slot * units, each = 64 / units;
                for (uint32_t r0 = wave * each; r0 < rows; r0 += kWaves * each) {
                    uint8_t *row = slot < each && r0 + slot < rows ? row_of(r0 + slot) : nullptr;
                    if (!row) continue;
                    const uint32_t e = 8 * j;
                    const Vec<float>::x8 w = from_mx4<float>(*(const uint32_t *)(row + e / 2), mx4_scale(row[x.dim / 2 + e / 32]));
                    float v[8], other[8] = {};
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = w[i];
                    if (!ADJACENT) {
                        const uint32_t p0 = partner(e, pairs), p1 = partner(e + 4, pairs);
                        const Vec<float>::x8 lo = from_mx4<float>(*(const uint16_t *)(row + p0 / 2), mx4_scale(row[x.dim / 2 + p0 / 32]));
                        const Vec<float>::x8 hi = from_mx4<float>(*(const uint16_t *)(row + p1 / 2), mx4_scale(row[x.dim / 2 + p1 / 32]));
#pragma unroll
                        for (int i = 0; i < 4; ++i) other[i] = lo[i], other[4 + i] = hi[i];
                    }
                    turn_wide<ADJACENT>(v, other, e, pairs, cs64);
                    const uint32_t s = mx4_scale_of(v);
                    *(uint32_t *)(row + e / 2) = to_mx4(v, s);
                    if (j % 4 == 0) row[x.dim / 2 + j / 4] = (uint8_t)s;
                }
            } else {
                // only the units that turn
                const uint32_t each = pairs / 4;
                for (uint32_t i = threadIdx.x; i < rows * each; i += kThreads) {
                    const uint32_t r = div_by(i, x.unit_magic, x.unit_shift), j = i - r * each;
                    uint8_t *row = row_of(r);
                    if (!row) continue;
                    const Unit<ADJACENT> unit(j, pairs);
                    float v[8];
                    if constexpr (CACHE == kE4m3) {
                        const Vec<__bf16>::x4 lo = from_e4m3<__bf16>(*(const uint32_t *)(row + unit.a));
                        const Vec<__bf16>::x4 hi = from_e4m3<__bf16>(*(const uint32_t *)(row + unit.b));
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = (float)lo[k], v[4 + k] = (float)hi[k];
                    } else {
                        load4(v, (const T *)row + unit.a);
                        load4(v + 4, (const T *)row + unit.b);
                    }
                    turn_unit<ADJACENT>(v, &cs[4 * j]);
                    if constexpr (CACHE == kE4m3) {
                        *(uint32_t *)(row + unit.a) = to_e4m3(v, 1.f);
                        *(uint32_t *)(row + unit.b) = to_e4m3(v + 4, 1.f);
                    } else {
                        store4((T *)row + unit.a, v);
                        store4((T *)row + unit.b, v + 4);
                    }
                }
            }
        }
        __syncthreads();
    }
}

template <bool ADJACENT>
const void *shift_kernel(int kv_type)
{
    switch (kv_type) {
    case KV_TYPE_MX4: return (const void *)&shift_keys<__bf16, kMx4, ADJACENT>;
    case KV_TYPE_E4M3: return (const void *)&shift_keys<__bf16, kE4m3, ADJACENT>;
    case KV_TYPE_F16: return (const void *)&shift_keys<_Float16, kHalves, ADJACENT>;
    default: return (const void *)&shift_keys<__bf16, kHalves, ADJACENT>;
    }
}

int launch_shift(const ShiftLaunch &a, int kv_type, hipStream_t stream)
{
    ShiftLaunch arg = a;
    // mx4 rows go by all their units, others by those that turn
    set_div(kv_type == KV_TYPE_MX4 ? (uint32_t)a.dim / 8 : a.rot.pairs / 4, &arg.unit_magic, &arg.unit_shift);
    set_div((uint32_t)a.heads, &arg.head_magic, &arg.head_shift);
    void *args[] = {&arg};
    const uint32_t items = (uint32_t)std::min(a.items, 1 << 20);
    const uint32_t layers = (uint32_t)std::min(a.layers, 65535);
    return (int)hipLaunchKernel(a.rot.adjacent ? shift_kernel<true>(kv_type) : shift_kernel<false>(kv_type), dim3(items, layers),
                                dim3(kThreads), args, 0, stream);
}

}  // namespace kvx

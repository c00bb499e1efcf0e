// kvxfer_attn_mx4.h -- attention of few rows over 4-bit pools: device code, instantiated for one query type by
// kvxfer_attn_mx4_f16.hip and kvxfer_attn_mx4_bf16.hip.  kvxfer_attn.h has the mathematics and the many-rows kernel.
#pragma once
#include "kvxfer_attn.h"

namespace kvx {

// The scale bytes from which on some elements are infinite or NaN as T: 4 * 2^126 and 4 * 2^14 are past the types' ranges.
template <class T>
constexpr uint32_t mx4_not_finite() { return __is_same(T, __bf16) ? 127 + 126 : 127 + 14; }

// x / d for whole numbers with x d < 2^16: a product and a shift instead of thirty instructions.  The factor is
// 65536 / d rounded down and one more; the reciprocal is exact for powers of two, and no other quotient lies within its
// error of a whole number.
struct SmallDiv {
    uint32_t factor;
    __device__ __forceinline__ explicit SmallDiv(uint32_t d) : factor((uint32_t)(65536.f * __builtin_amdgcn_rcpf((float)d)) + 1) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return x * factor >> 16; }
};

// Few rows over a 4-bit pool: the (token, query head) rows of several cache heads, at most 16 in all, are the columns of one
// product.  A wave works on 32 keys of all of its heads at a time: K_h Q^T is computed for every head h against all
// columns, and each column keeps the result of its own head, so one softmax serves all heads; and V_h^T P^T with zeros for
// the weights of other heads' columns, so one set of results does.
//
// A row of 4-bit values is no multiple of a cache line, and rows of one token's heads share lines.  So a wave reads the rows of
// all its heads, token by token, in 16-byte pieces, lane after lane, to shared memory, and from there in the
// order in which the product takes them.  (With a head to each wave the same lines were asked for by several waves, and
// those requests waited for each other: 3.9 TB/s with the loads alone.)
//
// The weights are rounded to the queries' type for the second product, as in the other kernels (weights of two such parts would
// take its products and its registers twice); scores, maxima, sums and results are held in 32 bits.  Against 64 bits bf16 results
// are off by 2.3e-3, 1.7e-3 with weights of 32 bits.
//
// 32 tokens on 1 K to 64 K each, 8 heads of 128, 494 MB: 106 us (4.6 TB/s); beside HBM it
// is the widening and the way through shared memory and back that a wave waits for.  One token on 128 K, 143 MB: 37 us
// and the join's 5.4.  Steps of 64 keys, two heads to a pack with three waves a SIMD, and steps held in two sets of registers
// were slower (114 to 152 us of the first); products of 4-bit operands as they are (the scaled matrix instructions) align their sums
// to 2^-15 of the largest product, which is no sum of 32 bits.
template <class T, int DP, int SHAPED>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void attend_few_mx4(const AttnLaunch a)
{
    typedef typename Vec<T>::x8 T8;
    typedef typename Vec<T>::x4 T4;
    constexpr int kStep = 32;
    constexpr int kS = DP / 32;
    constexpr int kVals = cache_values<kMx4, DP>(), kLoads = DP / (4 * kVals), kBytes = kVals / 2;
    // Wide values: rows 32 bytes beyond a multiple of all banks, and in rows 8 to 15 of 16 the 16-byte pieces exchanged in pairs:
    // the writes, 16 rows at a time, and the transposing reads, 32 bytes of four rows, meet all banks.
    constexpr int kRow = DP + 16;
    constexpr int kPieces = mx4_pieces(DP);  // of a lane for one step's keys, or values
    constexpr int kTile = kStep * kRow * 2, kRaw = mx4_raw(DP);
    constexpr int kSlice = kTile + kRaw;
    static_assert(kSlice >= 16 * DP * 4, "the end's results");
    __shared__ __attribute__((aligned(16))) char shared[4 * kSlice];
    __shared__ int64_t places[4][kStep];  // of a step's keys
    __shared__ float join_m[4][16], join_l[4][16];

    const AttnItem it = plan_record(a.items + blockIdx.x);
    const int32_t n_few = plan_record(a.head).n_few;
    asm volatile("" : : "s"(it.kv_len), "s"(n_few));
    if ((int32_t)blockIdx.x >= n_few) return;
    const Piece s = piece_of(a, it);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    char *const raw = shared + wave * kSlice;
    T *const tile = (T *)(raw + kRaw);

    // column n is row n mod s.rows of the pack's head n / s.rows; columns past the last repeat it
    const int heads = it.across, n_rows = heads * s.rows;
    const SmallDiv by_rows((uint32_t)s.rows), by_heads((uint32_t)heads);
    const int own = (int)by_rows((uint32_t)min(n, n_rows - 1));  // the lane's head
    const uint32_t R = (uint32_t)(min(n, n_rows - 1) - own * s.rows);
    const int32_t tok = (int32_t)div_by(R, a.group_magic, a.group_shift);
    const int32_t pos = s.first + tok, q_head = (s.head + own) * a.group + (int32_t)R - tok * a.group;
    const RowMask mask = row_mask(a, s, pos);
    float slope = 0.f;
    if (SHAPED && a.slopes) slope = a.slopes[q_head] * 1.4426950408889634f;

    const int32_t i1 = s.tile1 * 2;
    int32_t i = s.tile0 * 2 + wave;
    auto start = [&](int32_t i) { return s.walk.start(i >> 1) + (i & 1) * kStep; };
    auto mine = [&](int32_t i) { return seen_key(s, start(i) + (lane & 31)); };  // both halves of the wave the same
    auto place = [&](int32_t i, int32_t blk) __attribute__((always_inline)) {
        const int64_t at = key_offset(a, s, mine(i), blk);
        if (lane < 32) places[wave][lane] = at;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };

    // A row is read in 16-byte pieces, lane after lane in the order in which a token's rows (or, in head-major pages, a head's
    // rows) lie in memory; the last piece ends with the row.  In shared memory a row takes whole pieces, 16-byte aligned,
    // with its scales where the last piece puts them; the rows of a head lie together, and each head's one row further on:
    // the writes, in whichever order, and the reads of 16 rows meet all banks.
    const uint32_t per_row = (a.row + 15) / 16, pieces = kStep * (uint32_t)heads * per_row;
    const uint32_t key_step = per_row * 16, head_step = (kStep + 1) * key_step;
    const uint32_t end = key_step - 16, values = (uint32_t)a.dim / 2;
    const uint32_t scales = values >= end ? values + key_step - a.row : values;
    // piece k of the lane: where its key's place is, where from there on it lies, and where it goes
    const bool by_token = a.tok_stride > a.head_stride;
    const SmallDiv by_per_row(per_row);
    uint32_t key_of[kPieces], from[kPieces], to[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const uint32_t e = min((uint32_t)(64 * k + lane), pieces - 1);
        const uint32_t r = by_per_row(e), p = e - r * per_row, row_j = by_heads(r);
        const uint32_t h = by_token ? r - row_j * (uint32_t)heads : r / kStep, j = by_token ? row_j : r % kStep;
        key_of[k] = j;
        from[k] = h * a.head_stride + min(16 * p, a.row - 16);
        to[k] = h * head_step + j * key_step + 16 * p;
    }
    typedef u32x4 Piece16 __attribute__((aligned(4)));
    // A step's keys, then its values, then the next step's keys; the first step's values beside its keys, as nothing
    // else takes their registers yet.
    u32x4 flight[kPieces], first_values[kPieces];
    // pieces in groups, so that few heads do not read as many as fit
    auto each_piece = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 3; ++k) f(k);
        if (pieces > 3 * 64) {
#pragma unroll
            for (int k = 3; k < 5; ++k) f(k);
            if (pieces > 5 * 64) {
#pragma unroll
                for (int k = 5; k < kPieces; ++k) f(k);
            }
        }
    };
    auto load = [&](u32x4(&flight)[kPieces], const uint8_t *base) __attribute__((always_inline)) {
        each_piece([&](int k) __attribute__((always_inline)) {
            flight[k] = *(const KVX_GLOBAL Piece16 *)((const KVX_GLOBAL uint8_t *)base + places[wave][key_of[k]] + from[k]);
        });
    };
    auto put_raw = [&](const u32x4(&flight)[kPieces]) __attribute__((always_inline)) {
        each_piece([&](int k) __attribute__((always_inline)) { *(u32x4 *)(raw + to[k]) = flight[k]; });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    // Quarter p of load c of a row: its bytes and its scale.  Past the row's width the first group again, with a scale
    // that is no NaN: the queries are zeros there, and such columns are not stored.
    typedef typename std::conditional<kBytes == 16, u32x4, u32x2>::type Aligned;
    struct Quarter {
        Aligned r;
        uint32_t e;
    };
    auto quarter = [&](const char *row, int c, int p) __attribute__((always_inline)) {
        const bool live = (4 * c + p) * kVals < a.dim;
        const int at = live ? 4 * c + p : 0;
        Quarter x;
        x.r = *(const Aligned *)(row + at * kBytes);
        x.e = *(const uint8_t *)(row + scales + at * kVals / KVX_MX4_GROUP);
        x.e = live ? x.e : 0;
        return x;
    };
    auto widen = [&](const Quarter &x, int u) __attribute__((always_inline)) { return from_mx4<T>(x.r[u], mx4_scale(x.e)); };

    const T *const at = tile + (4 * g + (n >> 2)) * kRow + ((n & 3) * 4 ^ (g & 2) * 4);
    auto value = [&](int d) __attribute__((always_inline)) {
        const T4 lo = read_column<T>(at + 16 * d), hi = read_column<T>(at + 16 * kRow + 16 * d);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    // One head's values of the step in `raw`, wide and row-major; zeros in the place of infinities and NaN if `finite`.
    // Whether there are any of those.
    const char *const row_of_lane = raw + n * key_step;
    auto put_values = [&](int h, auto finite) __attribute__((always_inline)) {
        uint32_t most = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < kLoads; ++c) {
                const Quarter x = quarter(row_of_lane + 16 * t * key_step + h * head_step, c, g);
                most = max(most, x.e);
#pragma unroll
                for (int u = 0; u < kVals / 8; ++u) {
                    const T8 v = widen(x, u);
                    *(T8 *)(tile + (16 * t + n) * kRow + (4 * c + g) * kVals + (8 * u ^ (n & 8))) =
                        decltype(finite)::value ? only_finite<T>(v) : v;
                }
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        return __any(most >= mx4_not_finite<T>()) != 0;
    };

    int32_t blk = 0;
    if (i < i1) {
        blk = block_of(a, s, mine(i));
        const int32_t next = i + 4 < i1 ? block_of(a, s, mine(i + 4)) : 0;
        place(i, blk);
        load(flight, a.k_base);
        load(first_values, a.v_base);
        blk = next;
    }
    T8 q[kS];
    int64_t row = (int64_t)s.q_begin + tok;
    if (row >= a.n_tokens) row = a.n_tokens - 1;  // replays of a call with shorter arrays: not stored
    const T *qr = (const T *)a.q + row * a.q_token + (int64_t)q_head * a.q_head;
#pragma unroll
    for (int c = 0; c < kS; ++c) q[c] = load_q<T>(a, qr, (4 * (8 * c / kVals) + g) * kVals + 8 * c % kVals);

    f32x4 o[DP / 16];
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.f;
    bool any_odd = false;
    const float sc = SHAPED ? 1.f : a.scale_log2;
    const float slack = 8.f / sc;  // a maximum that grows by less than 2^8 is not worth a rescaling

    auto work = [&](auto is_first) __attribute__((always_inline)) {
        constexpr bool FIRST = decltype(is_first)::value;
        const int32_t j0 = start(i);
        const bool more = i + 4 < i1;
        auto next_keys = [&]() __attribute__((always_inline)) {
            if (!more) return;
            place(i + 4, blk);
            load(flight, a.k_base);
            if (i + 8 < i1) blk = block_of(a, s, mine(i + 8));
        };
        put_raw(flight);
        if (FIRST) next_keys();
        else load(flight, a.v_base);
        // S^T: keys 16 t + 4 g + r against row n, of the row's own head
        f32x4 x[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll 1
        for (int h = 0; h < heads; ++h) {
            const char *const key_row = raw + n * key_step + h * head_step;
            f32x4 y[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
            for (int c = 0; c < kLoads; ++c)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Quarter k = quarter(key_row + 16 * t * key_step, c, g);
#pragma unroll
                    for (int u = 0; u < kVals / 8; ++u) y[t] = mfma16(widen(k, u), q[c * (kVals / 8) + u], y[t]);
                }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[t][r] = own == h ? y[t][r] : x[t][r];
        }
        const bool masked = !all_see(a, s, j0, kStep);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            auto key = [&](int r) { return j0 + 16 * t + 4 * g + r; };
            if (SHAPED) shape<SHAPED, 4>(a, x[t], slope, pos, key);
            if (masked) hide<4>(x[t], mask, key);
        }
        float mx = x[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) mx = fmaxf(mx, x[t][r]);
        mx = max_of_quarters(max_of_halves(mx));
        if (__any(mx > m + slack || (m == -INFINITY && mx > m))) {
            const float up = fmaxf(m, mx);
            const float by = up == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - up) * sc);
            m = up;
            l *= by;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) o[d] *= keep(by);
        }
        const float mm = m == -INFINITY ? 0.f : m * sc - weight_shift<T>();
        float sum[2] = {0.f, 0.f};
        T8 w;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r], sc, -mm));
                sum[t] += e;
                w[4 * t + r] = (T)e;
            }
        l += sum[0] + sum[1];
        if (FIRST) {
            put_raw(first_values);
        } else {
            put_raw(flight);
            next_keys();
        }
#pragma unroll 1
        for (int h = 0; h < heads; ++h) {
            // A zero weight would turn an infinity or NaN among the values into NaN, in rows that do not see it and in
            // other heads' rows: they are left out, and added after the loop.
            if (__builtin_expect(put_values(h, std::false_type{}), 0)) any_odd = put_values(h, std::true_type{});
            const T8 wh = own == h ? w : T8{};
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) o[d] = mfma16(value(d), wh, o[d]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    };
    if (i < i1) {
        work(std::true_type{});
        for (i += 4; i < i1; i += 4) work(std::false_type{});
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (__builtin_expect(any_odd, 0)) {
        // what each row sees of infinities and NaN: where a product of ones, for seen keys and such values, is not zero
        for (i = s.tile0 * 2 + wave; i < i1; i += 4) {
            place(i, block_of(a, s, mine(i)));
            load(flight, a.v_base);
            put_raw(flight);
            const int32_t j0 = start(i);
#pragma unroll 1
            for (int h = 0; h < heads; ++h) {
                put_values(h, std::false_type{});
                T8 seen;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    seen[k] = (T)(own == h && mask.sees(j0 + 16 * (k >> 2) + 4 * g + (k & 3)) ? 1.f : 0.f);
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    const T8 v = value(d);
#pragma unroll
                    for (int kind = 0; kind < 3; ++kind) {
                        const f32x4 c = mfma16(ones_at<T>(v, kind), seen, f32x4{0, 0, 0, 0});
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[d][r] += c[r] != 0.f ? special(kind) : 0.f;
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        }
    }
    auto row_of = [&](int r) __attribute__((always_inline)) {
        const int h = (int)by_rows((uint32_t)r);
        const uint32_t x = (uint32_t)(r - h * s.rows);
        const int32_t t = (int32_t)div_by(x, a.group_magic, a.group_shift);
        return RowPlace{t, (s.head + h) * a.group + (int32_t)x - t * a.group};
    };
    finish_few<T, DP, kSlice>(a, s, false, n_rows, row_of, shared, join_m, join_l, m,
                              m == -INFINITY ? m : m * sc - weight_shift<T>(), l, o);
}

}  // namespace kvx

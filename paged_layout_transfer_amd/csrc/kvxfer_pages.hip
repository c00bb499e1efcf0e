// kvxfer_pages.hip -- kernels that change pages in place in the pool: page copies within
// the pool, block tables rewritten after moves, and new tokens appended to their pages.
#include <hip/hip_runtime.h>

#include "kvxfer_ops.h"

namespace kvx {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#define KVX_GLOBAL __attribute__((address_space(1)))
#define KVX_CONST __attribute__((address_space(4)))

static constexpr int kThreads = 256;
static constexpr int kWaves = kThreads / 64;

// A call's records: in the kernel's own arguments (at `off` of the one explicit argument)
// or in the pool's arena; either way not written while the kernel runs.
template <class Rec>
__device__ __forceinline__ const KVX_CONST Rec *records(const Rec *dev, size_t off)
{
    if (dev) return (const KVX_CONST Rec *)dev;
    return (const KVX_CONST Rec *)((const KVX_CONST uint8_t *)__builtin_amdgcn_kernarg_segment_ptr() + off);
}

// Pages copied within the pool: one wave copies one 4 KiB part of a (region, record) page, 4 vectors of
// 16 bytes a lane in flight, nontemporal (each byte is touched once).  Bound by HBM, and there
// by isolated page writes into one region after the other: regions outermost, and a contiguous
// stretch of the parts to each chiplet (workgroup b runs on chiplet b mod 8).  1024 pages of 64 regions x
// 32 KiB (4.3 GB moved): 756 us, 5.7 TB/s; records outermost with 8 KiB parts 800 us, 16 KiB
// parts 835 us, regions outermost without the chiplets' stretches 781 us.
__global__ __launch_bounds__(kThreads) void copy_pages(const CopyLaunch a)
{
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const KVX_CONST kv_page_copy *copies = records(a.copies, offsetof(CopyLaunch, inl));
    const int64_t step = (int64_t)gridDim.x * kWaves;
    const uint32_t stretch = gridDim.x / 8;
    const uint32_t block = blockIdx.x < stretch * 8 ? blockIdx.x % 8 * stretch + blockIdx.x / 8 : blockIdx.x;
    for (int64_t item = (int64_t)block * kWaves + wave; item < a.items; item += step) {
        const int64_t tile = item / a.parts;
        const uint32_t part = (uint32_t)(item - tile * a.parts);
        const uint32_t region = (uint32_t)(tile / a.n_copies);
        const int64_t c = tile - (int64_t)region * a.n_copies;
        const int32_t src = copies[c].src, dst = copies[c].dst;
        const uint32_t n_tok = (uint32_t)copies[c].n_tokens;
        uint8_t *base = ((uint8_t *const KVX_CONST *)a.regions)[region];
        const uint8_t *from = base + (int64_t)src * a.block_stride;
        uint8_t *to = base + (int64_t)dst * a.block_stride;
        const uint32_t begin = part * KVX_COPY_PART, total = n_tok * a.tok;
        if (begin >= total) continue;
        const uint32_t end = min(total, begin + (uint32_t)KVX_COPY_PART);
        if (a.hm_heads == 0 || n_tok == a.block_size) {
            // one stretch, whole 16-byte vectors
            const KVX_GLOBAL u32x4 *s = (const KVX_GLOBAL u32x4 *)(from + begin);
            KVX_GLOBAL u32x4 *d = (KVX_GLOBAL u32x4 *)(to + begin);
            const uint32_t n = (end - begin) / 16;
            if (n == KVX_COPY_PART / 16) {
                u32x4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __builtin_nontemporal_load(s + lane + 64 * i);
#pragma unroll
                for (int i = 0; i < 4; ++i) __builtin_nontemporal_store(v[i], d + lane + 64 * i);
            } else {
                for (uint32_t i = lane; i < n; i += 64)
                    __builtin_nontemporal_store(__builtin_nontemporal_load(s + i), d + i);
            }
            continue;
        }
        // the first tokens of a head-major page: a stretch of n_tok rows in each head
        const uint32_t seg = n_tok * a.hm_row, pitch = a.block_size * a.hm_row;
        if (a.word == 16) {
            for (uint32_t b = begin + lane * 16; b < end; b += 64 * 16) {
                const uint32_t off = b / seg * pitch + b % seg;
                *(KVX_GLOBAL u32x4 *)(to + off) = *(const KVX_GLOBAL u32x4 *)(from + off);
            }
        } else {
            for (uint32_t b = begin + lane * 4; b < end; b += 64 * 4) {
                const uint32_t off = b / seg * pitch + b % seg;
                *(KVX_GLOBAL uint32_t *)(to + off) = *(const KVX_GLOBAL uint32_t *)(from + off);
            }
        }
    }
}

int launch_copy_pages(const CopyLaunch &a, hipStream_t stream)
{
    const int64_t need = (a.items + kWaves - 1) / kWaves;
    const uint32_t grid = (uint32_t)(need < (1 << 20) ? need : (1 << 20));
    CopyLaunch arg = a;
    void *args[] = {&arg};
    return (int)hipLaunchKernel((const void *)&copy_pages, dim3(grid), dim3(kThreads), args, 0, stream);
}

// Table entries after moves: a binary search of each entry among the moves' sources, which sit
// in shared memory when they fit.  A million entries, 1024 moves: 10 us.
template <bool LDS>
__global__ __launch_bounds__(kThreads) void remap(const RemapLaunch a)
{
    __shared__ Move near[LDS ? KVX_REMAP_LDS : 1];
    const KVX_CONST Move *moves = records(a.moves, offsetof(RemapLaunch, inl));
    if (LDS) {
        for (int32_t i = threadIdx.x; i < a.n; i += kThreads) {
            near[i].src = moves[i].src;
            near[i].dst = moves[i].dst;
        }
        __syncthreads();
    }
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.count; i += step) {
        const int32_t id = a.in[i];
        int32_t lo = 0, n = a.n;  // first move whose source is not below id
        while (n > 0) {
            const int32_t half = n >> 1;
            const int32_t at = LDS ? near[lo + half].src : moves[lo + half].src;
            lo = at < id ? lo + half + 1 : lo;
            n = at < id ? n - half - 1 : half;
        }
        int32_t to = id;
        if (lo < a.n && (LDS ? near[lo].src : moves[lo].src) == id) to = LDS ? near[lo].dst : moves[lo].dst;
        a.out[i] = to;
    }
}

int launch_remap(const RemapLaunch &a, hipStream_t stream)
{
    const int64_t need = (a.count + kThreads - 1) / kThreads;
    const uint32_t grid = (uint32_t)(need < 2048 ? need : 2048);
    RemapLaunch arg = a;
    void *args[] = {&arg};
    const void *fn = a.n <= KVX_REMAP_LDS ? (const void *)&remap<true> : (const void *)&remap<false>;
    return (int)hipLaunchKernel(fn, dim3(grid), dim3(kThreads), args, 0, stream);
}

// ---- append ------------------------------------------------------------------

// Two values to e4m3: x / scale in 32 bits (correctly rounded), clamped to +-448, rounded to
// nearest even by the conversion.  v_med3 would turn NaN into a bound, so NaN passes by.
__device__ __forceinline__ float e4m3_of(float x, float scale)
{
    const float y = x / scale;
    return y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
}

// Four workgroups to an item, two of its tokens each.  A thread owns eight values of a token's row
// (of its keys, then its values): block ids and rows of both tokens first, then the stores.  Bound by
// the latency of that chain: 3.5 us for 64 tokens of a decode step, 12.1 us a pass with its launch for 7874 tokens in
// chunks into a 16-bit pool (64 MB), 11.5 for 4000 tokens of 8 x 256 bf16 (66 MB).  An 8-bit pool
// moves 48 MB of the same chunks in 13.5 to 15.0 us: the correctly rounded quotient of each element costs 4 us of
// them (with a product in its place 11.2).  One workgroup to an item, four tokens at a time, took 15.0 where this
// took 13.5, eight at a time 15.8.
template <class T, bool E4M3>
__global__ __launch_bounds__(kThreads) void append_tokens(const AttnLaunch a)
{
    typedef T T8 __attribute__((ext_vector_type(8)));
    constexpr int kBatch = KVX_APPEND_TOKENS / KVX_APPEND_SPLIT;
    const AppendItem it = a.append[blockIdx.x / KVX_APPEND_SPLIT];
    if ((int32_t)(blockIdx.x / KVX_APPEND_SPLIT) >= a.head->n_append) return;
    const uint32_t begin = blockIdx.x % KVX_APPEND_SPLIT * kBatch;
    const uint32_t end = min((uint32_t)it.count, begin + kBatch);
    const uint32_t chunks = (uint32_t)a.dim / 8;  // of one head
    const uint32_t per_tok = chunks * (uint32_t)a.heads;
    const uint32_t lanes = min(2 * per_tok, (uint32_t)kThreads), at_once = kThreads / lanes;
    const uint32_t t0 = threadIdx.x / lanes;
    if (t0 >= at_once) return;
    for (uint32_t c = threadIdx.x - t0 * lanes; c < 2 * per_tok; c += lanes) {
        const bool val = c >= per_tok;
        const uint32_t hc = val ? c - per_tok : c, h = hc / chunks, e = hc - h * chunks;
        const T *src = (val ? (const T *)a.v_new + (int64_t)h * a.v_head : (const T *)a.k_new + (int64_t)h * a.k_head) + e * 8;
        const int64_t src_tok = val ? a.v_token : a.k_token;
        uint8_t *dst = (val ? a.v_base : a.k_base) + (int64_t)h * a.head_stride + e * (E4M3 ? 8 : 16);
        const float scale = val ? a.v_scale : a.k_scale;
        for (uint32_t t = begin + t0; t < end; t += kBatch * at_once) {
            int32_t blk[kBatch];
            T8 x[kBatch];
            bool ok[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t tt = t + u * at_once;
                ok[u] = tt < end && (int64_t)it.row + tt < a.n_tokens;
                blk[u] = 0;
                if (ok[u]) {
                    blk[u] = it.table[div_by((uint32_t)it.pos + tt, a.bs_magic, a.bs_shift)];
                    x[u] = *(const T8 *)(src + ((int64_t)it.row + tt) * src_tok);
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (!ok[u]) continue;
                const uint32_t pos = (uint32_t)it.pos + t + u * at_once;
                const uint32_t slot = pos - div_by(pos, a.bs_magic, a.bs_shift) * a.block_size;
                if ((uint32_t)blk[u] >= a.num_blocks) {
                    if (c == 0) atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
                    continue;
                }
                uint8_t *to = dst + (int64_t)blk[u] * a.block_stride + (int64_t)slot * a.tok_stride;
                if (!E4M3) {
                    *(T8 *)to = x[u];
                    continue;
                }
                uint32_t w[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    int p = 0;
                    p = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_of((float)x[u][4 * k], scale),
                                                        e4m3_of((float)x[u][4 * k + 1], scale), p, false);
                    p = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_of((float)x[u][4 * k + 2], scale),
                                                        e4m3_of((float)x[u][4 * k + 3], scale), p, true);
                    w[k] = (uint32_t)p;
                }
                *(uint2 *)to = make_uint2(w[0], w[1]);
            }
        }
    }
}

int launch_append(const AttnLaunch &a, int q_type, int kv_type, uint32_t grid, hipStream_t stream)
{
    if (kv_type == KV_TYPE_MX4) return launch_append_mx4(a, q_type, grid, stream);
    AttnLaunch arg = a;
    void *args[] = {&arg};
    const bool e4m3 = kv_type == KV_TYPE_E4M3;
    const void *fn = q_type == KV_TYPE_F16
                         ? (e4m3 ? (const void *)&append_tokens<_Float16, true> : (const void *)&append_tokens<_Float16, false>)
                         : (e4m3 ? (const void *)&append_tokens<__bf16, true> : (const void *)&append_tokens<__bf16, false>);
    return (int)hipLaunchKernel(fn, dim3(grid * KVX_APPEND_SPLIT), dim3(kThreads), args, 0, stream);
}

}  // namespace kvx

/*
 * kvxfer.h -- paged KV-cache gather/scatter for AMD Instinct MI355X (gfx950).
 *
 * The library moves a request's KV pages between a paged pool (per-layer K/V
 * regions addressed through a block table) and large contiguous transfer
 * chunks, in either direction, with one kernel launch per call:
 *
 *   gather  (offload): pool pages  -> chunks   (Strata guide, "Implementation"
 *                      lifecycle figure, step 6: background eviction of cold
 *                      pages to host memory with a one-block kernel)
 *   scatter (reload) : chunks      -> pool pages (same figure, step 3, and
 *                      "Step 1: High-Performance GPU-Assisted I/O CUDA Kernel")
 *
 * Chunks may sit in HBM or in pinned host memory that the kernel reads and
 * writes directly with ordinary loads and stores, instead of one DMA per page
 * (Strata guide, "The Mechanics of GPU-Assisted I/O").  The layout change
 * between the pool (layer-first) and the chunk (layer-first or page-first) is
 * done by address arithmetic during the copy (Strata guide, "Two-Dimensional
 * Memory Layout Decoupling").  Host work per call is proportional to the number
 * of spans, not to pages x layers (Tutti summary, Q2 "Design 1": CPU work drops
 * from O(layer x blocks) to O(layer)).
 *
 * ---------------------------------------------------------------------------
 * Data model
 * ---------------------------------------------------------------------------
 * Pool.  For layer l < num_layers and kv < num_kv (2 = K and V, 1 = a single
 * latent) the caller provides one device region, bases[l*num_kv + kv].  Block
 * b of that region starts at bases[l*num_kv+kv] + b*block_stride and holds
 * block_size tokens, token-major ([block_size][H][D]) or, with page_layout
 * KV_PAGE_HEAD_MAJOR, head-major ([H][block_size][D]); a token is num_heads x
 * head_dim elements of elem_bytes bytes: tok = num_heads*head_dim*elem_bytes.  One
 * block id names the same page in every (layer, kv) region.  K and V are
 * separate objects per layer, as in the Tutti summary's Figure 4 (2L objects
 * per block).  block_stride >= block_size*tok; block_stride == block_size*tok
 * gives a vLLM-style [num_blocks][block_size][H][D] region, block_stride ==
 * num_kv*block_size*tok with bases offset by kv*block_size*tok gives a per-layer
 * [num_blocks][num_kv][block_size][H][D] pool.
 * Placement (measured on MI355X, not part of the contract): scattered page writes
 * into a pool whose regions all lie in one 64 GiB window of one plain allocation run
 * at about 68 % of HBM peak, and at about 80 % when the regions span two windows
 * (gathers lose 1-3 points there).  What decides is the physical memory behind the
 * addresses, which the library cannot see: the caller chooses where regions live,
 * and a pool larger than 64 GiB spans windows by its size alone.
 *
 * Span.  (block_table, t_begin, t_end, first_chunk): tokens [t_begin, t_end)
 * of one request, whose token t lives at slot t % block_size of block
 * block_table[t / block_size].  t_begin must be a multiple of block_size
 * (prefix matches end on page boundaries: Strata guide, "The Conflict Between
 * PagedAttention and Transfer Efficiency"); t_end is arbitrary, so the last
 * page may be partial.
 *
 * Chunks.  A call moves layers [layer_begin, layer_end).  Each span splits into
 * chunks of chunk_layers layers x chunk_tokens tokens, layer-chunk major:
 *     c = first_chunk + lc*n_tc + tc,  lc = (l - layer_begin) / chunk_layers,
 *     tc = (t - t_begin) / chunk_tokens,  n_tc = ceil((t_end - t_begin) / chunk_tokens)
 * and chunk c occupies slot (c mod n_slots), at base + (c mod n_slots)*slot_bytes.
 * With li = (l - layer_begin) % chunk_layers, a chunk is laid out as
 *     KV_LAYER_FIRST: [chunk_layers][num_kv][T_c][H][D], T_c = tokens in the
 *                     chunk (the span's last chunk may be short, and is dense)
 *     KV_PAGE_FIRST : [P_c][chunk_layers][num_kv][block_size][H][D], P_c = pages
 *                     in the chunk; a partial last page leaves pad bytes that
 *                     are neither written (gather) nor read (scatter).
 * The page-first order is the Strata guide's host-side [P, L, H, D] tensor
 * ("Two-Dimensional Memory Layout Decoupling", item 2); layer-first matches its
 * HBM-side [L, P, H, D] tensor (item 1).  Chunks are token-major in both; a
 * head-major pool is transposed to token-major on the way out and back on the way in.
 *
 * Nothing outside the referenced pool tokens and the chunk bytes is written.
 *
 * ---------------------------------------------------------------------------
 * Conventions
 * ---------------------------------------------------------------------------
 * Every function returns KV_OK (0) or a negative KV_ERR_* code; no exception
 * crosses the ABI.  A call that returns an error has launched nothing and
 * changed no state.
 * Pointers named "device" must be valid on the device current when the call
 * is made (HBM, or mapped pinned host memory from kv_ring_create / hipHostMalloc).
 * All device and chunk pointers, block_stride, slot_bytes and tok must be
 * multiples of 16 bytes (16-byte vector loads and stores).
 * Transfers are asynchronous on the given stream (0 = the null stream): the
 * caller keeps every buffer alive and unmodified until the stream has passed
 * the call.  Handles are not thread-safe.
 * The caller's buffers must hold what the call declares: each region
 * (num_blocks - 1) * block_stride + block_size * tok bytes, the staging area
 * n_slots * slot_bytes, each device block table table_len entries.  Where the
 * HIP runtime knows the allocation holding such a pointer (hipMalloc'd device
 * memory, hipHostMalloc'd or registered host memory, virtual-memory mappings),
 * a transfer whose declared extent runs past the end of that allocation and
 * any allocations adjoining it without a gap is refused with KV_ERR_RANGE
 * before anything is enqueued (an access past mapped memory would fault the
 * GPU); memory the runtime does not know is taken on trust.  A sub-allocator's
 * block (e.g. a torch tensor) is checked against the runtime allocation it lies
 * in, not against its own size.
 */
#ifndef KVXFER_H
#define KVXFER_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KV_API __attribute__((visibility("default")))

/* ---- error codes ------------------------------------------------------- */
#define KV_OK 0
#define KV_ERR_ARG (-1)    /* null pointer, bad shape, empty or inverted range */
#define KV_ERR_ALIGN (-2)  /* pointer, stride, slot size or token size not a multiple of 16 */
#define KV_ERR_RANGE (-3)  /* span past its block table, slot too small, block id out of range, buffer past its allocation */
#define KV_ERR_OOM (-4)    /* allocator exhausted, or a host/device allocation failed */
#define KV_ERR_RING (-5)   /* two chunks of one call share a staging slot */
#define KV_ERR_HIP (-6)    /* a HIP runtime call failed (no device, launch failure, ...) */
#define KV_ERR_DEVICE (-7) /* kv_pool_get_error: the device reported a bad block id */
#define KV_ERR_DUP (-8)    /* KV_FLAG_VALIDATE: a scatter writes one pool page twice */
#define KV_ERR_SCRATCH (-9) /* kv_transfer_chunks_noalloc: more regions than its static scratch holds */
#define KV_ERR_CAPTURE (-10) /* the stream is capturing a graph and this call cannot be captured */

/* ---- chunk layouts, in-page layouts, directions, flags ----------------- */
#define KV_LAYER_FIRST 0
#define KV_PAGE_FIRST 1

/* kv_pool_desc.page_layout: how a pool block orders its tokens and heads */
#define KV_PAGE_TOKEN_MAJOR 0 /* [block_size][H][D] (vLLM-style NHD) */
#define KV_PAGE_HEAD_MAJOR 1  /* [H][block_size][D] (HND); chunks stay token-major */

#define KV_GATHER 0  /* pool -> chunks (offload) */
#define KV_SCATTER 1 /* chunks -> pool (reload)  */

/* kv_chunk_spec.flags */
#define KV_FLAG_VALIDATE 0x1 /* copy the block tables to the host (synchronously) and check
                                ids in range and, for scatter, one writer per pool page */
#define KV_FLAG_DMA_STRIDED 0x2 /* read by the _dma entry points only: where the regions are
                                   evenly spaced, one strided copy per (chunk, page) covers
                                   the page's chunk_layers*num_kv tiles */
#define KV_FLAG_CACHED 0x4 /* kernel entry points: plain cached loads and stores instead of the
                              default nontemporal ones (same bytes, same result).  The default
                              keeps a transfer from evicting the working set of kernels that
                              run beside it (Strata guide, "Non-Intrusive Resource Sizing");
                              this flag is for callers that touch the moved bytes right after */
#define KV_FLAG_PAGE_RUNS 0x8 /* kernel scatters: a hint that the call's pages lie mostly in
                                 runs of adjacent block ids (as kv_pool_alloc_blocks hands them
                                 out on an unfragmented pool), so token-major tiles of 20 KiB
                                 to under 64 KiB are copied whole, one wave each, instead of in
                                 4 KiB parts by several.  Same bytes, same result; measured on
                                 MI355X with 32 KiB tiles: runs of adjacent blocks scatter at
                                 74-77 % of HBM peak whole against 71-72 % in parts, shuffled
                                 blocks at 68-69 % whole against 70-72 % in parts.  No passage:
                                 a performance hint of this library. */

/* device error bits reported through kv_pool_get_error */
#define KV_DEVERR_BLOCK_RANGE 0x1 /* a block table held an id outside [0, num_blocks); that
                                     (layer, kv, page) tile was skipped */

/* element types of the append and attention operators */
#define KV_TYPE_F16 0  /* IEEE half */
#define KV_TYPE_BF16 1 /* bfloat16 */
#define KV_TYPE_E4M3 2 /* 8-bit float, OCP e4m3fn (pools only) */
#define KV_TYPE_MX4 3  /* 4-bit floats with a shared power of two for each 32 (pools only): see
                          "Rows of KV_TYPE_MX4" below */

/* kv_attn_desc.flags */
#define KV_ATTN_FULL 0x1 /* every query sees every cached token (no causal mask) */

/* kv_ring_create flags */
#define KV_RING_COHERENT 0x0     /* hipHostMalloc coherent mapped memory (default) */
#define KV_RING_NONCOHERENT 0x1  /* hipHostMallocNonCoherent: the GPU may cache it */

/* Limits of one call. */
#define KV_MAX_SPANS 4096
#define KV_MAX_PAGE_COPIES 65536 /* records of one kv_copy_pages or kv_remap_tables call */
#define KV_MAX_SEQS 4096         /* sequences of one attention plan */
#define KV_MAX_ATTN_DIM 256      /* head_dim of the attention operators */
#define KV_MAX_SHIFTS 4096       /* records of one kv_rotate_cached call */

/* kv_rotation_desc.pairing: which two elements of a head turn together, of n pairs */
#define KV_ROT_HALVES 0   /* i and i + n */
#define KV_ROT_ADJACENT 1 /* 2i and 2i + 1 */

typedef struct kv_rotation kv_rotation; /* opaque, owned by the library */
typedef struct kv_pool kv_pool; /* opaque, owned by the library */
typedef struct kv_ring kv_ring; /* opaque, owned by the library */
typedef struct kv_attn_plan kv_attn_plan; /* opaque, owned by the library */

typedef struct {
    int32_t num_layers;   /* L >= 1 */
    int32_t num_kv;       /* 1 or 2 */
    int32_t num_heads;    /* H >= 1 */
    int32_t head_dim;     /* D >= 1 */
    int32_t elem_bytes;   /* 1, 2, 4 or 8 (the payload is moved as opaque bytes) */
    int32_t block_size;   /* tokens per page, >= 1 */
    int32_t page_layout;  /* KV_PAGE_TOKEN_MAJOR or KV_PAGE_HEAD_MAJOR; a head-major row,
                             head_dim*elem_bytes bytes, must be a multiple of 16 bytes, or a
                             multiple of 4 with tok <= 8192 (such rows are transposed
                             through LDS); other rows: KV_ERR_ALIGN, too large a token for
                             4-byte rows: KV_ERR_ARG */
    int64_t num_blocks;   /* blocks per (layer, kv) region, 1 .. 2^31-1 */
    int64_t block_stride; /* bytes between consecutive blocks of one region */
    void *const *bases;   /* host array of num_layers*num_kv device pointers; the
                             library copies it, the regions stay caller-owned */
} kv_pool_desc;

typedef struct {
    const int32_t *block_table; /* device array (host array for kv_validate_targets) */
    int64_t table_len;          /* entries in block_table; >= ceil(t_end / block_size), < 2^31 */
    int64_t t_begin;            /* first token, a multiple of block_size, >= 0 */
    int64_t t_end;              /* one past the last token, >= t_begin (an empty span moves nothing) */
    int64_t first_chunk;        /* chunk index of the span's first chunk, >= 0 */
} kv_span;

typedef struct {
    int32_t layout;        /* KV_LAYER_FIRST or KV_PAGE_FIRST */
    int32_t chunk_layers;  /* CL, divides layer_end - layer_begin */
    int64_t chunk_tokens;  /* CT, a multiple of block_size */
    int32_t layer_begin;   /* first layer moved */
    int32_t layer_end;     /* one past the last layer moved (<= num_layers) */
    void *base;            /* device-visible staging: HBM or mapped pinned host memory */
    int64_t slot_bytes;    /* bytes per staging slot, >= the largest chunk of the call */
    int64_t n_slots;       /* slots at base; chunk c uses slot c mod n_slots */
    int32_t max_workgroups;/* 0 = library default grid: the whole chip when base is device
                              memory, 16 workgroups of 256 threads when it is host memory
                              (a host-link-bound copy needs few: Strata guide,
                              "Non-Intrusive Resource Sizing"); the kind of memory is
                              looked up with hipPointerGetAttributes and remembered for
                              the last base the pool saw.  > 0 caps the grid.  A reload
                              and an offload over the host link at the same time do
                              best with smaller grids than either alone: 6 workgroups
                              for the scatter and 2 for the gather measured 95 GB/s
                              combined on MI355X (98 % of the link's two-way rate),
                              the default 16 each 71 GB/s */
    int32_t flags;         /* KV_FLAG_* */
} kv_chunk_spec;

/* Sizes of one call, as kv_check_transfer reports them. */
typedef struct {
    int64_t tiles;          /* (layer, kv, page) tiles the kernel copies */
    int64_t chunks;         /* chunks the call touches */
    int64_t payload_bytes;  /* bytes copied (each read once and written once) */
    int64_t max_chunk_bytes;/* largest chunk of the call */
} kv_transfer_info;

/* One page copied to another of the same pool, or moved (kv_pool_plan_compact). */
typedef struct {
    int32_t src, dst;  /* block ids */
    int32_t n_tokens;  /* tokens [0, n_tokens) are copied, 1 .. block_size */
} kv_page_copy;

/* One sequence of an attention plan.  Its cache holds kv_len tokens, the q_len newest of
 * them being the call's new tokens: row q_begin + i of the new tokens' arrays is the token
 * at position kv_len - q_len + i. */
typedef struct {
    const int32_t *block_table; /* device array */
    int64_t table_len;          /* entries in block_table; >= ceil(kv_len / block_size), < 2^31 */
    int64_t kv_len;             /* cached tokens, new ones included, 0 .. 2^31 - 4097 */
    int64_t q_begin;            /* first row of its new tokens, >= 0 */
    int32_t q_len;              /* new tokens, >= 0 */
    int32_t prefix_len;         /* cached tokens [0, prefix_len) that every query sees, >= 0 */
} kv_seq;

typedef struct {
    int32_t num_q_heads; /* query heads, a multiple of the pool's num_heads: query head h reads
                            the cache's head h / (num_q_heads / num_heads) */
    int32_t q_type;      /* of q, out and the appended k and v: KV_TYPE_F16 or KV_TYPE_BF16 */
    int32_t kv_type;     /* of the pool: q_type, KV_TYPE_E4M3 or KV_TYPE_MX4 */
    int32_t window;      /* > 0: a query sees its own token and the window - 1 before it; 0: all
                            before it.  KV_ERR_ARG together with KV_ATTN_FULL */
    int32_t flags;       /* KV_ATTN_* */
    int32_t max_seqs;    /* sequences of one kv_attn_plan_set, 1 .. KV_MAX_SEQS */
    int64_t max_tokens;  /* new tokens of one kv_attn_plan_set, 1 .. 2^24 */
} kv_attn_desc;

/* Strides are in elements and, like the pointers, multiples of 16 bytes; head_dim elements
 * of one head lie together. */
typedef struct {
    const void *k, *v;                      /* device, [n_tokens][num_heads][head_dim], q_type */
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t n_tokens;                       /* rows the arrays hold */
    float k_scale, v_scale;                 /* KV_TYPE_E4M3 pools: a pool element stands for its
                                               value times this (finite, > 0); else unused */
} kv_append_args;

typedef struct {
    const void *q;                          /* device, [n_tokens][num_q_heads][head_dim], q_type */
    void *out;                              /* device, the same shape and type */
    float *lse;                             /* device, [n_tokens][num_q_heads] packed, or NULL */
    const float *alibi_slopes;              /* device, [num_q_heads], or NULL */
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t n_tokens;                       /* rows the arrays hold */
    float scale;                            /* of the scores; finite */
    float softcap;                          /* > 0: scores become softcap * tanh(score / softcap);
                                               0: off */
    float k_scale, v_scale;                 /* as in kv_append_args */
} kv_attend_args;

typedef struct {
    int32_t pairs;          /* n, a multiple of 4 up to KV_MAX_ATTN_DIM / 2: the first 2n elements of a head turn */
    int32_t pairing;        /* KV_ROT_HALVES or KV_ROT_ADJACENT */
    float amplitude;        /* of the turned elements, finite, > 0; 1 for a plain rotation.  The formula takes these 32 bits */
    const double *inv_freq; /* host array of n angles a position turns pair i by, in radians, 0 .. 2^20 */
} kv_rotation_desc;

/* Strides as in kv_attend_args. */
typedef struct {
    const void *q;                          /* device, [n_tokens][num_q_heads][head_dim], q_type; NULL: k only */
    void *q_out;                            /* device, the same shape and type; may be q with its strides */
    const int32_t *positions;               /* device, [n_tokens]; NULL: each token's place in the cache */
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
} kv_rotate_args;

/* Cached tokens [t_begin, t_end) of one sequence, whose keys turn by `delta` positions. */
typedef struct {
    const int32_t *block_table; /* device array */
    int64_t table_len;          /* entries in block_table; >= ceil(t_end / block_size), < 2^31 */
    int64_t t_begin, t_end;     /* 0 <= t_begin <= t_end <= 2^31 - 4097; empty: nothing */
    int32_t delta;              /* positions, either sign */
} kv_shift;

/* Strides as in kv_attend_args; a layer stride is only used with more than one layer. */
typedef struct {
    void *k, *v;                            /* device, [layers][n_tokens][num_heads][head_dim], q_type; NULL: not read */
    int64_t k_layer_stride, k_token_stride, k_head_stride;
    int64_t v_layer_stride, v_token_stride, v_head_stride;
    int64_t n_tokens;                       /* rows the arrays hold */
    float k_scale, v_scale;                 /* as in kv_append_args */
} kv_read_args;

/* ---- pool ------------------------------------------------------------------ */

/* Validates desc and creates a pool handle with a host bitmap of free blocks (one
 * bit per block, all free).  Device-side state (a region
 * table, an error word, a 4 MiB span-record arena with its pinned mirror and 256
 * events) is created on the first transfer, on the device current then; later
 * transfers must run with the same device current.  Errors: KV_ERR_ARG,
 * KV_ERR_ALIGN (a base, block_stride or tok not 16-byte aligned, or a head-major
 * row neither 16- nor 4-byte aligned), KV_ERR_OOM. */
KV_API int kv_pool_create(const kv_pool_desc *desc, kv_pool **out);

/* Frees the handle and its device state, after waiting for the transfers it
 * queued that are still in flight (their fence events; other device work is not
 * waited for, unless the pool has copied pages or rewritten tables: then the device is idle
 * first, and where that cannot be waited for because a stream captures, which the attempt ends, the
 * call returns KV_ERR_HIP and the pool stays as it was; nor are replays of calls captured into
 * graphs: those must have finished, and such graphs must not run again).  The caller's regions are
 * untouched.  NULL is accepted.
 * No passage: library infrastructure (the handle's lifetime). */
KV_API int kv_pool_destroy(kv_pool *pool);

/* Block allocator (a host bitmap of free blocks, preallocated at create time, no
 * allocation on the call path: Tutti summary, "Key implementation details", item 1).
 * alloc: writes the n lowest free ids to out_ids in ascending order (so a request's
 * pages lie as close together as the pool's fragmentation allows, which makes
 * reloading them faster), or fails with KV_ERR_OOM and allocates nothing.
 * free: ids must be currently allocated and distinct, else KV_ERR_RANGE and
 * nothing is freed.  A block that kv_pool_share_blocks or kv_pool_fork_blocks gave more
 * references loses one; it is free when its last one goes. */
KV_API int kv_pool_alloc_blocks(kv_pool *pool, int32_t n, int32_t *out_ids);
KV_API int kv_pool_free_blocks(kv_pool *pool, int32_t n, const int32_t *ids);
/* Free blocks left in the allocator (same source as the two calls above). */
KV_API int kv_pool_free_count(const kv_pool *pool, int64_t *out);

/* References, for requests that share pages.  share: one more reference on each of the n
 * ids, which must be allocated (else KV_ERR_RANGE, nothing changed); an id may be listed
 * twice and then gains two.  block_refs: the references of one block, 0 if it is free.
 * Host only, like the allocator.  No passage: the pages share prefixes but print no
 * bookkeeping for it. */
KV_API int kv_pool_share_blocks(kv_pool *pool, int32_t n, const int32_t *ids);
KV_API int kv_pool_block_refs(const kv_pool *pool, int32_t id, int32_t *out);

/* Forks a request of n_tokens tokens in blocks ids[0 .. ceil(n_tokens / block_size)):
 * writes the child's block ids to child_ids (as many).  Whole pages are shared (one more
 * reference each); a partly filled last page gets a fresh block, and *tail is set to the
 * copy that fills it (tail->n_tokens is 0 when there is none), for the caller to pass to
 * kv_copy_pages, the tails of many forks in one call.  ids must be allocated and distinct
 * (KV_ERR_RANGE, KV_ERR_DUP); KV_ERR_OOM when no block is free.  On an error nothing has changed.
 * Host only. */
KV_API int kv_pool_fork_blocks(kv_pool *pool, int64_t n_tokens, const int32_t *ids, int32_t *child_ids,
                               kv_page_copy *tail);

/* Plans a compaction: pairs the highest allocated blocks with the lowest free ones, while
 * the first lie above the second, up to max_moves (0 .. KV_MAX_PAGE_COPIES) of them.  Writes
 * the moves, whole pages, src ascending, and their number.  The allocator then holds the dst
 * blocks with the src blocks' references, and each src block still, with one reference of
 * its own: the caller copies the pages (kv_copy_pages), rewrites the block tables on the
 * device (kv_remap_tables) and in its own memory, and, once nothing reads the old pages, frees the
 * src ids.  Until then no later plan moves a src block again, so a pool may be compacted a few
 * pages at a time: plan, copy and rewrite, then the next plan.  Host only. */
KV_API int kv_pool_plan_compact(kv_pool *pool, int32_t max_moves, kv_page_copy *moves, int32_t *n_moves);

/* ---- calls -------------------------------------------------------------------- */

/* Host-only dry run: validates a prospective call exactly as kv_gather_chunks /
 * kv_scatter_chunks do (shapes, alignment, span ranges, slot sizes, one slot per
 * chunk) and reports its sizes.  Makes no HIP call, so the allocation-extent
 * checks (Conventions above) are left to the transfer itself; info may be NULL.
 * No passage of its own: it is the host-side part of the transfer calls below
 * (their call decomposition, Tutti summary, Q2 "Design 1"), run without a launch. */
KV_API int kv_check_transfer(const kv_pool_desc *desc, const kv_span *spans, int32_t n_spans,
                      const kv_chunk_spec *spec, kv_transfer_info *info);

/* Bytes of a chunk holding `tokens` tokens (1 <= tokens <= chunk_tokens) in the
 * spec's layout (the two chunk layouts of the Data model above: Strata guide,
 * "Two-Dimensional Memory Layout Decoupling", items 1 and 2), so a caller can size
 * staging slots. */
KV_API int kv_chunk_bytes(const kv_pool_desc *desc, const kv_chunk_spec *spec, int64_t tokens,
                   int64_t *out);

/* Host-side check of the block tables of a call, given host copies of them
 * (host_tables[i] holds spans[i].table_len ids): every id of every referenced
 * page lies in [0, num_blocks) (else KV_ERR_RANGE) and, for KV_SCATTER, no pool
 * page receives two writers (else KV_ERR_DUP).  Gather may read a page twice.
 * No passage: the pages are silent on duplicate targets; this checks the
 * precondition the library states for scatter (one writer per pool page). */
KV_API int kv_validate_targets(const kv_pool_desc *desc, const kv_span *spans, int32_t n_spans,
                        const int32_t *const *host_tables, int32_t direction);

/* Gather (offload): for every span, layer in [layer_begin, layer_end), kv and
 * token, copies the pool token into its chunk position.  One kernel launch on
 * `stream`, preceded by one small stream-ordered descriptor upload.  spans is a
 * host array of n_spans (1 .. KV_MAX_SPANS) entries; each block_table is a
 * device pointer.  n_spans == 0, or spans that are all empty, is a no-op.  Loads
 * and stores are nontemporal.  Returns after enqueueing.
 * Under HIP graph capture (the same holds for kv_scatter_chunks): a call is captured as
 * its one kernel, every replay repeating the call, when its span records ride in the
 * kernel arguments (at most 16 non-empty spans), the pool has made a call outside the
 * capture before (the first call allocates the pool's device state), KV_FLAG_VALIDATE
 * is not set (its table check copies to the host) and the pool's timing is off.  Any
 * other call is refused with KV_ERR_CAPTURE and enqueues nothing (more records go
 * through the pool's arena, which is recycled under events the host waits on).  A
 * replay reads the pool's region table and writes its error word (kv_pool_get_error),
 * so the pool must outlive the graph, and kv_pool_destroy must not be called while a
 * replay may still run (it waits only for calls made outside a graph). */
KV_API int kv_gather_chunks(kv_pool *pool, const kv_span *spans, int32_t n_spans,
                     const kv_chunk_spec *spec, hipStream_t stream);

/* Scatter (reload): the inverse move, chunk positions -> pool tokens.  The
 * spans of one call must not write one pool page twice (checked only with
 * KV_FLAG_VALIDATE); then every written byte has exactly one writer. */
KV_API int kv_scatter_chunks(kv_pool *pool, const kv_span *spans, int32_t n_spans,
                      const kv_chunk_spec *spec, hipStream_t stream);

/* For callers that cannot allocate (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): kv_gather_chunks (direction KV_GATHER) or
 * kv_scatter_chunks (KV_SCATTER) with the same data model, validation, kernels and
 * results, but no allocation of any kind on any call, the first included.  The call's
 * region table and span records go to a static device array of 264.25 KiB that each
 * device the library runs on holds until the process ends (one stream-ordered
 * host-to-device copy per call from a host image the pool made at kv_pool_create; the
 * copy has taken the image's bytes when the call returns), instead of the pool's
 * arena.  Limits beyond the other entry points': num_layers*num_kv <= 1024 (else
 * KV_ERR_SCRATCH), and KV_FLAG_VALIDATE is refused (KV_ERR_ARG: its table check
 * copies to the host).  Every call on one device shares that device's array, which
 * keeps the last call's contents: calls that overlap on one device (different
 * streams, or other threads, with no ordering between them) race and must not be
 * made; calls on one stream are ordered and safe.  A block id out of range is
 * skipped, as in the other entry points, and its KV_DEVERR_* bit OR-ed into
 * *err_word, a caller-owned device int32 (4-byte aligned) that the caller clears
 * and reads; err_word may be NULL to ignore such ids.  kv_pool_get_error does not
 * see these calls.  Returns after enqueueing.
 * Under HIP graph capture: a call with at most 16 non-empty spans carries its span
 * records in the kernel arguments, and is captured as the copy of the pool's region
 * table (which the graph reads from the pool's host image each time it runs, so the
 * pool must outlive the graph) followed by the kernel; every replay repeats the
 * call.  A call with more non-empty spans is refused with KV_ERR_CAPTURE while
 * `stream` is capturing: the graph would read its records from the host image when
 * it runs, after later calls have rewritten them.  Replays share the device's static
 * array like any other call: a replay must not overlap another call on the device. */
KV_API int kv_transfer_chunks_noalloc(kv_pool *pool, int32_t direction, const kv_span *spans,
                                      int32_t n_spans, const kv_chunk_spec *spec, int32_t *err_word,
                                      hipStream_t stream);

/* The conventional engine, for comparison: the same transfer done by the copy
 * engine as one hipMemcpyAsync per (layer, kv, page) tile, issued from the host on
 * `stream` -- the per-page DMA loop whose submission overhead the Strata guide
 * measures ("The Conflict Between PagedAttention and Transfer Efficiency",
 * paged-fragmentation figure, and the framework comparison table).  Same data
 * model, validation and results as kv_gather_chunks / kv_scatter_chunks, except
 * that each spans[i].block_table is a HOST array (the host issues the copies), and
 * every block id of the call is checked on the host before any copy is issued
 * (KV_ERR_RANGE; for scatter also KV_ERR_DUP).  Host work is O(tiles).  The tables
 * are read during the call only.  A head-major pool takes one hipMemcpy2DAsync per
 * (tile, head) instead.  With KV_FLAG_DMA_STRIDED and token-major pages whose
 * regions are evenly spaced (bases[i+1] - bases[i] the same positive value for all
 * i), the tiles of one page in one chunk -- one per (layer, kv) of the chunk --
 * go as one hipMemcpy2DAsync of chunk_layers*num_kv rows (the "where strides allow"
 * variant of the conventional engine); otherwise the flag changes nothing. */
KV_API int kv_gather_chunks_dma(kv_pool *pool, const kv_span *spans, int32_t n_spans,
                                const kv_chunk_spec *spec, hipStream_t stream);
KV_API int kv_scatter_chunks_dma(kv_pool *pool, const kv_span *spans, int32_t n_spans,
                                 const kv_chunk_spec *spec, hipStream_t stream);

/* ---- pages within a pool --------------------------------------------------------- */

/* Copies pages within the pool: for every record, layer in [layer_begin, layer_end) and kv,
 * tokens [0, n_tokens) of block src to the same tokens of block dst; the rest of dst is left
 * as it was.  One kernel launch on `stream`.  copies is a host array of n (0 ..
 * KV_MAX_PAGE_COPIES) records.  Ids lie in [0, num_blocks) (KV_ERR_RANGE); no dst is named
 * twice or is the src of a record (KV_ERR_DUP): every byte has one writer and no byte that
 * is read is written.  Allocated or not is not looked at.  n == 0 is a no-op.  Returns after enqueueing.  Under
 * graph capture a call of at most 256 records is captured as its kernel once the pool has made a
 * call outside the capture; any other is refused with KV_ERR_CAPTURE.
 * No passage: the page maintenance next to the pages' transfers. */
KV_API int kv_copy_pages(kv_pool *pool, const kv_page_copy *copies, int32_t n, int32_t layer_begin,
                         int32_t layer_end, hipStream_t stream);

/* Rewrites `count` entries of block tables (device int32 arrays, 4-byte aligned) after
 * moves: out[i] = dst of the move whose src is in[i], or in[i] where there is none (entries out of range
 * included).  in == out rewrites in place; arrays that overlap otherwise are refused
 * (KV_ERR_ARG).  moves is a host array of n records as in kv_copy_pages (n_tokens is not
 * read), ids in range (KV_ERR_RANGE), no src twice (KV_ERR_DUP).  Asynchronous, one launch;
 * captured like kv_copy_pages. */
KV_API int kv_remap_tables(kv_pool *pool, const kv_page_copy *moves, int32_t n, const int32_t *in,
                           int32_t *out, int64_t count, hipStream_t stream);

/* ---- new tokens: append and attention -------------------------------------------- */

/* Rows of KV_TYPE_MX4.  A pool of 4-bit values is described to kv_pool_create by its bytes: elem_bytes 1 and
 * head_dim the bytes R of one head's row, a multiple of 4.  The row holds G = R / 17 (rounded down) groups of 32
 * elements, so the operators' head_dim is 32 G (at most KV_MAX_ATTN_DIM): 16 G bytes of elements, then
 * G bytes of scales, then what is left of R, which nothing reads or writes.  Element 2b is the low
 * half of byte b, 2b + 1 the high half: a sign bit over three bits of {0, 0.5, 1, 1.5, 2, 3, 4, 6} (OCP e2m1).  Scale
 * byte e stands for 2^(e - 127), 255 for NaN (OCP e8m0); an element is its value times its group's scale.  Transfers,
 * page copies, forks and compaction move such pools like any other.
 * What is written: the scale is the smallest power of two 2^s, -126 <= s <= 127, with |x| <= 7 * 2^s for all
 * 32 values (s is 127 where a turned key passes 7 * 2^127), and each element is x / 2^s rounded to nearest even and saturated
 * at 6: values over 6 are off by no more than others of their size, and the group keeps the finer scale.  A group that holds an infinity or NaN becomes NaN
 * whole (scale byte 255, elements 0).  What is read is rounded to q_type (exact but for halves below 2^-24, and past the type's range).
 * kv_mx4_row_bytes: the smallest R for head_dim elements with which a token of num_heads rows is the multiple
 * of 16 bytes that a pool needs.  head_dim a multiple of 32 up to KV_MAX_ATTN_DIM (KV_ERR_ARG).
 * Host only.  No passage. */
KV_API int kv_mx4_row_bytes(int32_t head_dim, int32_t num_heads, int32_t *out);

/* A plan holds, on the device, one step's sequences, the split of their attention over the
 * chip, and the workspace of partial results (up to 200 MiB); it is set once a step and used
 * by every layer.  The pool has num_kv 2, elem_bytes 1 for KV_TYPE_E4M3 and KV_TYPE_MX4 and 2 else, head_dim <=
 * KV_MAX_ATTN_DIM, and num_q_heads * max_tokens < 2^31 (else KV_ERR_ARG), and head_dim *
 * elem_bytes a multiple of 16, of 4 for KV_TYPE_MX4 (KV_ERR_ALIGN); a KV_TYPE_MX4 token has at most 2^27 elements,
 * keys and values together (KV_ERR_ARG).  create allocates all device memory the plan
 * will use, on the current device, which is then the pool's, and waits for the device; it must
 * not be made while a stream captures (KV_ERR_HIP).  destroy waits for the device to be idle
 * first (KV_ERR_HIP, and the plan stays, while a stream captures, as for kv_pool_destroy); NULL is accepted.  A plan is destroyed before its pool, and graphs that hold its calls do not
 * run again.  No passage for this section: the attention that reads the cache the pages move. */
KV_API int kv_attn_plan_create(kv_pool *pool, const kv_attn_desc *desc, kv_attn_plan **out);
KV_API int kv_attn_plan_destroy(kv_attn_plan *plan);

/* Sets the plan to n (0 .. max_seqs) sequences: host work proportional to the pieces of work,
 * and one stream-ordered upload.  Errors: KV_ERR_ARG (negative lengths, null table of a
 * sequence with kv_len > 0, more sequences or new tokens than the plan holds, another device
 * current), KV_ERR_ALIGN (a table not 4-byte aligned), KV_ERR_RANGE (a table too short or past
 * its allocation, kv_len or a row over its limit), KV_ERR_DUP (two sequences own one row),
 * KV_ERR_CAPTURE (the stream is capturing); the plan then stays as it was (after KV_ERR_HIP it has to
 * be set again).  The tables stay the caller's and are read when append and attend run.
 * The calls that use one plan -- set, append, attend, replays of graphs they were captured
 * into -- share its memory: two that could overlap (different streams with no ordering
 * between them) must not be made. */
KV_API int kv_attn_plan_set(kv_attn_plan *plan, const kv_seq *seqs, int32_t n, hipStream_t stream);

/* Writes the new tokens' k and v rows into their pages of one layer: the token at position p
 * goes to slot p % block_size of block block_table[p / block_size].  An e4m3 pool gets
 * x / scale (in 32 bits), rounded to nearest even and saturated at +-448; NaN stays NaN; a KV_TYPE_MX4 pool gets rows as
 * above.  Nothing else is written, and rows of no sequence are not read.  Two sequences must not write one pool token.  A block id
 * out of range is skipped and reported (kv_pool_get_error).  Errors: KV_ERR_ARG (layer, null or
 * negative arguments, scales, a sequence with q_len > kv_len, another device current),
 * KV_ERR_ALIGN, KV_ERR_RANGE (n_tokens below a row the plan names, an array past its allocation).
 * Append and attend make their launches and nothing else, so both can be captured into a
 * graph; a replay works on what the last kv_attn_plan_set before it set, within the arrays
 * the captured call named (rows past its n_tokens are neither read nor written; with a
 * sequence of q_len > kv_len set, nothing is appended). */
KV_API int kv_append_tokens(kv_attn_plan *plan, int32_t layer, const kv_append_args *args, hipStream_t stream);

/* Attention of the new tokens over the cache of one layer.  With p = kv_len - q_len + i the
 * position of a query, it sees cached token j < kv_len where KV_ATTN_FULL is set, or
 * j < prefix_len, or j <= p and (window == 0 or j > p - window).  Scores are
 * s = scale * k_scale * <q, k_j>, then softcap * tanh(s / softcap) if softcap > 0, then
 * s - slope * |p - j| if slopes are given; out = v_scale * sum_j softmax(s)_j v_j,
 * lse = log sum_j exp(s_j) (natural).  A query that sees nothing gets out = 0 and
 * lse = -infinity.  Cached tokens that a query does not see do not reach its result, whatever
 * they hold (infinities and NaN too); pages that no query sees are not read and their table entries
 * may be anything.  Sums, maxima and both products' sums are held in 32 bits; the weights are rounded to
 * q_type for the second product (half weights below 2^-32 of the largest to zero; infinite
 * and NaN values that a query sees reach it all the same).  Rows of no sequence are left as they were.  The same call
 * gives the same bits: no atomics take part, and split sums are joined in a fixed order.  The
 * new tokens must be in the cache already (kv_append_tokens on the same stream).  out may be q
 * itself, with its strides; it overlaps nothing else that the call reads.  A block id out of range is
 * reported (kv_pool_get_error) and block 0 read in its place: the result of the queries that
 * see it is undefined.  A cap adds at most 2^-21 softcap to a score's error up to softcap 64, and beyond a few
 * units in the last place of the score.  Errors: as kv_append_tokens; also KV_ERR_ARG for scale or softcap that
 * are not finite, softcap < 0, scale * k_scale, softcap or scale * k_scale / softcap over the 32-bit range, or
 * rows of out that overlap.
 * Captured, a call holds the kernels for any sequences within the plan's limits. */
KV_API int kv_attend(kv_attn_plan *plan, int32_t layer, const kv_attend_args *args, hipStream_t stream);

/* Position rotation.  A token at position p turns pair i of a head by p * inv_freq[i]: of the pair's elements
 * (x, y) it makes amplitude * (x cos - y sin, x sin + y cos); elements from 2 * pairs on stay as they are.  Angles
 * are taken as fractions of a turn in 64 bits, p times inv_freq[i] / 2 pi rounded to 2^-64, so that they are
 * good to |p| 2^-64 turns at any position (and to 2^-22 of themselves where sums are held in 32 bits).  Products, sums and
 * quotients are held in 32 bits, each rounded to them, in 64 for keys on their way into a KV_TYPE_MX4 pool; the result is then
 * rounded to what is written.
 * create copies the frequencies to the current device, where the rotation is then used, and waits for the
 * copy (KV_ERR_HIP while a stream captures); KV_ERR_ARG for pairs not 1 .. KV_MAX_ATTN_DIM / 2, an unknown
 * pairing, or frequencies or an amplitude out of range, KV_ERR_ALIGN for pairs no multiple of 4.  destroy waits for the device
 * like kv_attn_plan_destroy; NULL is accepted.  No passage. */
KV_API int kv_rotation_create(const kv_rotation_desc *desc, kv_rotation **out);
KV_API int kv_rotation_destroy(kv_rotation *rotation);

/* kv_append_tokens with the rotation applied on the way, one launch: the new tokens' k rows are rotated, each to its
 * position, and written to their pages with the v rows; their q rows are rotated into q_out.  Rotated
 * values are rounded to the pool's type (e4m3: the quotient by k_scale, in 32 bits) or q_type.  positions[row] is a
 * token's position, of either sign; NULL takes its place in the cache.  Rows of no sequence are neither read
 * nor written.  q_out may be q with its strides; otherwise it overlaps nothing that the call reads.
 * Errors and capture as kv_append_tokens; also KV_ERR_ARG for a rotation wider than head_dim or of another
 * device, rows of q_out that overlap, and a token's q, k and v of more than 2^27 elements.  A bad block id skips the
 * token's k and v, not its q. */
KV_API int kv_append_rotated(kv_attn_plan *plan, int32_t layer, const kv_rotation *rotation, const kv_rotate_args *rotate,
                             const kv_append_args *args, hipStream_t stream);

/* The inverse of append: the new tokens' places in the cache of layers [layer_begin, layer_end), read as
 * q_type rows: 16-bit pools' rows as they are, k_scale or v_scale times an e4m3 element in 32 bits, KV_TYPE_MX4 rows' values,
 * each then rounded.  A plan whose sequences have q_len = kv_len reads caches whole.  Rows of no sequence, and of tokens
 * whose block id is out of range (reported), are left as they were.  One launch.  Errors and capture as
 * kv_append_tokens; also KV_ERR_ARG for an empty layer range, no array at all, rows of an array that
 * overlap (layers, tokens and heads may lie in any order, each stride over all that the smaller ones span), and a token's
 * k and v of more than 2^27 elements.  The two arrays overlap neither each other nor the pool. */
KV_API int kv_read_tokens(kv_attn_plan *plan, int32_t layer_begin, int32_t layer_end, const kv_read_args *args,
                          hipStream_t stream);

/* Moves cached keys to other positions: in layers [layer_begin, layer_end) the keys of each record's tokens
 * turn by delta positions, in place, without amplitude, and are rounded to the pool's type again; values
 * stay. For tokens that were appended rotated and whose places change: the middle of a conversation is
 * dropped and the rest moves up, or a reloaded chunk is used behind another prefix. kv_type is the pool's
 * element type, the pool as for kv_attn_plan_create. An e4m3 element saturates at +-448; its scale does not
 * matter. No page position may be named twice (KV_ERR_DUP for records of one table that overlap; tables
 * that share pages are not looked into), and pages that others share turn for them too
 * (kv_pool_fork_blocks, kv_copy_pages). A block id out of range is skipped and reported. shifts is a host
 * array of n (0 .. KV_MAX_SHIFTS) records, the tables are read when the call runs. One launch. Errors:
 * KV_ERR_ARG, KV_ERR_ALIGN, KV_ERR_RANGE as for kv_attn_plan_create and kv_attn_plan_set, KV_ERR_ARG for a
 * rotation wider than head_dim or of another device, and a token's k and v of more than 2^27 elements.
 * Under capture a call of at most 64 records that are not empty is captured as its kernel once the pool has
 * made a call outside the capture; any other is refused with KV_ERR_CAPTURE. */
KV_API int kv_rotate_cached(kv_pool *pool, const kv_rotation *rotation, int32_t kv_type, const kv_shift *shifts, int32_t n,
                            int32_t layer_begin, int32_t layer_end, hipStream_t stream);

/* Synchronizes `stream`, then reads and clears the pool's sticky device error
 * word.  *out_bits receives KV_DEVERR_* bits (0 if none); the return value is
 * KV_ERR_DEVICE when any bit was set, else KV_OK.
 * No passage: library infrastructure (failure detection: how a bad block id the
 * kernel skipped is reported to the caller). */
KV_API int kv_pool_get_error(kv_pool *pool, hipStream_t stream, int32_t *out_bits);

/* Kernel timing.  After kv_pool_timing_start, every transfer records a HIP
 * event pair around its kernel launch on its stream (up to 4096 launches).
 * kv_pool_timing_read synchronizes those events, writes the summed kernel time
 * in milliseconds and the number of launches timed, and stops timing.
 * kv_pool_timing_read_each does the same but writes each launch's time, in launch
 * order, to ms_each[0 .. min(cap, *launches)) (caller-owned; may be null when cap
 * is 0). */
/* No passage: library infrastructure (measurement of the kernel alone, as the
 * pages' bandwidth figures are rates of the transfer itself). */
KV_API int kv_pool_timing_start(kv_pool *pool);
KV_API int kv_pool_timing_read(kv_pool *pool, double *total_ms, int64_t *launches);
KV_API int kv_pool_timing_read_each(kv_pool *pool, double *ms_each, int64_t cap, int64_t *launches);

/* ---- pinned-host staging ring ------------------------------------------------ */

/* Allocates and pins n_slots*slot_bytes bytes of host memory once, mapped into
 * the device address space of the current device (hipHostMalloc; pinning is done
 * up front, never on the transfer path: Strata guide, "Production Cluster Sizing
 * and Configuration Guidelines", item 2).  slot_bytes must be a multiple of 16.
 * The memory is zero-filled.  Use kv_ring_slot's device pointer as
 * kv_chunk_spec.base. */
KV_API int kv_ring_create(int64_t slot_bytes, int64_t n_slots, int32_t flags, kv_ring **out);

/* Host and device addresses of slot i (0 <= i < n_slots); either out may be NULL.
 * Same source as kv_ring_create. */
KV_API int kv_ring_slot(const kv_ring *ring, int64_t i, void **host_ptr, void **dev_ptr);

/* Frees the pinned memory; the caller must have synchronized every transfer
 * that uses it.  NULL is accepted.  No passage: library infrastructure (the
 * ring's lifetime). */
KV_API int kv_ring_destroy(kv_ring *ring);

/* Slot fencing, for using the ring as a queue between the GPU and the host (slot
 * reuse across calls is fenced by events, as the Tutti summary's GPU io_uring
 * orders its I/O with events, Figure 5).  kv_ring_record marks slots
 * [first, first+count) (taken mod n_slots) as used by the work enqueued so far on
 * `stream` (one event per call).  kv_ring_wait blocks the host until the last work
 * recorded on every slot of the range has finished -- e.g. before the host reads
 * slots an offload wrote, or refills slots a reload read.  kv_ring_stream_wait
 * makes `stream` wait for that work instead.  A slot never recorded is free.
 * 1 <= count <= n_slots, 0 <= first < n_slots, else KV_ERR_ARG.  Not thread-safe. */
KV_API int kv_ring_record(kv_ring *ring, int64_t first, int64_t count, hipStream_t stream);
KV_API int kv_ring_wait(kv_ring *ring, int64_t first, int64_t count);
KV_API int kv_ring_stream_wait(kv_ring *ring, int64_t first, int64_t count, hipStream_t stream);

/* ---- misc ------------------------------------------------------------------------ */

/* Static description of a KV_* return code.  No passage: library infrastructure
 * (error reporting). */
KV_API const char *kv_strerror(int code);

/* Library version: major*10000 + minor*100 + patch (KV_VERSION of the header the
 * library was built with).  No passage: library infrastructure. */
#define KV_VERSION 400
KV_API int kv_version(void);

/* The hipError_t of the last HIP runtime call that failed inside the library on
 * the calling thread (0 if none), and in *where (if not NULL) the call's text.
 * Lets a caller that got KV_ERR_HIP see which call failed and why.  No passage:
 * library infrastructure (failure detection). */
KV_API int kv_last_hip_error(const char **where);

#ifdef __cplusplus
}
#endif

#endif /* KVXFER_H */

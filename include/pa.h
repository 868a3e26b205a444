/*
 * pa.h -- C ABI of the paged-KV attention library (GB300, sm_103a).
 *
 * The operations follow the pages on vLLM's PagedAttention:
 *   "vLLM PagedAttention chuyen sau: Phan manh bo nho KV Cache, Prefill theo
 *   khoi & Prefix Caching" (locionic.com) -- sections "Tuong tu phan trang bo
 *   nho ao" (logical blocks, physical blocks, block table, dynamic growth),
 *   "Co che PagedAttention" (look up, gather, attend), "Chunked Prefill"
 *   (mechanism, KV accumulation) and "Co che APC" step 3 (copy-on-write);
 *   "vLLM" (tellworld.net), section "PagedAttention" (fixed-size blocks
 *   located through a table; sharing).
 *
 * Conventions for every entry point
 * ---------------------------------
 * Pointers.  Every data pointer is a DEVICE pointer owned by the caller; the
 *   library allocates nothing and keeps no pointer after a call returns.
 *   16-bit tensors must be 16-byte aligned.  The only host arguments are the
 *   scalars.
 * Streams.  `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *   stream).  Every call only enqueues work on it and returns; results are
 *   ready when the stream is synchronised.
 * Cache layout.  k_cache and v_cache are each
 *   [num_blocks][num_kv_heads][block_size][head_dim], row-major, elements of
 *   `dtype`.  Token slot t of the pool is block t / block_size, offset
 *   t % block_size.  One (block, kv head) tile is block_size*head_dim
 *   contiguous elements.
 * Head grouping.  Query head h reads KV head h / (num_heads / num_kv_heads).
 * Argument errors (null pointers, bad sizes, unsupported shapes, misaligned
 *   pointers, a too-small workspace) are found on the host before anything
 *   is launched: the call returns a negative pa_status and enqueues nothing.
 * Data errors (a slot or table entry outside the pool, a context length past
 *   the table, a conflicting copy pair, a pipeline wait that gave up) are
 *   found on the device: the offending unit is skipped and a PA_DEVERR_* bit
 *   is OR-ed into *d_err (d_err may be NULL to ignore them).  No kernel traps;
 *   the context stays usable.  Read *d_err after the stream synchronises.
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PA_F16 = 0, PA_BF16 = 1 } pa_dtype;

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = -1,   /* null pointer, non-positive size, bad enum */
    PA_ERR_UNSUPPORTED = -2,   /* a shape this build has no kernel for */
    PA_ERR_OUT_OF_RANGE = -3,  /* a host scalar outside its allowed range */
    PA_ERR_CUDA = -4,          /* a CUDA runtime call failed (launch, attribute) */
    PA_ERR_WORKSPACE = -5,     /* workspace missing or smaller than required */
    PA_ERR_ALIGNMENT = -6,     /* a pointer is not 16-byte aligned */
    PA_ERR_SCRATCH_LIMIT = -7, /* pa_decode_noalloc: partials exceed its fixed scratch array */
    PA_ERR_NO_BLOCKS = -8      /* block manager: no free block and nothing evictable */
} pa_status;

/* Size of the device array pa_decode_noalloc keeps its split-K partials in. */
#define PA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* Bits OR-ed into *d_err by the kernels. */
#define PA_DEVERR_SLOT_RANGE 0x1    /* slot_mapping entry >= num_blocks*block_size */
#define PA_DEVERR_BLOCK_RANGE 0x2   /* block-table entry outside [0, num_blocks) */
#define PA_DEVERR_CONTEXT_RANGE 0x4 /* context length < 0, > max_context_len or > table */
#define PA_DEVERR_COPY_PAIR 0x8     /* copy pair out of pool, src==dst, or dst conflict; pa_evict: a new
                                       block named twice or still read */
#define PA_DEVERR_TIMEOUT 0x10      /* a bounded pipeline wait gave up */
#define PA_DEVERR_PREFIX 0x20       /* table rows that must be the same differ: a group's prefix
                                       (pa_decode_shared_prefix, pa_decode_common_prefix), a row of
                                       totals' positions (pa_decode_weights) */

/* Human-readable name of a pa_status value. */
PA_API const char *pa_status_string(int status);

/*
 * pa_reshape_and_cache -- write new tokens' K and V rows into their slots.
 * ("vLLM PagedAttention chuyen sau" (locionic.com), section "Tuong tu phan
 * trang bo nho ao": a growing sequence gets each new token a slot in one of
 * its physical blocks; section "Chunked Prefill", mechanism step 3: a
 * chunk's KV accumulates in the cache the same way.)
 *
 *   key, value     [num_tokens][num_kv_heads][head_dim] dtype, contiguous
 *   k_cache,v_cache pool as above, written in place
 *   slot_mapping   int64 [num_tokens]; slot < 0 = padding, nothing written;
 *                  slot >= num_blocks*block_size sets PA_DEVERR_SLOT_RANGE
 * Requires head_dim % 8 == 0.  num_tokens == 0 is a no-op.  Two tokens with
 * the same slot race (one of them wins); the caller must not do that.
 * The copy is bit-exact.
 */
PA_API int pa_reshape_and_cache(const void *key, const void *value, void *k_cache, void *v_cache,
                         const int64_t *slot_mapping, int num_tokens, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                         int *d_err, void *stream);

/*
 * pa_decode_partition_tokens -- the split-K partition length pa_decode uses
 * for these arguments: partition_tokens itself when > 0, otherwise the
 * automatic choice (a power of two in [256, 4096] that grows with
 * num_seqs * max_context_len * num_kv_heads, so units stay few and long when
 * the batch alone fills the GPU and get shorter when it does not).  Returns 0
 * when the arguments are invalid.
 */
PA_API int pa_decode_partition_tokens(int num_seqs, int num_heads, int num_kv_heads, int block_size,
                                      int max_context_len, int partition_tokens);

/*
 * pa_decode_workspace_bytes -- device workspace pa_decode needs for split-K
 * partials with these arguments (0 when every sequence fits one partition).
 * Layout (internal): fp32 partial accumulators and (max, sum) pairs per
 * (sequence, query head, partition).
 */
PA_API size_t pa_decode_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                        int block_size, int max_context_len, int partition_tokens);

/*
 * pa_decode -- single-query paged attention (one decode step).
 * For each sequence s and query head h, with L = context_lens[s] and
 * kvh = h / (num_heads/num_kv_heads):
 *   1. look up physical block block_tables[s][j / block_size] for j < L,
 *   2. gather K and V rows from those blocks,
 *   3. out[s][h] = sum_j softmax_j(scale * q[s][h] . K_j) V_j,
 * accumulated in fp32 and rounded once to dtype (round to nearest even).
 * Groups of 8 at head_dim 128 run on the tensor cores: the products
 * accumulate in fp32, and each softmax weight enters the weighted sum as
 * two dtype values (its rounding and the rounded residual), which keeps it
 * to about twice dtype's precision (smaller groups, and head_dim 64, keep
 * the weights in fp32).
 *
 *   out            [num_seqs][num_heads][head_dim] dtype (written)
 *   query          [num_seqs][num_heads][head_dim] dtype
 *   block_tables   int32 [num_seqs][max_blocks_per_seq]; entries past
 *                  ceil(L/block_size) are never read
 *   context_lens   int32 [num_seqs], includes the newest token; 0 gives zeros
 *   max_context_len  host upper bound on every context_lens[s]
 *   partition_tokens 0 = automatic; otherwise a positive multiple of
 *                  block_size: each sequence is split into partitions of this
 *                  many tokens, attended independently, then merged by a
 *                  log-sum-exp reduction (a second kernel on the same stream)
 *   workspace      device buffer of >= pa_decode_workspace_bytes(...) bytes
 *                  (may be NULL when that is 0); its contents are scratch
 * Supported: head_dim in {64, 128}; block_size in {8, 16, 32, 64, 128};
 *   num_heads / num_kv_heads in {1, 2, 4, 8}; dtype f16 or bf16.
 * Invalid lengths are clamped to [0, min(max_context_len,
 * max_blocks_per_seq*block_size)] and flagged; invalid table entries are
 * flagged and the keys they would supply are left out of the softmax (on
 * the CUDA-core path at block_size 8, the whole 16-key tile holding such a
 * block).
 */
PA_API int pa_decode(void *out, const void *query, const void *k_cache, const void *v_cache,
              const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
              int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
              int num_blocks, int max_context_len, float scale, int partition_tokens,
              pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err,
              void *stream);

/*
 * pa_decode_shared_prefix -- pa_decode for batches in which consecutive
 * groups of sequences share the physical blocks of a common prefix (several
 * samples of one prompt; the pages' parallel sampling / shared-prefix case:
 * "vLLM PagedAttention chuyen sau" (locionic.com), "Co che APC", and "vLLM"
 * (tellworld.net), "PagedAttention").  Each shared block is read from memory
 * once per group instead of once per sequence.
 *
 * Same arguments, layout, results and errors as pa_decode, plus:
 *   group_size     sequences g*group_size .. g*group_size+group_size-1 form
 *                  group g; num_seqs % group_size == 0, and group_size times
 *                  num_heads/num_kv_heads must be 1, 2, 4 or 8
 *   prefix_blocks  >= 1: the first prefix_blocks entries of every block-table
 *                  row of a group are the same physical blocks, and every
 *                  sequence's context covers them (context_lens[s] >=
 *                  prefix_blocks*block_size).  A group whose rows differ there
 *                  sets PA_DEVERR_PREFIX (its outputs are then undefined); a
 *                  context shorter than the prefix sets PA_DEVERR_CONTEXT_RANGE.
 *   workspace      always required: pa_decode_shared_prefix_workspace_bytes().
 * The output equals pa_decode's within the attention tolerance (the same
 * softmax, merged from partials of the prefix and of each sequence's own
 * tokens; not bit-identical to pa_decode).  Internally: one pass attends each
 * group's queries over its shared blocks as one head group, one pass attends
 * each sequence over its own tokens, and a log-sum-exp merge combines them.
 */
PA_API size_t pa_decode_shared_prefix_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                                      int head_dim, int block_size, int max_context_len,
                                                      int prefix_blocks, int partition_tokens);
PA_API int pa_decode_shared_prefix(void *out, const void *query, const void *k_cache,
                                   const void *v_cache, const int32_t *block_tables,
                                   int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                                   int group_size, int prefix_blocks, int num_heads, int num_kv_heads,
                                   int head_dim, int block_size, int num_blocks, int max_context_len,
                                   float scale, int partition_tokens, pa_dtype dtype, void *workspace,
                                   size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_decode_noalloc -- pa_decode for callers that must not allocate device
 * memory.  The pages have no counterpart; this exists for hosts that cannot
 * call cudaMalloc on this path: an inference engine that has already handed
 * nearly all HBM to its KV-cache pool (there is nothing left to allocate from,
 * and a failed allocation mid-step is fatal), or a latency-critical loop that
 * cannot afford the device-wide synchronisation cudaMalloc/cudaFree imply.
 *
 * Same arguments, results and errors as pa_decode, minus the workspace: the
 * split-K partials go to one array of PA_NOALLOC_SCRATCH_BYTES (64 MiB) that
 * the library declares as a static device variable.  Every GPU that loads the
 * library holds that array until the process exits, whether or not this entry
 * point is ever called.
 *   - Sizes whose partials would not fit (pa_decode_workspace_bytes(...) >
 *     PA_NOALLOC_SCRATCH_BYTES) return PA_ERR_SCRATCH_LIMIT and launch
 *     nothing; use pa_decode with a caller-owned workspace, or a longer
 *     partition_tokens, for those.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - All calls on a device share the one array.  Calls whose kernels can
 *     overlap on the GPU (different streams, no ordering between them) race
 *     on it and corrupt each other's results; serialise them.  The array
 *     needs no clearing: every partial is written before it is read.
 * Nothing here calls cudaMalloc, cudaFree or any allocating routine.
 */
PA_API int pa_decode_noalloc(void *out, const void *query, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, int num_seqs, int num_heads,
                             int num_kv_heads, int head_dim, int block_size, int num_blocks,
                             int max_context_len, float scale, int partition_tokens,
                             pa_dtype dtype, int *d_err, void *stream);

/*
 * pa_decode_step_host -- one whole decode step whose inputs sit in host
 * memory, as a scheduler holds them (the step the pages' engine runs per
 * generated token: copy-on-write of shared blocks, the new tokens' K/V into
 * their slots, then attention; "vLLM PagedAttention chuyen sau"
 * (locionic.com), sections "Co che PagedAttention" and "Co che APC").
 * In order on `stream`: the host inputs are brought into `staging` -- those
 * in page-locked host memory the device can address by one gather kernel
 * that reads them all, any other with its own cudaMemcpyAsync -- then
 * pa_copy_blocks (when num_pairs > 0),
 * pa_reshape_and_cache (when num_new_tokens > 0), pa_decode -- or
 * pa_decode_shared_prefix when group_size > 1 -- and the output lands in
 * out_host: written there by the kernels when out_host is page-locked host
 * memory the device can address (16-byte aligned), else written into staging
 * and copied with cudaMemcpyAsync.  All of it is asynchronous: the host buffers
 * must stay valid and unchanged until the stream has finished the step, and
 * out_host holds the result only after the caller synchronises.  Host
 * buffers should be page-locked (pinned) for the copies to be asynchronous.
 *   out_host           [num_seqs][num_heads][head_dim] dtype (written)
 *   query_host         [num_seqs][num_heads][head_dim] dtype
 *   new_key_host, new_value_host  [num_new_tokens][num_kv_heads][head_dim] dtype
 *   slot_mapping_host  int64 [num_new_tokens] (as for pa_reshape_and_cache)
 *   pairs_host         int64 [num_pairs][2] (as for pa_copy_blocks; NULL if 0)
 *   block_tables_host  int32 [num_seqs][max_blocks_per_seq]
 *   context_lens_host  int32 [num_seqs]
 *   k_cache, v_cache   the device pool, as for pa_decode
 *   group_size, prefix_blocks  0 and 0 for plain decode; otherwise as for
 *                      pa_decode_shared_prefix
 *   staging            device buffer of >= pa_decode_step_host_staging_bytes
 *                      (same shape arguments) bytes, 256-byte aligned; its
 *                      contents are scratch (it also holds the decode workspace)
 * Returns the first failing call's status (argument checks happen before any
 * copy is queued); PA_ERR_WORKSPACE if staging is missing or too small.
 */
PA_API size_t pa_decode_step_host_staging_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int block_size, int max_blocks_per_seq, int max_context_len,
                                                int num_new_tokens, int num_pairs, int group_size,
                                                int prefix_blocks, int partition_tokens);
PA_API int pa_decode_step_host(void *out_host, const void *query_host, const void *new_key_host,
                               const void *new_value_host, const int64_t *slot_mapping_host, int num_new_tokens,
                               const int64_t *pairs_host, int num_pairs, const int32_t *block_tables_host,
                               int max_blocks_per_seq, const int32_t *context_lens_host, int num_seqs,
                               int group_size, int prefix_blocks, int num_heads, int num_kv_heads, int head_dim,
                               int block_size, int num_blocks, void *k_cache, void *v_cache,
                               int max_context_len, float scale, int partition_tokens, pa_dtype dtype,
                               void *staging, size_t staging_bytes, int *d_err, void *stream);

/*
 * pa_mixed_step -- one continuous-batching step over one pool: the prompt
 * chunks of num_prefill sequences (as pa_prefill_batch) and one decode token
 * for each of num_decode other sequences (as pa_decode), together.  The
 * pages' chunked prefill, whose point is to batch prompt chunks with decodes
 * ("vLLM PagedAttention chuyen sau" (locionic.com), "Chunked Prefill",
 * mechanism steps 2 and 4).  Both halves read the pool as it is when the call
 * is reached on `stream`: write the step's new K/V first (pa_reshape_and_cache).
 * Arguments as for pa_prefill_batch (prefill_*, prefix_lens, chunk_lens on
 * the host) and pa_decode (decode_*, context_lens on the device), with the
 * pool and the model shape shared.
 *
 * One launch: with head_dim 128, 2, 4 or 8 query heads per kv head, block_size 16 to
 * 128, max_context_len <= 16384, at most 64 non-empty chunks, and a
 * workspace of at least pa_mixed_step_workspace_bytes(...) bytes, 256-byte
 * aligned and ZERO-FILLED before its first use, the step is one kernel of one
 * CTA per SM: some CTAs run the chunks (the stream-K prefill over those
 * CTAs), the others decode (sequence, kv head) units drawn from a queue the
 * whole grid shares (one partition each, so no reduce), and the chunks' CTAs
 * join the queue when their share of the chunks is done; the split of the
 * SMs follows the chunks' key tiles and the decodes' estimated K/V bytes, so
 * the tensor cores and HBM work at the same time.  The calls leave the
 * workspace's counters at zero, so one workspace serves every later step
 * whose sizes it covers; two steps must not run on one workspace at the same
 * time.  Results equal the separate calls' up to rounding.
 * Two launches otherwise (or when the workspace is smaller, e.g. only
 * pa_decode's): the chunks' kernel first on a high-priority stream the library
 * forks from `stream` and joins back into it, the decode on `stream` over the
 * SMs the chunks leave free; the workspace is then pa_decode's.  The fork
 * stream and its two events are created on the first such call on a device
 * and kept; calls from several host threads are serialised around the fork.
 * A half with no sequences is skipped.  Returns the first failing half's
 * status (the other half may have been queued).
 */
PA_API size_t pa_mixed_step_workspace_bytes(int num_prefill, int total_chunk_len, int num_decode, int num_heads,
                                            int num_kv_heads, int head_dim, int block_size, int max_context_len,
                                            int partition_tokens);
PA_API int pa_mixed_step(void *prefill_out, const void *prefill_query, const int32_t *prefill_block_tables,
                         int prefill_max_blocks, const int *prefix_lens, const int *chunk_lens, int num_prefill,
                         void *decode_out, const void *decode_query, const int32_t *decode_block_tables,
                         int decode_max_blocks, const int32_t *context_lens, int num_decode, int max_context_len,
                         int partition_tokens, void *workspace, size_t workspace_bytes, const void *k_cache,
                         const void *v_cache, int num_heads, int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, float scale, pa_dtype dtype, int *d_err, void *stream);

/*
 * pa_rotary_and_cache -- rotate the new tokens' queries and keys by their
 * positions and write keys and values into their slots: the step before
 * attention, with pa_reshape_and_cache's cache write in it.  Positions are
 * explicit and have num_axes coordinates (1 for text; time, height and width
 * for images and video), so they need not be the tokens' places in the cache.
 *   angle(t, i) = positions[pair_axis[i]][t] * inv_freq[i],   i < rot_dim / 2
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * where pair i of a head is its dimensions (i, rot_dim/2 + i), or (2i, 2i + 1)
 * when `interleaved` is non-zero; dimensions from rot_dim on pass unchanged.
 * The angle is reduced to one turn in 64-bit fixed point, so that no digits are
 * lost to a far position or a high frequency (it is off by up to |position| *
 * 2^-64 turns), the rotation is fp32, each result is rounded once.
 *
 *   query, query_out  [num_tokens][num_heads][head_dim] dtype; query_out may be
 *                     query itself (same pointer and stride) but must not
 *                     overlap it otherwise, nor key, value or the caches
 *   key, value     [num_tokens][num_kv_heads][head_dim] dtype
 *   *_stride       elements from one token's row to the next, a multiple of 8
 *                  and at least a row's elements (so slices of one fused
 *                  projection can be passed as they are); heads are contiguous
 *   positions      int32 [num_axes][num_tokens], any sign
 *   slot_mapping   as for pa_reshape_and_cache; a token whose slot is negative
 *                  still gets its query_out row
 *   inv_freq       float [rot_dim / 2] (device), finite
 *   pair_axis      int [rot_dim / 2] in HOST memory, or NULL for axis 0 throughout
 * Supported: head_dim a multiple of 16 up to 256, rot_dim a multiple of 16 up
 * to head_dim (0: a plain cache write, positions and inv_freq may be NULL), up
 * to 8 axes, any block_size.
 * num_tokens == 0 is a no-op.  The cache write of the values is bit-exact.
 */
PA_API int pa_rotary_and_cache(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                               const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                               void *k_cache, void *v_cache, const int32_t *positions, const int64_t *slot_mapping,
                               const float *inv_freq, const int *pair_axis, int num_axes, int rot_dim, int interleaved,
                               int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, pa_dtype dtype, int *d_err, void *stream);

/*
 * pa_decode_weights -- pa_decode that also adds up how much attention each
 * cached token receives, the totals pa_evict chooses by:
 *   weights_out[r][kvh][j] = weights[r][kvh][j] + sum softmax_j(...)
 * over row r's queries and the query heads of kv head kvh, for every j below
 * the longest of the row's contexts; entries from there on are left as they
 * are.  out as from pa_decode (the same kernels; equal to it up to rounding).
 *   weights, weights_out  float [num_seqs / queries_per_row][num_kv_heads]
 *                  [weights_len]; weights_out may be weights itself, else the
 *                  two must not overlap
 *   weights_len    >= max_context_len
 *   queries_per_row  consecutive sequences r*queries_per_row .. that add to one
 *                  row: 1 for plain decode; several query positions over one
 *                  cache (the last positions of a prompt observing it, several
 *                  new tokens at once) repeat the sequence's block-table row,
 *                  each with its own context length, and need scale > 0.  From 4
 *                  positions and 16 query rows (positions times heads per kv head)
 *                  on, at head_dim 128 and block_size >= 16, they may be attended
 *                  together on the tensor cores (by a rule on these numbers and
 *                  max_context_len): the row of the first position is the one
 *                  that counts (another that differs in a position's context
 *                  sets PA_DEVERR_PREFIX, outputs and totals undefined), and
 *                  partition_tokens then has no effect.  (Where V holds a NaN or
 *                  infinity within the longest of the contexts, the outputs of
 *                  the row are computed again key by key, so that it reaches
 *                  those alone that see it: 16 positions over 8191 tokens take
 *                  2.4 ms then.)
 *   workspace      >= pa_decode_weights_workspace_bytes(...) bytes, 256-byte
 *                  aligned, scratch: the partials, and every score in fp32
 *                  (num_seqs * num_heads * max_context_len * 4 bytes; rows that may
 *                  be attended together take whole sets of 32 query rows): pass
 *                  the batch's own longest length, not the model's
 * The weights are fp32 from fp32 scores; sums run in a fixed order.  Keys that
 * an invalid table entry leaves out of the softmax weigh 0.  Shapes,
 * partition_tokens, data errors as for pa_decode.
 */
PA_API size_t pa_decode_weights_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int block_size, int max_context_len, int queries_per_row,
                                                int partition_tokens);
PA_API int pa_decode_weights(void *out, const void *query, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                             int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                             int num_blocks, int max_context_len, float scale, int partition_tokens,
                             const float *weights, float *weights_out, int weights_len, int queries_per_row,
                             pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_evict -- cut sequences' caches down to `keep` tokens by their accumulated
 * attention weight.  Each kv head of a sequence of L tokens chooses for itself:
 * n = min(L, keep); when L > keep it keeps its first `sink` tokens, its last
 * `recent`, and of those between the keep - sink - recent with the largest
 * weights (the lower index first among equals; NaN counts as the least), else
 * all of them.  The kept tokens keep their order:
 *   kept[s][h][i]     index of the i-th kept token (int32; -1 from n to keep)
 *   new K/V row i     = K/V row kept[s][h][i], bit-exact, in the blocks of the
 *                     sequence's row of new_block_tables; rows past n in the
 *                     last block are left as they are
 *   new_weights[s][h][i] = weights[s][h][kept[s][h][i]], 0 from n to weights_len
 *   new_context_lens[s] = n
 * The old blocks are only read (other sequences may share them); the caller
 * drops them afterwards (pa_bm_evict_sequences).  Tokens keep the positions they
 * were rotated with, so a later token's position is no longer its index.
 *   weights, new_weights  float [num_seqs][num_kv_heads][weights_len], not
 *                  overlapping; weights_len >= max_context_len
 *   block_tables   int32 [num_seqs][max_blocks_per_seq], context_lens int32
 *   new_block_tables  int32 [num_seqs][new_max_blocks_per_seq], which must hold
 *                  min(keep, max_context_len) tokens; the entries of a row past
 *                  ceil(n / block_size) are never read.  A new block named twice, or
 *                  that one of the call's sequences still reads, sets
 *                  PA_DEVERR_COPY_PAIR and is not written
 *   new_context_lens  must not be context_lens
 *   workspace      >= pa_evict_workspace_bytes(num_blocks) bytes, 16-byte
 *                  aligned, scratch; its content on entry is ignored; not to be
 *                  shared with work that overlaps the call on the device
 * Needs sink + recent <= keep and keep >= 1.  Supported: head_dim in {64, 128},
 * block_size in {8, 16, 32, 64, 128}.  Invalid lengths are clamped and flagged
 * as in pa_decode; a row whose old table entry is out of the pool is flagged
 * and not written.
 */
PA_API size_t pa_evict_workspace_bytes(int num_blocks);
PA_API int pa_evict(void *k_cache, void *v_cache, const float *weights, float *new_weights, int weights_len,
                    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                    const int32_t *new_block_tables, int new_max_blocks_per_seq, int32_t *new_context_lens,
                    int32_t *kept, int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                    int max_context_len, int keep, int sink, int recent, pa_dtype dtype, void *workspace,
                    size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_decode_common_prefix -- pa_decode_shared_prefix for groups of any size: a
 * whole batch behind one long system prompt, tens of samples of a prompt.  The
 * prefix is attended once for the whole group on the tensor cores, with the
 * group's queries (group_size times the heads of a kv head) as rows, each
 * sequence's own tokens as in pa_decode, and the partials are merged.
 * Arguments, layout and data errors as for pa_decode_shared_prefix (an invalid
 * entry among a group's prefix blocks is flagged and that group's outputs are
 * undefined), and:
 *   group_size     any divisor of num_seqs
 *   scale          finite and > 0
 *   partition_tokens  splits the sequences' own tokens (0 = automatic)
 *   workspace      >= pa_decode_common_prefix_workspace_bytes(...) bytes,
 *                  256-byte aligned, ZERO-FILLED before its first use (its first
 *                  256 bytes hold a counter that every call that completes
 *                  leaves at zero again, so one workspace serves every later
 *                  call whose sizes it covers; after a call that set
 *                  PA_DEVERR_TIMEOUT, zero-fill it again).  It must not be shared
 *                  with work that overlaps the call on the device
 * Supported: head_dim 128, block_size in {16, 32, 64, 128}, num_heads /
 * num_kv_heads in {1, 2, 4, 8}.  Groups of more than 128 query rows (group_size
 * times heads per kv head) round the softmax weights of prefix keys to dtype, once,
 * for their product with V, as pa_prefill_chunk does; smaller ones, like pa_decode
 * with 8 heads per kv head, send them as two values of dtype, about twice its bits
 * (so that an infinity in V comes out as NaN).
 * Groups of 1, 2, 4 or 8 rows can take either call: pa_decode_shared_prefix reads
 * their prefixes at the memory's rate and is the faster one, but for a single group
 * of few kv heads.  This call / that one / pa_decode in us, own tokens up to 256:
 *   1 x 8 sequences, 8/8 heads, prefix 1024: 13/16/10, 32768: 58/119/125;
 *   8 x 2, 32/8 heads, 1024: 25/20/20, 8192: 92/65/92;
 *   64 x 8, 8/8 heads, 1024: 161/95/215, 8192: 673/349/1194.
 */
PA_API size_t pa_decode_common_prefix_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                      int block_size, int max_context_len, int group_size,
                                                      int prefix_blocks, int partition_tokens);
PA_API int pa_decode_common_prefix(void *out, const void *query, const void *k_cache, const void *v_cache,
                                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                   int num_seqs, int group_size, int prefix_blocks, int num_heads, int num_kv_heads,
                                   int head_dim, int block_size, int num_blocks, int max_context_len, float scale,
                                   int partition_tokens, pa_dtype dtype, void *workspace, size_t workspace_bytes,
                                   int *d_err, void *stream);

/*
 * pa_norm_rotary_and_cache -- pa_rotary_and_cache for models that normalise their
 * queries and keys head by head: before the rotation each head of query and key
 * becomes
 *   x[d] / sqrt(mean(x^2) + eps) * norm[d],   d < head_dim
 * in fp32 like the rotation, so that each result is rounded once.  That holds for heads
 * whose root mean square is below 2^59, and above 2^-50 or eps above 2^-80: fp32 does not
 * hold the squares of what bf16 has beyond.  Values pass unchanged.
 *   query_norm, key_norm  [head_dim] dtype (device), both required
 *   eps            finite, >= 0
 * Everything else as for pa_rotary_and_cache.
 */
PA_API int pa_norm_rotary_and_cache(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                                    const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                                    void *k_cache, void *v_cache, const int32_t *positions, const int64_t *slot_mapping,
                                    const float *inv_freq, const int *pair_axis, int num_axes, int rot_dim,
                                    int interleaved, const void *query_norm, const void *key_norm, float eps,
                                    int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                    int num_blocks, pa_dtype dtype, int *d_err, void *stream);

/*
 * Caches of 8 bits.  k_cache and v_cache hold e4m3 codes (1 sign, 4 exponent, 3
 * mantissa bits, no infinities), [num_blocks][num_kv_heads][block_size][head_dim];
 * k_scales and v_scales, uint8 [num_blocks][num_kv_heads], hold one power of two for
 * each block and kv head, 2^(byte - 127) (e8m0; 255 is NaN).  A row's values are its
 * codes times its block's scale.  Everything outside the cache stays dtype (fp16 or
 * bf16): queries, outputs, new keys and values.
 *
 * Writing (pa_reshape_and_cache_fp8, pa_rotary_and_cache_fp8).  A call decides the
 * scale of each block that it writes to, per kv head and for K and V apart:
 *   need = the smallest power of two, from 2^-64 on, with |x| <= 448 need for every
 *          element x of the rows that the call writes to the block
 *   the new scale is need when the block's first row is among them (the block starts
 *   afresh: what it held counts for nothing), else the larger of the old scale and need.
 * So a sequence fills a block from its first row on, in as many calls as it likes.  Rows
 * that the call does not write are moved to a scale that grew (rounded to nearest even
 * where their codes become subnormal, exact otherwise); in a block that starts afresh,
 * and under a scale that stays, they are left as they are.  Each new element is rounded
 * once, from fp32, to nearest even: within 2^-4 of itself, or 2^-10 need.  An infinity
 * or NaN becomes NaN and does not count towards the scale; with dtype fp16, magnitudes
 * above 61440 (the largest code times a power of two that fp16 holds) become 61440.
 * The result does not depend on the order in which the device works: where two tokens
 * name the same slot, the later one (the larger token index) is written.
 *
 *   arguments      as for pa_reshape_and_cache and pa_rotary_and_cache; k_scales and
 *                  v_scales are read and written; query_norm, key_norm and eps as for
 *                  pa_norm_rotary_and_cache, or both norms NULL for none
 * Supported: head_dim a multiple of 16 up to 256, block_size in {8, 16, 32, 64, 128}, up
 * to 65535 kv heads.  num_tokens == 0 is a no-op.
 * To find a block's tokens the slots of the whole call are looked through once a block (and
 * once more for every eight kv heads, and for a token behind padding or behind one of
 * another block): next to nothing up to some 8192 tokens, but it grows with their square.
 * Longer prompts are written faster in several calls.
 * Reading.  The attention calls take scales from 2^-64 (byte 63) on, which is what the
 * writing calls leave; caches filled in another way keep to that too.
 */
PA_API int pa_reshape_and_cache_fp8(const void *key, const void *value, uint8_t *k_cache, uint8_t *v_cache,
                                    uint8_t *k_scales, uint8_t *v_scales, const int64_t *slot_mapping, int num_tokens,
                                    int num_kv_heads, int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                                    int *d_err, void *stream);
PA_API int pa_rotary_and_cache_fp8(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                                   const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                                   uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scales, uint8_t *v_scales,
                                   const int32_t *positions, const int64_t *slot_mapping, const float *inv_freq,
                                   const int *pair_axis, int num_axes, int rot_dim, int interleaved,
                                   const void *query_norm, const void *key_norm, float eps, int num_tokens,
                                   int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                   pa_dtype dtype, int *d_err, void *stream);

/*
 * pa_decode_fp8 -- pa_decode over an 8-bit cache: softmax(scale * q . k) v with the
 * cached values as above, sums in fp32, the output rounded once to dtype.  On the
 * tensor cores for all shapes: scores are fp32 sums of exact products, of a query whose
 * elements are exact unless they are below 2^-21 (fp16) or 2^-24 (bf16) of their head's
 * largest one, and then off by up to 2^-32 of that one.  A softmax weight, times its
 * block's value scale, enters the weighted sum off by up to 2^-12 of itself or 2^-37 of
 * the largest such product, the greater of the two; into the sum of weights that divides
 * it, in fp32.  A query with an infinity or NaN gives NaN.
 * Arguments, shapes and data errors as for pa_decode (invalid table entries are flagged
 * and the keys they would supply are left out), without partition_tokens: contexts are
 * cut where that shares the batch out evenly, so that a row's last bits depend on the
 * batch that it is in.  The same call gives the same bits.
 *   workspace      >= pa_decode_fp8_workspace_bytes(...) bytes, 256-byte aligned (may
 *                  be NULL when that is 0; its size depends on the device), ZERO-FILLED
 *                  before its first use: its first 4 KB hold counters that every call
 *                  that completes leaves at zero again, so one workspace serves every
 *                  later call whose sizes it covers (after a call that set
 *                  PA_DEVERR_TIMEOUT, or whose context_lens were written while it
 *                  ran, zero-fill it again).  Not to be shared with work
 *                  that overlaps the call on the device, nor, without zero-filling
 *                  those 4 KB again, with other calls between two of these: counters
 *                  that another call left anything in are not noticed, and contexts
 *                  that were cut stay unwritten
 * max_blocks_per_seq * block_size, num_seqs * num_heads and num_blocks * num_kv_heads *
 * block_size must stay below 2^31 - 256.
 */
PA_API size_t pa_decode_fp8_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                            int block_size, int max_context_len);
PA_API int pa_decode_fp8(void *out, const void *query, const uint8_t *k_cache, const uint8_t *v_cache,
                         const uint8_t *k_scales, const uint8_t *v_scales, const int32_t *block_tables,
                         int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int num_heads,
                         int num_kv_heads, int head_dim, int block_size, int num_blocks, int max_context_len,
                         float scale, pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err,
                         void *stream);

/*
 * pa_prefill_batch_fp8 -- pa_prefill_batch over an 8-bit cache: causal attention of
 * prompt chunks whose own keys and values are in the cache already.  The sequences'
 * cached values are laid out once in 16 bits and attended as pa_prefill_batch does, but
 * with softmax weights of more bits than dtype has, so that the output's rounding is the
 * only one that counts.
 *   bf16  keys exact; values in fp16 over the greatest scale among each 128 keys of a
 *         sequence's kv head: exact where a value's scale is not below 2^-22 of that one,
 *         off by up to 2^-32 of it elsewhere; weights off by up to 2^-12 of themselves or
 *         2^-32 of the largest, times scales
 *   fp16  keys and values exact as far as fp16 reaches; weights as two fp16 values
 *   prefix_lens, chunk_lens  int [num_seqs], HOST memory
 *   workspace      >= pa_prefill_batch_fp8_workspace_bytes(...) bytes, 256-byte
 *                  aligned, required; its content on entry is ignored; not to be shared
 *                  with work that overlaps the call on the device.  It holds the
 *                  sequences' cached values in 16 bits: 4 * head_dim * num_kv_heads
 *                  bytes a token of prefix and chunk, rounded up to whole blocks (of
 *                  the 64 sequences that have most, where the batch has more)
 * Shapes, arguments and errors as for pa_prefill_batch (an invalid table entry is
 * flagged and that sequence's outputs are undefined).
 */
PA_API size_t pa_prefill_batch_fp8_workspace_bytes(const int *prefix_lens, const int *chunk_lens, int num_seqs,
                                                   int num_heads, int num_kv_heads, int head_dim, int block_size);
PA_API int pa_prefill_batch_fp8(void *out, const void *query, const uint8_t *k_cache, const uint8_t *v_cache,
                                const uint8_t *k_scales, const uint8_t *v_scales, const int32_t *block_tables,
                                int max_blocks_per_seq, const int *prefix_lens, const int *chunk_lens, int num_seqs,
                                int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                float scale, pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err,
                                void *stream);

/*
 * pa_copy_blocks_fp8 -- pa_copy_blocks for an 8-bit cache: codes and scales of each
 * pair's blocks, with the same rules and workspace (pa_copy_blocks_workspace_bytes).
 */
PA_API int pa_copy_blocks_fp8(uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scales, uint8_t *v_scales,
                              const int64_t *pairs, int num_pairs, int num_kv_heads, int head_dim, int block_size,
                              int num_blocks, void *workspace, size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_call_packed -- one of the calls above with its arguments in an array, for callers
 * whose foreign-function interface costs more per argument than these calls' kernels
 * take (the Python binding): args[i] is argument i of the call's prototype, a pointer or
 * integer as a 64-bit integer, a float as a double.  A host array (pair_axis, prefix_lens,
 * chunk_lens) may lie behind the arguments: -k points k bytes into args.  Results and
 * errors are the call's; PA_ERR_INVALID_ARG for an unknown call or a null array,
 * PA_ERR_OUT_OF_RANGE for an int that does not fit 32 bits.
 */
enum {
    PA_CALL_NORM_ROTARY_AND_CACHE = 0,
    PA_CALL_ROTARY_AND_CACHE_FP8 = 1,
    PA_CALL_RESHAPE_AND_CACHE_FP8 = 2,
    PA_CALL_DECODE_FP8 = 3,
    PA_CALL_PREFILL_BATCH_FP8 = 4,
    PA_CALL_COPY_BLOCKS_FP8 = 5
};
PA_API int pa_call_packed(int call, const int64_t *args);

/*
 * Failure detection.  Every wait inside the kernels (on TMA copies, MMA
 * completions, other warps) is bounded: after pa_bounded_wait_polls() polls
 * it gives up, ORs PA_DEVERR_TIMEOUT into *d_err and lets the kernel finish,
 * so a stuck pipeline is reported and the context stays usable.
 * pa_selftest_bounded_wait runs that same wait, with max_polls polls, on a
 * barrier nothing ever arrives on: it must set PA_DEVERR_TIMEOUT in *d_err
 * (device int) and, if d_cycles is not NULL, write the SM clock cycles the
 * wait took to *d_cycles (device long long).  Asynchronous on `stream`.
 */
PA_API int pa_bounded_wait_polls(void);
PA_API int pa_selftest_bounded_wait(int max_polls, int *d_err, long long *d_cycles, void *stream);

/*
 * pa_copy_blocks -- copy-on-write of shared blocks ("vLLM PagedAttention
 * chuyen sau" (locionic.com), section "Co che APC", step 3: a block that
 * several sequences share is copied before one of them writes into it).
 * For each pair (src, dst) of `pairs` (int64 [num_pairs][2], device), copy
 * the whole K block and V block (all kv heads) of src to dst, bit-exact.  A
 * pair is skipped and PA_DEVERR_COPY_PAIR set when an id is outside the
 * pool, src == dst, its dst appears as another pair's dst, or its dst is any
 * pair's src -- so the result never depends on the order in which pairs run.
 *
 *   workspace  device scratch of at least
 *              pa_copy_blocks_workspace_bytes(num_pairs) bytes, 16-byte
 *              aligned, owned by the caller (NULL allowed when num_pairs is
 *              0).  The call counts, in one pass over the pairs, how often
 *              each block id appears as a dst and as a src (a hash table in
 *              the workspace); each pair's copy then reads its dst's counts
 *              once, so validation costs O(num_pairs) in total.  Its content
 *              on entry is ignored; it must not be shared with work that
 *              overlaps the call on the device.
 * num_pairs above PA_COPY_MAX_PAIRS returns PA_ERR_OUT_OF_RANGE; a missing
 * or too small workspace returns PA_ERR_WORKSPACE.  One launch up to 1024
 * pairs (each copy looks through the list), three beyond (clear the table,
 * count, copy).
 */
#define PA_COPY_MAX_PAIRS (1 << 26)
PA_API size_t pa_copy_blocks_workspace_bytes(int num_pairs);
PA_API int pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *pairs, int num_pairs,
                   int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_prefill_chunk -- attention of one prompt chunk over its sequence's paged
 * KV ("vLLM PagedAttention chuyen sau" (locionic.com), section "Chunked
 * Prefill", mechanism: a long prompt is processed chunk by chunk, each chunk
 * attending to the KV its sequence has accumulated so far), causal: row i
 * (absolute position prefix_len + i) attends to keys 0 .. prefix_len + i.  The chunk's own K/V must already be in the cache
 * (pa_reshape_and_cache).  QK^T and PV run on the 5th-generation tensor cores
 * (tcgen05.mma, accumulators in TMEM) with fp32 accumulation; P is rounded
 * to dtype for the PV product;
 * the output is rounded once to dtype.
 *
 *   out    [chunk_len][num_heads][head_dim] dtype (written)
 *   query  [chunk_len][num_heads][head_dim] dtype
 *   block_table int32 [>= ceil((prefix_len+chunk_len)/block_size)]
 * scale must be finite and > 0.
 * Supported: head_dim 128, block_size in {16, 32, 64, 128}, group size in {1,2,4,8},
 * dtype f16 or bf16.
 *
 *   workspace  NULL, or device scratch of at least
 *              pa_prefill_workspace_bytes(1, chunk_len, ...) bytes, 256-byte
 *              aligned, owned by the caller, ZERO-FILLED before its first use.
 *              The work is cut into units of 256 query rows (chunk positions
 *              x the heads of one kv head).  With a workspace the kernel runs
 *              one CTA per SM, each over an equal share of the units' key
 *              tiles; a unit shared by several CTAs is finished by merging
 *              their log-sum-exp partials, which live in the workspace with a
 *              counter per unit.  Every call that completes leaves the
 *              counters at zero again, so no call needs to clear anything;
 *              after a call that set PA_DEVERR_TIMEOUT, zero-fill the
 *              workspace again.  It must not be shared with work that overlaps
 *              the call on the device.  Without a workspace each CTA computes
 *              one whole unit: the same result up to rounding, slower when the
 *              units do not fill the GPU.  A non-NULL workspace that is too
 *              small returns PA_ERR_WORKSPACE; one not 256-byte aligned,
 *              PA_ERR_ALIGNMENT.
 */
PA_API int pa_prefill_chunk(void *out, const void *query, const void *k_cache, const void *v_cache,
                     const int32_t *block_table, int prefix_len, int chunk_len, int num_heads,
                     int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                     pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_prefill_batch -- pa_prefill_chunk for several sequences in one launch
 * (continuous batching of prompt chunks: "vLLM PagedAttention chuyen sau"
 * (locionic.com), section "Chunked Prefill").  Sequence i's chunk is rows
 * row_i .. row_i + chunk_lens[i] - 1 of query and out, where row_i is the sum
 * of the earlier chunk lengths; its row r (absolute position prefix_lens[i] +
 * r) attends to keys 0 .. prefix_lens[i] + r of its own block-table row.
 *
 *   out, query    [sum(chunk_lens)][num_heads][head_dim] dtype (device)
 *   block_tables  int32 [num_seqs][max_blocks_per_seq] (device)
 *   prefix_lens, chunk_lens  int [num_seqs], HOST memory (scheduling
 *                 metadata the caller knows when it builds the batch); a
 *                 chunk length of 0 skips the sequence; prefix + chunk must
 *                 fit in max_blocks_per_seq * block_size
 * Same numerics, shapes, workspace and errors as pa_prefill_chunk; one
 * launch per 64 sequences with a non-empty chunk.  Without a workspace a
 * sequence's rows are bit-identical to a pa_prefill_chunk call on it alone
 * without one (every unit is computed whole, in the same order); with one,
 * where the key tiles are cut depends on the whole batch.
 */
PA_API int pa_prefill_batch(void *out, const void *query, const void *k_cache, const void *v_cache,
                            const int32_t *block_tables, int max_blocks_per_seq, const int *prefix_lens,
                            const int *chunk_lens, int num_seqs, int num_heads, int num_kv_heads,
                            int head_dim, int block_size, int num_blocks, float scale, pa_dtype dtype,
                            void *workspace, size_t workspace_bytes, int *d_err, void *stream);

/*
 * pa_prefill_workspace_bytes -- workspace for pa_prefill_chunk (num_seqs 1)
 * or pa_prefill_batch: enough for any num_seqs chunks whose lengths add up
 * to at most total_chunk_len, on the current device.  0 for invalid arguments.
 */
PA_API size_t pa_prefill_workspace_bytes(int num_seqs, int total_chunk_len, int num_heads, int num_kv_heads,
                                         int head_dim);

/*
 * Block manager -- host bookkeeping of the paged pool: which physical blocks
 * each sequence's block table holds, reference counts of shared blocks,
 * copy-on-write, and automatic prefix caching ("vLLM PagedAttention chuyen
 * sau" (locionic.com), "Tuong tu phan trang bo nho ao" and "Co che APC").
 * It produces exactly what the kernels consume: block-table rows, slot
 * mappings for pa_reshape_and_cache and (src, dst) pairs for pa_copy_blocks.
 * Pure host code; no GPU needed.  Not thread-safe: one owner per manager.
 *
 *   pa_bm_create(num_blocks, block_size, enable_prefix_cache)
 *       -> manager, or NULL on bad sizes.  Free blocks go out in id order.
 *   pa_bm_add_sequence(m, seq_id, tokens, n, slots, num_cached)
 *       registers a new sequence with its n prompt token ids.  With prefix
 *       caching, the longest run of whole blocks whose token ids match blocks
 *       already cached (a path in the prefix tree) is linked into the table
 *       and counted as hits; those tokens get slot -1.  Every other token
 *       gets the slot its K/V must be written to.  Each block that fills up
 *       joins the prefix tree.  PA_ERR_INVALID_ARG for a known seq_id,
 *       PA_ERR_NO_BLOCKS (nothing changed) when the pool runs out.
 *   pa_bm_fork(m, parent, child)
 *       child starts with all of parent's blocks, shared (parallel sampling).
 *   pa_bm_append_token(m, seq_id, token, slot, copy_src, copy_dst)
 *       one more token (decode step): its slot; a new block when the last
 *       one is full; if the last block is partially filled and shared, a
 *       private copy first (copy-on-write) whose (src, dst) is returned, else
 *       src = dst = -1.  The caller copies the block before writing the slot.
 *   pa_bm_free_sequence(m, seq_id)
 *       drops the sequence's references.  Unreferenced blocks in the prefix
 *       tree stay cached (reusable) until evicted; the others are free.
 *       Allocation evicts the least recently released cached leaf block when
 *       no free block is left.
 *   pa_bm_evict_sequences(m, seq_ids, num_seqs, keep)
 *       each sequence keeps min(its length, keep) tokens in fresh private
 *       blocks, for one pa_evict over the batch: read the old tables first, call
 *       this, then read the new ones.  Every new block is taken before any old
 *       one is given up, so no new table names a block that an old one of the
 *       batch does.  The references to the old blocks are dropped; their
 *       contents stay valid until work enqueued after the copy writes them.  The
 *       kept blocks no longer spell a prefix, so none of them joins the prefix
 *       tree.  All or nothing: PA_ERR_INVALID_ARG for an unknown seq_id or one
 *       named twice, PA_ERR_OUT_OF_RANGE for keep < 0, PA_ERR_NO_BLOCKS (every
 *       sequence unchanged) when the pool cannot hold the old and the new blocks.
 *   pa_bm_evict_sequence(m, seq_id, new_len)
 *       the same for one sequence and a pa_evict over it alone: what the next
 *       call of this or of any allocating function hands out may be this
 *       sequence's old blocks, so sequences that one pa_evict cuts down go
 *       through pa_bm_evict_sequences together.  PA_ERR_OUT_OF_RANGE unless
 *       0 <= new_len <= the length; PA_ERR_NO_BLOCKS (the sequence unchanged).
 *   pa_bm_block_table(m, seq_id, out, max_blocks) -> number of blocks, or
 *       PA_ERR_OUT_OF_RANGE if max_blocks is too small.
 *   pa_bm_seq_len, pa_bm_block_refcount, pa_bm_stats: introspection.  The
 *       prefix-cache hit rate is hit_tokens / query_tokens.
 */
typedef struct pa_block_manager pa_block_manager;
typedef struct {
    int num_blocks, free_blocks, cached_free_blocks, used_blocks, num_sequences;
    long long query_tokens, hit_tokens, evictions, cow_copies;
} pa_bm_counters;
PA_API pa_block_manager *pa_bm_create(int num_blocks, int block_size, int enable_prefix_cache);
PA_API void pa_bm_destroy(pa_block_manager *m);
PA_API int pa_bm_add_sequence(pa_block_manager *m, int64_t seq_id, const int32_t *tokens, int num_tokens,
                              int64_t *slots, int *num_cached_tokens);
PA_API int pa_bm_fork(pa_block_manager *m, int64_t parent_id, int64_t child_id);
PA_API int pa_bm_append_token(pa_block_manager *m, int64_t seq_id, int32_t token, int64_t *slot,
                              int64_t *copy_src, int64_t *copy_dst);
PA_API int pa_bm_free_sequence(pa_block_manager *m, int64_t seq_id);
PA_API int pa_bm_evict_sequence(pa_block_manager *m, int64_t seq_id, int new_len);
PA_API int pa_bm_evict_sequences(pa_block_manager *m, const int64_t *seq_ids, int num_seqs, int keep);
PA_API int pa_bm_block_table(const pa_block_manager *m, int64_t seq_id, int32_t *out, int max_blocks);
PA_API int64_t pa_bm_seq_len(const pa_block_manager *m, int64_t seq_id);
PA_API int pa_bm_block_refcount(const pa_block_manager *m, int block);
PA_API int pa_bm_stats(const pa_block_manager *m, pa_bm_counters *out);

#ifdef __cplusplus
}
#endif

#endif /* PA_H */

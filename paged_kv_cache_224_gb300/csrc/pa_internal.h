// Host-side declarations shared by the C-ABI layer and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pa.h"

namespace pa {

// Streaming multiprocessors of the current device, queried once per device
// (152 on a GB300; also the answer when no device is present).
inline int sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Raise a kernel's dynamic shared-memory limit once per device (the attribute
// is per device; `done` is the caller's per-kernel record of devices set).
template <typename Kernel>
int ensure_smem_attr(Kernel kern, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return PA_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return PA_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
    return PA_OK;
}

// Everything a decode launch needs; passed by value to the kernels.
struct DecodeParams {
    void *out;                   // [B][Hq][D] dtype
    const void *query;           // [B][Hq][D] dtype
    const void *k_cache;         // [NB][Hkv][bs][D]
    const void *v_cache;
    const int32_t *block_tables; // [B][MB]
    const int32_t *context_lens; // [B]
    float *ws_acc;               // [B][Hq][max_partitions][D] unnormalised partial sums
    float2 *ws_ml;               // [B][Hq][max_partitions] (running max in log2 units, sum)
    int *d_err;
    int num_seqs, num_heads, num_kv_heads, max_blocks_per_seq, num_blocks, max_context_len;
    int block_size, partition_tokens, max_partitions;
    float scale_log2;            // scale * log2(e)
    // Kernel sequence s and its head (kvh, h < G) stand for the real row
    // ((s*grp_size + h / grp_inner) * num_heads + kvh*grp_inner + h % grp_inner) of
    // query/out; ordinary decode has grp_size 1 and grp_inner G.  The
    // shared-prefix pass sets grp_size to the sequences sharing a prefix.
    int grp_size, grp_inner;
    int table_stride;            // block-table entries between kernel sequences
    int len_fixed;               // > 0: every kernel sequence has this many tokens
    int len_offset;              // tokens before this position are skipped (multiple of block_size)
    int part_base;               // partials go to partition slot part_base + part ...
    int slots;                   // ... of `slots` per (row); the reduce merges slots
    int force_partials;          // write partials even for one-partition units; no reduce
    int red_fixed_slots;         // reduce: slots before the per-sequence ones
    // Kept scores (the kernels instantiated with kScores): the scaled score, in
    // log2 units, of every (token, head of the group), as [sequence][kv head]
    // [score_stride tokens][G] (-inf for a key left out), and ws_ml is written
    // for whole-sequence units too.
    float *scores;
    long long score_stride;
    // With weights_out set (every sequence is one unit, one sequence to a row of
    // weights_width totals), the unit adds its weights to the totals itself.
    const float *weights;
    float *weights_out;
    int weights_width;
};

// One sequence's chunk in a prefill launch.  Its work units are (kv head,
// row tile of 256 query rows); their key tiles are laid end to end after the
// previous sequences' (the launcher fills in the schedule fields).
struct PrefillSeq {
    const int32_t *block_table;  // [>= ceil((prefix_len+chunk_len)/bs)]
    int prefix_len, chunk_len;
    int row_start;               // first row of the chunk in query/out
    int row_tiles;               // row tiles of the chunk (ceil(chunk_len * group / 256))
    int tiles_per_head;          // key tiles of all its row tiles for one kv head
    int tile_start;              // global index of its first key tile
    int unit_start;              // global index of its first unit
};

constexpr int kPrefillMaxSeqs = 64;  // sequences per launch (kernel-parameter table)

struct PrefillParams {
    void *out;                   // [rows][Hq][D], the chunks one after another
    const void *query;           // [rows][Hq][D]
    const void *k_cache;
    const void *v_cache;
    int *d_err;
    int num_heads, num_kv_heads, num_blocks;
    float scale_log2;
    int num_seqs;                // entries of seqs in use (1 .. kPrefillMaxSeqs)
    int query_rows;              // rows of query/out (all chunks of the call, across launches)
    int total_tiles;             // key tiles of all units
    int split;                   // 1: stream-K ranges over gridDim.x CTAs, with merging; 0: one unit per CTA
    float *part_o;               // split: [2 * CTAs][2 Q tiles][128 rows][128] unnormalised O of partial units
    float2 *part_ml;             // split: [2 * CTAs][2 Q tiles][128 rows] (running max, sum)
    unsigned *counters;          // split: [units][2 Q tiles] segments counted so far; zero on entry, and
                                 // the merging segment resets its unit's to zero before the call ends
    int part_slots;              // shared prefix: part_o and part_ml are [row][Hq][part_slots], one slot per piece
    // several queries over one cache (kWindow): query row r of the call has
    // context_lens[r] tokens, at most len_cap; the scores (not scaled) go to
    // [row_base + entry of seqs][kv head][plane of 32 query rows][score_stride keys][32]
    const int32_t *context_lens;
    int len_cap, row_base;
    float *scores;
    long long score_stride;
    PrefillSeq seqs[kPrefillMaxSeqs];
};

// One launch of a continuous-batching step: CTAs 0 .. prefill_ctas-1 run the
// prompt chunks (the stream-K prefill over those CTAs), the others the decodes
// as a persistent role (one partition per sequence, so no reduce).
struct MixedParams {
    PrefillParams pp;
    DecodeParams dp;
    int prefill_ctas;
    int decode_units;            // sequences x kv heads
    unsigned *decode_next;       // the decode CTAs' shared unit queue (0 between launches)
};

// One launch of the rotary cache write.
constexpr int kRotaryMaxDim = 256;   // largest head_dim
constexpr int kRotaryMaxAxes = 8;
struct RotaryParams {
    void *query_out;             // [T][Hq][D], token stride query_out_stride
    const void *query;           // [T][Hq][D], token stride query_stride
    const void *key;             // [T][Hkv][D]
    const void *value;
    void *k_cache;               // [NB][Hkv][bs][D]
    void *v_cache;
    const int32_t *positions;    // [axes][T]
    const int64_t *slots;        // [T]
    const float *inv_freq;       // [rot_dim / 2]
    int *d_err;
    long long query_out_stride, query_stride, key_stride, value_stride;  // elements
    int num_tokens, num_heads, num_kv_heads, head_dim, rot_dim, interleaved;
    int block_size, num_blocks;
    uint8_t pair_axis[kRotaryMaxDim / 2];
};

// One eviction (see pa_evict): the kernels mark, select and copy.
struct EvictParams {
    void *k_cache;               // [NB][Hkv][bs][D]
    void *v_cache;
    const float *weights;        // [B][Hkv][width]
    float *new_weights;          // [B][Hkv][width]
    const int32_t *block_tables; // [B][max_blocks]
    const int32_t *new_block_tables;  // [B][new_max_blocks]
    const int32_t *context_lens; // [B]
    int32_t *new_context_lens;   // [B]
    int32_t *kept;               // [B][Hkv][keep]
    int *owner;                  // workspace: [NB]
    int *d_err;
    int num_seqs, num_kv_heads, head_dim, block_size, num_blocks, max_blocks, new_max_blocks;
    int width, max_context_len, keep, sink, recent;
    int one_check;               // one CTA beside the selecting ones marks and checks all blocks
};

// Split-K partition length for the automatic setting.
int auto_partition_tokens(int num_seqs, int num_heads, int num_kv_heads, int block_size, int max_context_len);

// Kernel launchers.  Each returns PA_OK, PA_ERR_UNSUPPORTED (no instance for
// the shape) or PA_ERR_CUDA (launch / attribute failure).
int launch_decode(pa_dtype dt, int head_dim, int block_size, int group, const DecodeParams &p,
                  cudaStream_t stream);
// Groups whose decode runs on the tensor cores at head_dim 128: only groups
// of 8, where every K/V byte feeds 8 dot products and 8 weighted sums and the
// CUDA-core kernel runs out of issue slots well below the HBM bound.  Groups
// of 1, 2 and 4 are HBM-bound on the CUDA cores and stay there.
inline bool decode_tc_group(int group) { return group == 8; }
// Decode on the tensor cores (the decode kernel only; the caller launches the
// reduce).  PA_ERR_UNSUPPORTED for any other shape, or when the driver
// refuses the kernel's tensor maps.
int launch_decode_tc(pa_dtype dt, int head_dim, int block_size, int group, const DecodeParams &p,
                     cudaStream_t stream);
// The decode kernels that keep their scores (p.scores), without a merge of the
// partials: launch_weights_merge does that together with the totals.
int launch_decode_scores(pa_dtype dt, int head_dim, int block_size, int group, const DecodeParams &p,
                         cudaStream_t stream);
int launch_decode_scores_bf16(int head_dim, int block_size, int group, const DecodeParams &p, cudaStream_t stream);
int launch_decode_scores_f16(int head_dim, int block_size, int group, const DecodeParams &p, cudaStream_t stream);
int launch_decode_tc_scores(pa_dtype dt, int head_dim, int block_size, int group, const DecodeParams &p,
                            cudaStream_t stream);
// Partition length when the caller leaves it open.
int weights_partition_tokens(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                             int max_context_len);
// After launch_decode_scores: merges split sequences' partials into p.out and
// adds every token's weights to its row's total, queries_per_row sequences to
// a row of `width` totals.  one_table: flags sequences of a row whose table rows differ.
int launch_weights_merge(pa_dtype dt, int head_dim, int group, const DecodeParams &p, const float *weights,
                         float *weights_out, int width, int queries_per_row, bool one_table, cudaStream_t stream);
// Log-sum-exp merge of the partials in p's workspace into p.out.
int launch_decode_reduce(pa_dtype dt, int head_dim, const DecodeParams &p, cudaStream_t stream);
int launch_reshape_and_cache(const void *key, const void *value, void *k_cache, void *v_cache,
                             const int64_t *slots, int num_tokens, int num_kv_heads, int head_dim,
                             int block_size, int num_blocks, int *d_err, cudaStream_t stream);
int launch_rotary(pa_dtype dt, const RotaryParams &p, cudaStream_t stream);
int launch_evict(const EvictParams &p, cudaStream_t stream);
// Copies of up to kGatherMax buffers in one launch, each from memory the
// device can address (pinned host memory through its device view included)
// to device memory: 16-byte vectors where both ends and the size allow,
// bytes otherwise.
constexpr int kGatherMax = 8;
struct GatherList {
    const void *src[kGatherMax];
    void *dst[kGatherMax];
    unsigned long long bytes[kGatherMax];
    int n;
};
int launch_gather(const GatherList &list, cudaStream_t stream);
size_t copy_blocks_workspace_bytes(int num_pairs);
int launch_copy_blocks(void *k_cache, void *v_cache, const int64_t *pairs, int num_pairs,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks, void *workspace,
                       int *d_err, cudaStream_t stream);
// Workspace for the stream-K prefill schedule (an upper bound for any batch of
// num_seqs chunks totalling total_chunk_len rows).
size_t prefill_workspace_bytes(int num_seqs, long long total_chunk_len, int group, int num_kv_heads);
// workspace may be NULL (or too small): each CTA then computes one whole unit.
int launch_prefill(pa_dtype dt, int head_dim, int block_size, int group, const PrefillParams &p,
                   void *workspace, size_t workspace_bytes, cudaStream_t stream);
// Attention of a batch over long shared prefixes (pa_decode_common_prefix):
// `groups` groups of group_size consecutive sequences, each over the first
// prefix_tokens tokens of its first sequence's table, and every sequence over
// its own tokens.  A unit's key tiles are shared out over the CTAs as in the
// stream-K prefill, and each piece of a unit leaves an unnormalised partial in
// its own slot; prefix_pieces is the most pieces a unit can be cut into.
// The schedule of one launch, of up to kPrefillMaxSeqs groups.
struct PrefixSchedule {
    long long tiles;  // key tiles of all units
    int row_tiles;    // units per (group, kv head)
    int n;            // key tiles per unit
    int ctas;         // CTAs that the tiles are shared out to
};
// The launches of a call: full ones, whose CTAs have nothing to decode (none, if
// the groups fit one launch), and the last, with the own tokens of all sequences.
struct PrefixSchedules {
    PrefixSchedule full, last;
    int last_groups;
};
struct PrefixParams {
    DecodeParams d;              // of the own tokens: d.slots, d.part_base (= pieces), d.len_offset
    int groups, group_size, prefix_tokens;
    PrefixSchedules sched;
    unsigned *queue;             // the decode instances' shared unit queue, one counter
};
// One launch: the prefixes of up to kPrefillMaxSeqs groups; the last one also
// runs the own tokens of every sequence.
struct PrefixLaunch {
    PrefillParams pp;
    DecodeParams dp;
    int prefix_ctas, decode_units;
    unsigned *decode_next;
};
// Whether a group's softmax weights over its prefix go to their product with V as
// two values (pa_prefill.cuh): its rows fit one of a unit's two Q tiles.
inline bool prefix_two_values(int group_size, int group) { return (long long)group_size * group <= 128; }
PrefixSchedules prefix_schedules(int groups, int group_size, int prefix_tokens, int group, int num_kv_heads,
                                 int longest_own, int partitions, int num_seqs);
int prefix_pieces(int groups, const PrefixSchedules &x);
// Partition length of the own tokens when the caller leaves it open: the
// decode instances take units from a queue, so a sequence is split only as far
// as it takes to give each about four.
int prefix_partition_tokens(int num_seqs, int num_kv_heads, int block_size, int longest_own);
int launch_prefix(pa_dtype dt, int block_size, int group, const PrefixParams &pp, cudaStream_t stream);
int launch_prefix_merge(pa_dtype dt, int group, const PrefixParams &pp, cudaStream_t stream);
int launch_prefix_bf16(int block_size, int group, const PrefixLaunch &pl, unsigned grid, cudaStream_t stream);
int launch_prefix_f16(int block_size, int group, const PrefixLaunch &pl, unsigned grid, cudaStream_t stream);
// Several query positions over one cache, with the totals of their weights
// (pa_decode_weights with enough queries per row): every row of queries_per_row
// consecutive sequences is attended together on the tensor cores, its scores
// kept (window_score_floats in all), and then merged and added up.  window_pieces: the most pieces (partials) of a unit.
bool window_supported(int head_dim, int block_size, int group, int queries_per_row);
bool window_preferred(int group, int queries_per_row, int max_context_len);
int window_pieces(int rows, int queries_per_row, int group, int num_kv_heads, int max_context_len);
inline long long window_score_stride(int max_context_len) { return ((long long)max_context_len + 127) / 128 * 128; }
inline size_t window_score_floats(int rows, int num_kv_heads, int query_rows, int max_context_len) {
    return (size_t)rows * num_kv_heads * (((size_t)query_rows + 31) / 32 * 32) * window_score_stride(max_context_len);
}
int launch_window(pa_dtype dt, int block_size, int group, const DecodeParams &d, int queries_per_row,
                  const float *weights, float *weights_out, int width, cudaStream_t stream);
int launch_window_bf16(int block_size, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream);
int launch_window_f16(int block_size, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream);
// Whether launch_mixed has a kernel for these (head_dim 128, a tensor-core
// decode group, block_size 16..128).
bool mixed_supported(int head_dim, int block_size, int group);
// The one-launch step's kernel instances, one translation unit per dtype.
int launch_mixed_bf16(int block_size, int group, const MixedParams &mp, unsigned grid, cudaStream_t stream);
int launch_mixed_f16(int block_size, int group, const MixedParams &mp, unsigned grid, cudaStream_t stream);
// The fused step: pp as for launch_prefill (at most kPrefillMaxSeqs chunks),
// dp as for launch_decode with one partition per sequence; prefill_ws as for
// launch_prefill (required); decode_bytes: the decodes' K/V bytes, estimated,
// to split the SMs between the two halves.
int launch_mixed(pa_dtype dt, int block_size, int group, const PrefillParams &pp, const DecodeParams &dp,
                 void *workspace, size_t workspace_bytes, double decode_bytes, cudaStream_t stream);

}  // namespace pa

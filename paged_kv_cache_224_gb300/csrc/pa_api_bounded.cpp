// C-ABI entry points of the bounded and the shared cache: rotary cache write,
// decode with attention weights, eviction, decode over a long shared prefix.
// Host-side argument validation, then kernel dispatch; nothing here allocates
// device memory or synchronises the stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }
bool aligned16(const void *p) { return aligned(p, 16); }

bool good_dtype(pa_dtype d) { return d == PA_F16 || d == PA_BF16; }

bool good_block(int bs) { return bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs == 128; }

bool good_group(int g) { return g == 1 || g == 2 || g == 4 || g == 8; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// A caller's partition_tokens, at most what holds the longest length: the kernels
// add a length to it in 32 bits.
int clamp_partition(int partition_tokens, int longest, int block_size) {
    const long long whole = ((long long)std::max(longest, 1) + block_size - 1) / block_size * block_size;
    return (int)std::min<long long>(partition_tokens, whole);
}

// Partials: fp32 accumulators, then (max, sum) pairs, `slots` per (sequence, head).
struct PartialWs {
    size_t acc, ml;
    PartialWs(int num_seqs, int num_heads, int head_dim, int slots) {
        const size_t n = (size_t)num_seqs * num_heads * slots;
        acc = round256(n * head_dim * sizeof(float));
        ml = round256(n * 2 * sizeof(float));
    }
};

// Decode with kept scores: the partials, then the scores.  `window`: the rows of
// several queries are attended together; where a shape allows that, the workspace
// holds either form.
struct WeightsWs {
    int pt = 1, slots;
    long long stride;  // tokens of a row's scores
    size_t acc, ml, scores, bytes;
    bool one_table, window, ok;  // one_table: the queries of a row are to have the same table row
    WeightsWs(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int max_context_len,
              int queries_per_row, int partition_tokens) {
        const int group = num_heads / num_kv_heads;
        one_table = pa::window_supported(head_dim, block_size, group, queries_per_row);
        window = one_table && pa::window_preferred(group, queries_per_row, max_context_len);
        ok = partition_tokens >= 0 && partition_tokens % block_size == 0;
        if (!ok) return;
        const int rows = num_seqs / queries_per_row;
        bytes = 0;
        for (const bool together : {!window, window}) {  // the form that is not taken, then the one that is
            if (together && !one_table) continue;
            if (together) {
                slots = pa::window_pieces(rows, queries_per_row, group, num_kv_heads, max_context_len);
                stride = pa::window_score_stride(max_context_len);
            } else {
                pt = partition_tokens ? clamp_partition(partition_tokens, max_context_len, block_size)
                                      : pa::weights_partition_tokens(num_seqs, num_heads, num_kv_heads, head_dim,
                                                                     block_size, max_context_len);
                slots = std::max(1, (int)(((long long)max_context_len + pt - 1) / pt));
                stride = ((long long)max_context_len + 3) / 4 * 4;
            }
            const PartialWs w(num_seqs, num_heads, head_dim, slots);
            acc = slots > 1 || together ? w.acc : 0;
            ml = w.ml;
            scores = round256((together ? pa::window_score_floats(rows, num_kv_heads, queries_per_row * group, max_context_len)
                                        : (size_t)num_seqs * num_heads * stride) *
                              sizeof(float));
            bytes = std::max(bytes, acc + ml + scores);
        }
    }
    size_t total() const { return bytes; }
};

// The shared-prefix step: the decode instances' queue counter, then the partials.
constexpr size_t kQueueBytes = 256;
struct PrefixWs {
    int pt, pieces, slots;
    pa::PrefixSchedules sched;
    size_t acc, ml;
    bool ok;
    PrefixWs(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int max_context_len,
             int group_size, int prefix_blocks, int partition_tokens) {
        const int prefix = prefix_blocks * block_size;
        const int longest = max_context_len - prefix;
        ok = partition_tokens >= 0 && partition_tokens % block_size == 0;
        if (!ok) return;
        pt = partition_tokens ? clamp_partition(partition_tokens, longest, block_size)
                              : pa::prefix_partition_tokens(num_seqs, num_kv_heads, block_size, longest);
        const int partitions = std::max(1, (int)(((long long)longest + pt - 1) / pt));
        const int groups = num_seqs / group_size;
        sched = pa::prefix_schedules(groups, group_size, prefix, num_heads / num_kv_heads, num_kv_heads, longest,
                                     partitions, num_seqs);
        pieces = pa::prefix_pieces(groups, sched);
        slots = pieces + partitions;
        const PartialWs w(num_seqs, num_heads, head_dim, slots);
        acc = w.acc;
        ml = w.ml;
    }
    size_t total() const { return kQueueBytes + acc + ml; }
};

bool prefix_sizes_ok(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int max_context_len,
                     int group_size, int prefix_blocks) {
    return num_seqs > 0 && num_heads > 0 && num_kv_heads > 0 && num_heads % num_kv_heads == 0 && head_dim > 0 &&
           block_size > 0 && max_context_len >= 0 && group_size > 0 && num_seqs % group_size == 0 && prefix_blocks > 0 &&
           (long long)prefix_blocks * block_size <= max_context_len;
}

pa::DecodeParams decode_params(void *out, const void *query, const void *k_cache, const void *v_cache,
                               const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                               int num_seqs, int num_heads, int num_kv_heads, int block_size, int num_blocks,
                               int max_context_len, float scale, int pt, int *d_err) {
    pa::DecodeParams p{};
    p.out = out;
    p.query = query;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.d_err = d_err;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.max_context_len = max_context_len;
    p.block_size = block_size;
    p.partition_tokens = pt;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.grp_size = 1;
    p.grp_inner = num_heads / num_kv_heads;
    p.table_stride = max_blocks_per_seq;
    return p;
}

}  // namespace

extern "C" {

int pa_rotary_and_cache(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                        const void *key, int64_t key_stride, const void *value, int64_t value_stride, void *k_cache,
                        void *v_cache, const int32_t *positions, const int64_t *slot_mapping, const float *inv_freq,
                        const int *pair_axis, int num_axes, int rot_dim, int interleaved, int num_tokens, int num_heads,
                        int num_kv_heads, int head_dim, int block_size, int num_blocks, pa_dtype dtype, int *d_err,
                        void *stream) {
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        num_axes <= 0 || rot_dim < 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_axes > pa::kRotaryMaxAxes || head_dim > pa::kRotaryMaxDim || head_dim % 16 || rot_dim % 16)
        return PA_ERR_UNSUPPORTED;
    if (rot_dim > head_dim) return PA_ERR_OUT_OF_RANGE;
    if ((long long)num_heads + 2LL * num_kv_heads > 0x7fffffffLL / head_dim) return PA_ERR_UNSUPPORTED;
    const int64_t qrow = (int64_t)num_heads * head_dim, krow = (int64_t)num_kv_heads * head_dim;
    if (query_out_stride < qrow || query_stride < qrow || key_stride < krow || value_stride < krow)
        return PA_ERR_OUT_OF_RANGE;
    pa::RotaryParams p{};
    for (int i = 0; i < rot_dim / 2; ++i) {
        const int a = pair_axis ? pair_axis[i] : 0;
        if (a < 0 || a >= num_axes) return PA_ERR_OUT_OF_RANGE;
        p.pair_axis[i] = (uint8_t)a;
    }
    if (num_tokens == 0) return PA_OK;
    if (!query_out || !query || !key || !value || !k_cache || !v_cache || !slot_mapping ||
        (rot_dim > 0 && (!positions || !inv_freq)))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query_out) || !aligned16(query) || !aligned16(key) || !aligned16(value) || !aligned16(k_cache) ||
        !aligned16(v_cache) || (query_out_stride | query_stride | key_stride | value_stride) % 8)
        return PA_ERR_ALIGNMENT;
    p.query_out = query_out;
    p.query = query;
    p.key = key;
    p.value = value;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.positions = positions;
    p.slots = slot_mapping;
    p.inv_freq = inv_freq;
    p.d_err = d_err;
    p.query_out_stride = query_out_stride;
    p.query_stride = query_stride;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved != 0;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    return pa::launch_rotary(dtype, p, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_weights_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                         int max_context_len, int queries_per_row, int partition_tokens) {
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        block_size <= 0 || max_context_len < 0 || queries_per_row <= 0 || num_seqs % queries_per_row)
        return 0;
    const WeightsWs w(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, queries_per_row,
                      partition_tokens);
    return w.ok ? w.total() : 0;
}

int pa_decode_weights(void *out, const void *query, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                      int max_context_len, float scale, int partition_tokens, const float *weights, float *weights_out,
                      int weights_len, int queries_per_row, pa_dtype dtype, void *workspace, size_t workspace_bytes,
                      int *d_err, void *stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || weights_len < 0 || queries_per_row <= 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads || num_seqs % queries_per_row) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || max_context_len > weights_len) return PA_ERR_OUT_OF_RANGE;
    if (queries_per_row > 1 && !(scale > 0.f)) return PA_ERR_OUT_OF_RANGE;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens ||
        (weights_len > 0 && (!weights || !weights_out)))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if ((head_dim != 64 && head_dim != 128) || !good_block(block_size) || !good_group(group)) return PA_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGNMENT;
    const size_t totals = (size_t)(num_seqs / queries_per_row) * num_kv_heads * weights_len * sizeof(float);
    if (weights != weights_out && overlap(weights, totals, weights_out, totals)) return PA_ERR_INVALID_ARG;
    const WeightsWs w(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, queries_per_row,
                      partition_tokens);
    if (!w.ok) return PA_ERR_OUT_OF_RANGE;
    if (!workspace || workspace_bytes < w.total()) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PA_ERR_ALIGNMENT;
    pa::DecodeParams p =
        decode_params(out, query, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_heads,
                      num_kv_heads, block_size, num_blocks, max_context_len, scale, w.pt, d_err);
    p.max_partitions = w.slots;
    p.slots = w.slots;
    char *base = static_cast<char *>(workspace);
    p.ws_acc = reinterpret_cast<float *>(base);
    p.ws_ml = reinterpret_cast<float2 *>(base + w.acc);
    p.scores = reinterpret_cast<float *>(base + w.acc + w.ml);
    p.score_stride = w.stride;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (w.window)
        return pa::launch_window(dtype, block_size, group, p, queries_per_row, weights, weights_out, weights_len, st);
    const bool whole = w.slots == 1 && queries_per_row == 1;  // every sequence is one unit
    if (whole) {
        p.weights = weights;
        p.weights_out = weights_out;
        p.weights_width = weights_len;
    }
    const int rc = pa::launch_decode_scores(dtype, head_dim, block_size, group, p, st);
    if (rc != PA_OK || whole) return rc;
    return pa::launch_weights_merge(dtype, head_dim, group, p, weights, weights_out, weights_len, queries_per_row,
                                    w.one_table, st);
}

size_t pa_evict_workspace_bytes(int num_blocks) {
    return num_blocks > 0 ? round256((size_t)num_blocks * sizeof(int)) : 0;
}

int pa_evict(void *k_cache, void *v_cache, const float *weights, float *new_weights, int weights_len,
             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
             const int32_t *new_block_tables, int new_max_blocks_per_seq, int32_t *new_context_lens, int32_t *kept,
             int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks, int max_context_len, int keep,
             int sink, int recent, pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err, void *stream) {
    if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || new_max_blocks_per_seq <= 0 || max_context_len < 0 || weights_len < 0 || keep <= 0 ||
        sink < 0 || recent < 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if ((long long)sink + recent > keep || max_context_len > weights_len) return PA_ERR_OUT_OF_RANGE;
    if ((long long)new_max_blocks_per_seq * block_size < std::min(keep, max_context_len)) return PA_ERR_OUT_OF_RANGE;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || (weights_len > 0 && (!weights || !new_weights)) || !block_tables || !context_lens ||
        !new_block_tables || !new_context_lens || !kept)
        return PA_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || !good_block(block_size)) return PA_ERR_UNSUPPORTED;
    if ((long long)num_seqs * new_max_blocks_per_seq > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGNMENT;
    const size_t totals = (size_t)num_seqs * num_kv_heads * weights_len * sizeof(float);
    if (overlap(weights, totals, new_weights, totals) ||
        overlap(context_lens, (size_t)num_seqs * 4, new_context_lens, (size_t)num_seqs * 4))
        return PA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < pa_evict_workspace_bytes(num_blocks)) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_ALIGNMENT;
    pa::EvictParams p{};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.weights = weights;
    p.new_weights = new_weights;
    p.block_tables = block_tables;
    p.new_block_tables = new_block_tables;
    p.context_lens = context_lens;
    p.new_context_lens = new_context_lens;
    p.kept = kept;
    p.owner = static_cast<int *>(workspace);
    p.d_err = d_err;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.new_max_blocks = new_max_blocks_per_seq;
    p.width = weights_len;
    p.max_context_len = max_context_len;
    p.keep = keep;
    p.sink = sink;
    p.recent = recent;
    return pa::launch_evict(p, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_common_prefix_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                               int block_size, int max_context_len, int group_size, int prefix_blocks,
                                               int partition_tokens) {
    if (!prefix_sizes_ok(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, group_size,
                         prefix_blocks))
        return 0;
    const PrefixWs w(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, group_size, prefix_blocks,
                     partition_tokens);
    return w.ok ? w.total() : 0;
}

int pa_decode_common_prefix(void *out, const void *query, const void *k_cache, const void *v_cache,
                            const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                            int num_seqs, int group_size, int prefix_blocks, int num_heads, int num_kv_heads,
                            int head_dim, int block_size, int num_blocks, int max_context_len, float scale,
                            int partition_tokens, pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err,
                            void *stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || group_size <= 0 || prefix_blocks <= 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads || num_seqs % group_size) return PA_ERR_INVALID_ARG;
    if (prefix_blocks > max_blocks_per_seq || (long long)prefix_blocks * block_size > max_context_len)
        return PA_ERR_OUT_OF_RANGE;
    if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_OUT_OF_RANGE;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (head_dim != 128 || !good_block(block_size) || block_size < 16 || !good_group(group)) return PA_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGNMENT;
    const PrefixWs w(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, group_size, prefix_blocks,
                     partition_tokens);
    if (!w.ok) return PA_ERR_OUT_OF_RANGE;
    if (!workspace || workspace_bytes < w.total()) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PA_ERR_ALIGNMENT;
    pa::PrefixParams pp{};
    pp.groups = num_seqs / group_size;
    pp.group_size = group_size;
    pp.prefix_tokens = prefix_blocks * block_size;
    pp.sched = w.sched;
    pp.d = decode_params(out, query, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                         num_heads, num_kv_heads, block_size, num_blocks, max_context_len, scale, w.pt, d_err);
    pa::DecodeParams &d = pp.d;
    // the queue's counter comes first, so that it stays put whatever the call's sizes
    char *base = static_cast<char *>(workspace);
    pp.queue = reinterpret_cast<unsigned *>(base);
    d.ws_acc = reinterpret_cast<float *>(base + kQueueBytes);
    d.ws_ml = reinterpret_cast<float2 *>(base + kQueueBytes + w.acc);
    d.len_offset = pp.prefix_tokens;
    d.part_base = w.pieces;
    d.slots = w.slots;
    d.max_partitions = w.slots - w.pieces;
    d.force_partials = 1;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = pa::launch_prefix(dtype, block_size, group, pp, st);
    if (rc != PA_OK) return rc;
    return pa::launch_prefix_merge(dtype, group, pp, st);
}

}  // extern "C"

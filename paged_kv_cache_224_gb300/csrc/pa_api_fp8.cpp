// C-ABI entry points of 8-bit caches, and of the norms of queries and keys that may
// go with either kind of cache.  Host-side argument validation, then kernel dispatch;
// nothing here allocates device memory or synchronises the stream.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

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
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// The rotary call's checks, in p what they leave.  PA_OK with p.num_tokens 0: nothing to do.
int rotary_params(pa::RotaryParams &p, void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                  const void *key, int64_t key_stride, const void *value, int64_t value_stride, void *k_cache,
                  void *v_cache, const int32_t *positions, const int64_t *slot_mapping, const float *inv_freq,
                  const int *pair_axis, int num_axes, int rot_dim, int interleaved, const void *query_norm,
                  const void *key_norm, float eps, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                  int block_size, int num_blocks, pa_dtype dtype, int *d_err) {
    if (num_tokens < 0 || num_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        num_axes <= 0 || rot_dim < 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_axes > pa::kRotaryMaxAxes || head_dim > pa::kRotaryMaxDim || head_dim % 16 || rot_dim % 16)
        return PA_ERR_UNSUPPORTED;
    if (rot_dim > head_dim) return PA_ERR_OUT_OF_RANGE;
    if ((long long)num_heads + 2LL * num_kv_heads > 0x7fffffffLL / head_dim) return PA_ERR_UNSUPPORTED;
    const int64_t qrow = (int64_t)num_heads * head_dim, krow = (int64_t)num_kv_heads * head_dim;
    if (query_out_stride < qrow || query_stride < qrow || key_stride < krow || value_stride < krow)
        return PA_ERR_OUT_OF_RANGE;
    if (!std::isfinite(eps) || eps < 0.f) return PA_ERR_OUT_OF_RANGE;
    if ((query_norm == nullptr) != (key_norm == nullptr)) return PA_ERR_INVALID_ARG;
    p.one_axis = 1;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const int a = pair_axis ? pair_axis[i] : 0;
        if (a < 0 || a >= num_axes) return PA_ERR_OUT_OF_RANGE;
        p.pair_axis[i] = (uint8_t)a;
        if (a) p.one_axis = 0;
    }
    p.num_tokens = num_tokens;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping || (num_heads > 0 && (!query_out || !query)) ||
        (rot_dim > 0 && (!positions || !inv_freq)))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query_out) || !aligned16(query) || !aligned16(key) || !aligned16(value) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(query_norm) || !aligned16(key_norm) || (query_out_stride | query_stride | key_stride | value_stride) % 8)
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
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved != 0;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.query_norm = query_norm;
    p.key_norm = key_norm;
    p.eps = eps;
    return PA_OK;
}

int store_fp8(pa::RotaryParams &p, uint8_t *k_scales, uint8_t *v_scales, pa_dtype dtype, void *stream) {
    if (!good_block(p.block_size) || p.num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (!k_scales || !v_scales || k_scales == v_scales || p.k_cache == p.v_cache) return PA_ERR_INVALID_ARG;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    return pa::launch_store_fp8(dtype, p, static_cast<cudaStream_t>(stream));
}

// The decode's workspace: counters (where they are does not depend on the call), the
// partials' accumulators and (max, sum) pairs.  None where every context is a single tile.
struct DecodeWs {
    int ctas;
    size_t counters = 0, acc = 0, ml = 0;
    DecodeWs(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_context_len) {
        ctas = pa::fp8_decode_ctas(num_seqs, num_kv_heads, num_heads / num_kv_heads, head_dim, max_context_len);
        if (max_context_len <= 128) return;
        const size_t n = (size_t)2 * ctas * (num_heads / num_kv_heads);
        counters = pa::kFp8MaxCtas * sizeof(unsigned);
        acc = round256(n * head_dim * sizeof(float));
        ml = round256(n * 2 * sizeof(float));
    }
    size_t total() const { return counters + acc + ml; }
};

// The prefill's own workspace for a launch of up to kPrefillMaxSeqs chunks, then the
// expanded blocks' table, keys and values.  The launches of a call take turns in it.
struct PrefillWs {
    size_t pre = 0, table = 0, pool = 0;
    long long blocks = 0;  // of the launch that has most
    PrefillWs(const int *prefix_lens, const int *chunk_lens, int num_seqs, int group, int num_kv_heads, int head_dim,
              int block_size) {
        long long rows = 0, b = 0;
        int n = 0;
        for (int i = 0; i < num_seqs; ++i) {
            if (chunk_lens[i] > 0) {
                rows += chunk_lens[i];
                b += ((long long)prefix_lens[i] + chunk_lens[i] + block_size - 1) / block_size;
                ++n;
            }
            if (n == pa::kPrefillMaxSeqs || i == num_seqs - 1) {
                if (n) pre = std::max(pre, pa::prefill_workspace_bytes(n, rows, group, num_kv_heads));
                blocks = std::max(blocks, b);
                rows = b = n = 0;
            }
        }
        pre = round256(pre);
        table = round256((size_t)blocks * (block_size / pa::kExpandRows) * sizeof(int32_t));
        pool = round256((size_t)blocks * num_kv_heads * block_size * head_dim * 2);
    }
    size_t total() const { return pre + table + 2 * pool; }
};

int prefill_lens_ok(const int *prefix_lens, const int *chunk_lens, int num_seqs) {
    long long rows = 0;
    for (int i = 0; i < num_seqs; ++i) {
        if (prefix_lens[i] < 0 || chunk_lens[i] < 0) return PA_ERR_INVALID_ARG;
        if ((long long)prefix_lens[i] + chunk_lens[i] > 0x7fffffffLL) return PA_ERR_OUT_OF_RANGE;
        rows += chunk_lens[i];
    }
    return rows > 0x7fffffffLL ? PA_ERR_OUT_OF_RANGE : PA_OK;
}

}  // namespace

extern "C" {

int pa_norm_rotary_and_cache(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                             const void *key, int64_t key_stride, const void *value, int64_t value_stride, void *k_cache,
                             void *v_cache, const int32_t *positions, const int64_t *slot_mapping, const float *inv_freq,
                             const int *pair_axis, int num_axes, int rot_dim, int interleaved, const void *query_norm,
                             const void *key_norm, float eps, int num_tokens, int num_heads, int num_kv_heads,
                             int head_dim, int block_size, int num_blocks, pa_dtype dtype, int *d_err, void *stream) {
    pa::RotaryParams p{};
    const int rc = rotary_params(p, query_out, query_out_stride, query, query_stride, key, key_stride, value, value_stride,
                                 k_cache, v_cache, positions, slot_mapping, inv_freq, pair_axis, num_axes, rot_dim,
                                 interleaved, query_norm, key_norm, eps, num_tokens, num_heads, num_kv_heads, head_dim,
                                 block_size, num_blocks, dtype, d_err);
    if (rc != PA_OK) return rc;
    if (num_heads == 0) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!query_norm) return PA_ERR_INVALID_ARG;
    return pa::launch_norm_rotary(dtype, p, static_cast<cudaStream_t>(stream));
}

int pa_rotary_and_cache_fp8(void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
                            const void *key, int64_t key_stride, const void *value, int64_t value_stride,
                            uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scales, uint8_t *v_scales,
                            const int32_t *positions, const int64_t *slot_mapping, const float *inv_freq,
                            const int *pair_axis, int num_axes, int rot_dim, int interleaved, const void *query_norm,
                            const void *key_norm, float eps, int num_tokens, int num_heads, int num_kv_heads,
                            int head_dim, int block_size, int num_blocks, pa_dtype dtype, int *d_err, void *stream) {
    pa::RotaryParams p{};
    const int rc = rotary_params(p, query_out, query_out_stride, query, query_stride, key, key_stride, value, value_stride,
                                 k_cache, v_cache, positions, slot_mapping, inv_freq, pair_axis, num_axes, rot_dim,
                                 interleaved, query_norm, key_norm, eps, num_tokens, num_heads, num_kv_heads, head_dim,
                                 block_size, num_blocks, dtype, d_err);
    if (rc != PA_OK) return rc;
    if (num_heads == 0) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    return store_fp8(p, k_scales, v_scales, dtype, stream);
}

int pa_reshape_and_cache_fp8(const void *key, const void *value, uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scales,
                             uint8_t *v_scales, const int64_t *slot_mapping, int num_tokens, int num_kv_heads,
                             int head_dim, int block_size, int num_blocks, pa_dtype dtype, int *d_err, void *stream) {
    pa::RotaryParams p{};
    const int64_t row = num_kv_heads > 0 && head_dim > 0 ? (int64_t)num_kv_heads * head_dim : 0;
    const int rc = rotary_params(p, nullptr, 0, nullptr, 0, key, row, value, row, k_cache, v_cache, nullptr, slot_mapping,
                                 nullptr, nullptr, 1, 0, 0, nullptr, nullptr, 0.f, num_tokens, 0, num_kv_heads, head_dim,
                                 block_size, num_blocks, dtype, d_err);
    if (rc != PA_OK || num_tokens == 0) return rc;
    return store_fp8(p, k_scales, v_scales, dtype, stream);
}

size_t pa_decode_fp8_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                     int max_context_len) {
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        !good_block(block_size) || max_context_len < 0)
        return 0;
    return DecodeWs(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len).total();
}

int pa_decode_fp8(void *out, const void *query, const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_scales,
                  const uint8_t *v_scales, const int32_t *block_tables, int max_blocks_per_seq,
                  const int32_t *context_lens, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                  int num_blocks, int max_context_len, float scale, pa_dtype dtype, void *workspace,
                  size_t workspace_bytes, int *d_err, void *stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PA_ERR_OUT_OF_RANGE;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if ((head_dim != 64 && head_dim != 128) || !good_block(block_size) || !good_group(group)) return PA_ERR_UNSUPPORTED;
    // tokens of a table, rows of a pool (TMA coordinates) and query heads are counted in 32 bits
    if ((long long)max_blocks_per_seq * block_size > 0x7fffff00LL || (long long)num_seqs * num_heads > 0x7fffff00LL ||
        (long long)num_blocks * num_kv_heads > 0x7fffff00LL / block_size)
        return PA_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGNMENT;
    const DecodeWs w(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len);
    if (w.total() > 0) {
        if (!workspace || workspace_bytes < w.total()) return PA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return PA_ERR_ALIGNMENT;
    }
    pa::Fp8DecodeParams p{};
    pa::DecodeParams &d = p.d;
    d.out = out;
    d.query = query;
    d.k_cache = k_cache;
    d.v_cache = v_cache;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.d_err = d_err;
    d.num_seqs = num_seqs;
    d.num_heads = num_heads;
    d.num_kv_heads = num_kv_heads;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.num_blocks = num_blocks;
    d.max_context_len = max_context_len;
    d.block_size = block_size;
    d.scale_log2 = scale * 1.4426950408889634f;
    d.grp_size = 1;
    d.grp_inner = group;
    d.table_stride = max_blocks_per_seq;
    if (w.total() > 0) {
        char *base = static_cast<char *>(workspace);
        p.counters = reinterpret_cast<unsigned *>(base);
        d.ws_acc = reinterpret_cast<float *>(base + w.counters);
        d.ws_ml = reinterpret_cast<float2 *>(base + w.counters + w.acc);
    }
    p.ctas = w.ctas;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    return pa::launch_decode_fp8(dtype, head_dim, group, p, static_cast<cudaStream_t>(stream));
}

size_t pa_prefill_batch_fp8_workspace_bytes(const int *prefix_lens, const int *chunk_lens, int num_seqs, int num_heads,
                                            int num_kv_heads, int head_dim, int block_size) {
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        block_size <= 0 || !prefix_lens || !chunk_lens || prefill_lens_ok(prefix_lens, chunk_lens, num_seqs) != PA_OK)
        return 0;
    return PrefillWs(prefix_lens, chunk_lens, num_seqs, num_heads / num_kv_heads, num_kv_heads, head_dim, block_size).total();
}

int pa_prefill_batch_fp8(void *out, const void *query, const uint8_t *k_cache, const uint8_t *v_cache,
                         const uint8_t *k_scales, const uint8_t *v_scales, const int32_t *block_tables,
                         int max_blocks_per_seq, const int *prefix_lens, const int *chunk_lens, int num_seqs,
                         int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                         pa_dtype dtype, void *workspace, size_t workspace_bytes, int *d_err, void *stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || !good_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_OUT_OF_RANGE;
    if (num_seqs == 0) return PA_OK;
    if (!prefix_lens || !chunk_lens) return PA_ERR_INVALID_ARG;
    if (const int rc = prefill_lens_ok(prefix_lens, chunk_lens, num_seqs)) return rc;
    long long rows = 0;
    for (int i = 0; i < num_seqs; ++i) {
        if ((long long)prefix_lens[i] + chunk_lens[i] > (long long)max_blocks_per_seq * block_size) return PA_ERR_OUT_OF_RANGE;
        rows += chunk_lens[i];
    }
    if (rows == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables) return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (head_dim != 128 || !good_block(block_size) || block_size < 16 || !good_group(group)) return PA_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGNMENT;
    const PrefillWs w(prefix_lens, chunk_lens, num_seqs, group, num_kv_heads, head_dim, block_size);
    // rows of the expanded blocks are 32-bit TMA coordinates
    if (w.blocks * num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < w.total()) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PA_ERR_ALIGNMENT;
    char *base = static_cast<char *>(workspace);
    const size_t counters = pa::prefill_counters_offset();
    pa::Fp8ExpandParams x{};
    x.k_cache = k_cache;
    x.v_cache = v_cache;
    x.k_scales = k_scales;
    x.v_scales = v_scales;
    x.table = reinterpret_cast<int32_t *>(base + w.pre);
    x.k_out = base + w.pre + w.table;
    x.v_out = base + w.pre + w.table + w.pool;
    x.zero = reinterpret_cast<unsigned *>(base + counters);
    x.num_zero = (int)((w.pre - counters) / sizeof(unsigned));
    x.d_err = d_err;
    x.num_kv_heads = num_kv_heads;
    x.head_dim = head_dim;
    x.block_size = block_size;
    x.num_blocks = num_blocks;
    pa::PrefillParams p{};
    p.out = out;
    p.query = query;
    p.k_cache = x.k_out;
    p.v_cache = x.v_out;
    p.d_err = d_err;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.query_rows = (int)rows;
    p.v_scales = v_scales;
    p.tables = block_tables;
    p.table_stride = max_blocks_per_seq;
    p.pool_blocks = num_blocks;
    p.block_shift = __builtin_ctz(block_size);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int parts = block_size / pa::kExpandRows;
    int row = 0;
    for (int i = 0; i < num_seqs; ++i) {
        if (chunk_lens[i] > 0) {
            const int n = p.num_seqs++;
            x.tables[n] = block_tables + (size_t)i * max_blocks_per_seq;
            x.first[n + 1] = x.first[n] + (prefix_lens[i] + chunk_lens[i] - 1) / block_size + 1;
            pa::PrefillSeq &q = p.seqs[n];
            q.block_table = x.table + (size_t)x.first[n] * parts;
            q.prefix_len = prefix_lens[i];
            q.chunk_len = chunk_lens[i];
            q.row_start = row;
            q.table_row = i;
        }
        row += chunk_lens[i];
        if (p.num_seqs == pa::kPrefillMaxSeqs || (i == num_seqs - 1 && p.num_seqs > 0)) {
            x.num_seqs = p.num_seqs;
            p.num_blocks = x.first[p.num_seqs] * parts;
            int rc = pa::launch_expand_fp8(dtype, x, st);
            if (rc == PA_OK) rc = pa::launch_prefill(dtype, head_dim, pa::kExpandRows, group, p, workspace, w.pre, st, true);
            if (rc != PA_OK) return rc;
            p.num_seqs = 0;
        }
    }
    return PA_OK;
}

int pa_copy_blocks_fp8(uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scales, uint8_t *v_scales, const int64_t *pairs,
                       int num_pairs, int num_kv_heads, int head_dim, int block_size, int num_blocks, void *workspace,
                       size_t workspace_bytes, int *d_err, void *stream) {
    if (num_pairs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
    if (num_pairs > PA_COPY_MAX_PAIRS) return PA_ERR_OUT_OF_RANGE;
    if (num_pairs == 0) return PA_OK;
    if (!k_cache || !v_cache || !k_scales || !v_scales || !pairs) return PA_ERR_INVALID_ARG;
    const long long bytes = (long long)num_kv_heads * block_size * head_dim;
    if (bytes % 16) return PA_ERR_UNSUPPORTED;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < pa::copy_blocks_workspace_bytes(num_pairs)) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_ALIGNMENT;
    return pa::launch_copy_blocks(k_cache, v_cache, pairs, num_pairs, bytes, k_scales, v_scales, num_kv_heads, num_blocks,
                                  workspace, d_err, static_cast<cudaStream_t>(stream));
}

// One call with its arguments in an array, in the order of its prototype: pointers and
// integers as 64-bit integers, floats as doubles, host arrays behind the arguments.
int pa_call_packed(int call, const int64_t *a) {
    // the arguments that are ints (bit i: argument i), of each call
    static constexpr uint32_t kInts[] = {0x07f1c000u, 0x1fc70000u, 0x00001f80u, 0x0002fe80u, 0x0002fc80u, 0x000003e0u};
    if (!a || call < 0 || call > PA_CALL_COPY_BLOCKS_FP8) return PA_ERR_INVALID_ARG;
    for (uint32_t left = kInts[call]; left; left &= left - 1) {
        const int64_t v = a[__builtin_ctz(left)];
        if (v != (int32_t)v) return PA_ERR_OUT_OF_RANGE;
    }
    const auto I = [a](int k) { return (int)a[k]; };
    const auto F = [a](int k) {
        double d;
        memcpy(&d, a + k, sizeof d);
        return (float)d;
    };
    const auto P = [a](int k) { return reinterpret_cast<void *>(a[k]); };
    const auto U8 = [a](int k) { return reinterpret_cast<uint8_t *>(a[k]); };
    const auto I32 = [a](int k) { return reinterpret_cast<int32_t *>(a[k]); };
    const auto H32 = [a](int k) {  // host integers, maybe behind the arguments
        const char *tail = reinterpret_cast<const char *>(a);
        return a[k] < 0 ? reinterpret_cast<const int *>(tail - a[k]) : reinterpret_cast<const int *>(a[k]);
    };
    const auto I64 = [a](int k) { return reinterpret_cast<int64_t *>(a[k]); };
    const auto F32 = [a](int k) { return reinterpret_cast<float *>(a[k]); };
    switch (call) {
        case PA_CALL_NORM_ROTARY_AND_CACHE:
            return pa_norm_rotary_and_cache(P(0), a[1], P(2), a[3], P(4), a[5], P(6), a[7], P(8), P(9), I32(10), I64(11),
                                            F32(12), H32(13), I(14), I(15), I(16), P(17), P(18), F(19), I(20), I(21), I(22),
                                            I(23), I(24), I(25), (pa_dtype)I(26), I32(27), P(28));
        case PA_CALL_ROTARY_AND_CACHE_FP8:
            return pa_rotary_and_cache_fp8(P(0), a[1], P(2), a[3], P(4), a[5], P(6), a[7], U8(8), U8(9), U8(10), U8(11),
                                           I32(12), I64(13), F32(14), H32(15), I(16), I(17), I(18), P(19), P(20), F(21),
                                           I(22), I(23), I(24), I(25), I(26), I(27), (pa_dtype)I(28), I32(29), P(30));
        case PA_CALL_RESHAPE_AND_CACHE_FP8:
            return pa_reshape_and_cache_fp8(P(0), P(1), U8(2), U8(3), U8(4), U8(5), I64(6), I(7), I(8), I(9), I(10), I(11),
                                            (pa_dtype)I(12), I32(13), P(14));
        case PA_CALL_DECODE_FP8:
            return pa_decode_fp8(P(0), P(1), U8(2), U8(3), U8(4), U8(5), I32(6), I(7), I32(8), I(9), I(10), I(11), I(12),
                                 I(13), I(14), I(15), F(16), (pa_dtype)I(17), P(18), (size_t)a[19], I32(20), P(21));
        case PA_CALL_PREFILL_BATCH_FP8:
            return pa_prefill_batch_fp8(P(0), P(1), U8(2), U8(3), U8(4), U8(5), I32(6), I(7), H32(8), H32(9), I(10), I(11),
                                        I(12), I(13), I(14), I(15), F(16), (pa_dtype)I(17), P(18), (size_t)a[19], I32(20),
                                        P(21));
        case PA_CALL_COPY_BLOCKS_FP8:
            return pa_copy_blocks_fp8(U8(0), U8(1), U8(2), U8(3), I64(4), I(5), I(6), I(7), I(8), I(9), P(10), (size_t)a[11],
                                      I32(12), P(13));
        default: return PA_ERR_INVALID_ARG;
    }
}

}  // extern "C"

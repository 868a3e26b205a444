// Accumulated attention weights: what follows the decode kernels that keep
// their scores (pa_decode_weights).
//
// A softmax weight is known only once the sequence's maximum and sum are, and
// those only once all its partitions are done.  Reading K a second time to
// recompute the scores would cost half of the decode's traffic again; keeping
// the fp32 scores costs 8 bytes (one write, one read) per (token, query head)
// against 4 D bytes of K and V per (token, kv head): 1.6% of it at one query
// head per kv head and head_dim 128, 12.5% at eight.
//
// Measured: 256 sequences of up to 4096 tokens, 32/8 heads, bf16, 358 us, 6.1 TB/s
// of what the call cannot do without (91% of the copy rate), 326 of them the
// decode kernel with its score stores, 23 this one; 8 of 16384 to 65536, 64/8
// heads, 285 us (88%), 256 and 27.  Finishing a sequence in the decode kernel, by
// its last unit to arrive, took as long: the units that do it are missing from
// the K/V stream.
//
// Where every sequence is a single unit the decode kernel adds the weights up
// itself, from scores it has just written (one launch less: 2 us of a short
// batch's 12).  Otherwise one kernel, two kinds of CTA (and, for positions that
// might be attended together (pa_window.cu), one that looks at their table rows):
//   merge    the log-sum-exp merge of a split sequence's partials, a warp (a CTA,
//            with many partials) per (sequence, head): out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p;
//   totals   one CTA per (row of totals, kv head, chunk of tokens): each
//            token's weight is sum_h 2^(score_h - M_h) / l_h over the group's
//            heads, added up over the row's sequences in their order (so the
//            result does not depend on scheduling) and then to its total.
#include <algorithm>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kMembers = 16;  // sequences of a row taken together

// the decode kernels' clamping of a sequence's length
__device__ __forceinline__ int clamped_len(const DecodeParams &p, int s) {
    const int cap = (int)min((long long)p.max_context_len, (long long)p.max_blocks_per_seq * p.block_size);
    return max(0, min(p.context_lens[s], cap));
}

// Partials from which a row is merged by a whole CTA: a warp takes some 0.15 us a
// partial (246 of them, three sequences of 65536 tokens: 43 us by a warp each,
// 19 by a CTA).
constexpr int kWideMerge = 17;

// One (sequence, head) by one warp (kParts 1), or by a CTA of kParts warps, each
// with every kParts-th partial, their sums added in the warps' order.
template <typename T, int D, int kParts>
__device__ __forceinline__ void merge_row(const DecodeParams &p, int pair, int lane, int part) {
    constexpr int VPL = D / 32;  // values per lane
    const int s = pair / p.num_heads;
    const int L = clamped_len(p, s);
    const int nparts = (L + p.partition_tokens - 1) / p.partition_tokens;
    if (nparts <= 1) return;  // the decode kernel wrote the output
    const size_t base = (size_t)pair * p.slots;
    float M = -INFINITY;
    for (int i = lane; i < nparts; i += 32) M = fmaxf(M, p.ws_ml[base + i].x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, m));
    float lsum = 0.f, o[VPL];
#pragma unroll
    for (int d = 0; d < VPL; ++d) o[d] = 0.f;
    if (M != -INFINITY) {  // else every key was left out: zeros
#pragma unroll 4
        for (int i = part; i < nparts; i += kParts) {
            const float2 ml = p.ws_ml[base + i];
            const float w = fast_exp2(ml.x - M);
            lsum = fmaf(w, ml.y, lsum);
            const float *a = p.ws_acc + (base + i) * D + lane * VPL;
            if constexpr (VPL == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(a);
                o[0] = fmaf(w, x.x, o[0]); o[1] = fmaf(w, x.y, o[1]);
                o[2] = fmaf(w, x.z, o[2]); o[3] = fmaf(w, x.w, o[3]);
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(a);
                o[0] = fmaf(w, x.x, o[0]); o[1] = fmaf(w, x.y, o[1]);
            }
        }
    }
    if constexpr (kParts > 1) {
        __shared__ float s_o[kParts][D];
        __shared__ float s_l[kParts];
#pragma unroll
        for (int d = 0; d < VPL; ++d) s_o[part][lane * VPL + d] = o[d];
        if (lane == 0) s_l[part] = lsum;
        __syncthreads();
        if (part) return;
#pragma unroll
        for (int q = 1; q < kParts; ++q) {
#pragma unroll
            for (int d = 0; d < VPL; ++d) o[d] += s_o[q][lane * VPL + d];
            lsum += s_l[q];
        }
    }
    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
    T *orow = static_cast<T *>(p.out) + (size_t)pair * D + lane * VPL;
    if constexpr (VPL == 4) {
        uint2 u;
        u.x = Elem<T>::pack2(o[0] * inv, o[1] * inv);
        u.y = Elem<T>::pack2(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2 *>(orow) = u;
    } else {
        *reinterpret_cast<uint32_t *>(orow) = Elem<T>::pack2(o[0] * inv, o[1] * inv);
    }
}

// kItems tokens per thread: 2 (8 or 4 at a time measured 33 against 23 us over 256
// sequences of up to 4096 tokens), or 1 when the rows are too few to fill the GPU.
// kMany: several sequences add to a row.
template <typename T, int D, int G, int kItems, bool kMany>
__global__ void __launch_bounds__(kThreads)
    weights_merge_kernel(const __grid_constant__ DecodeParams p, const float *weights, float *weights_out, int width,
                         int queries_per_row, int loops, int chunks, int merge_ctas, int total_ctas) {
    __shared__ float2 s_ml[(kMany ? kMembers : 1) * G];  // (maximum, 1 / sum) per sequence and head
    __shared__ int s_len[kMany ? kMembers : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();  // the decode kernel's scores and partials are complete and visible
    pdl_trigger();
    if ((int)blockIdx.x < merge_ctas) {
        if (p.slots >= kWideMerge) {
            merge_row<T, D, kThreads / 32>(p, blockIdx.x, lane, warp);
        } else {
            const int pair = blockIdx.x * (kThreads / 32) + warp;
            if (pair < p.num_seqs * p.num_heads) merge_row<T, D, 1>(p, pair, lane, 0);
        }
        return;
    }
    const int u = blockIdx.x - merge_ctas;
    if (kMany && u >= total_ctas) {  // a sequence's table row against its row's first one's
        const int s = u - total_ctas;
        const int32_t *row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const int32_t *lead = p.block_tables + (size_t)(s - s % queries_per_row) * p.max_blocks_per_seq;
        bool same = true;
        for (int j = tid; j < (clamped_len(p, s) + p.block_size - 1) / p.block_size; j += kThreads) same = same && row[j] == lead[j];
        if (!same) flag_error(p.d_err, PA_DEVERR_PREFIX);
        return;
    }
    const int chunk = u % chunks, rh = u / chunks;
    const int r = rh / p.num_kv_heads, kvh = rh - r * p.num_kv_heads;
    const int j0 = chunk * loops * kThreads * kItems + tid;  // this thread's first tokens: j0 + i * kThreads
    const int s0 = r * queries_per_row;
    float acc[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) acc[i] = 0.f;
    auto load = [&](int s, int L, float (&x)[kItems][G]) {
        const float *sc = p.scores + ((size_t)(s * p.num_kv_heads + kvh) * p.score_stride + j0) * G;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (j0 + i * kThreads < L) {
                load_scores<G>(sc + (size_t)i * kThreads * G, x[i]);
            } else {
#pragma unroll
                for (int h = 0; h < G; ++h) x[i][h] = -INFINITY;
            }
        }
    };
    // (maximum, 1 / sum) of a sequence's head over its partitions, by a warp
    auto max_sum = [&](int s, int h, int L) {
        const int nparts = (L + p.partition_tokens - 1) / p.partition_tokens;
        const float2 *ml = p.ws_ml + ((size_t)s * p.num_heads + kvh * G + h) * p.slots;
        const float2 mine = lane < nparts ? ml[lane] : make_float2(-INFINITY, 0.f);
        float M = mine.x;
        for (int i = lane + 32; i < nparts; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, k));
        if (M == -INFINITY) return make_float2(0.f, 0.f);  // no key attended: 2^(-inf - 0) = 0 for every one of them
        float sum = fast_exp2(mine.x - M) * mine.y;
        for (int i = lane + 32; i < nparts; i += 32) sum = fmaf(fast_exp2(ml[i].x - M), ml[i].y, sum);
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(kFull, sum, k);
        return make_float2(M, 1.f / sum);
    };
    const size_t at = (size_t)rh * width + j0;
    if constexpr (!kMany) {
        // Everything that does not depend on the maxima and sums is under way
        // while they are put together, and the next tokens' while these are
        // summed.
        const int L = clamped_len(p, s0);
        if (j0 - tid >= L) return;
        const float *sc = p.scores + ((size_t)rh * p.score_stride + j0) * G;
        float x[kItems][G], w[kItems];
        load(s0, L, x);
#pragma unroll
        for (int i = 0; i < kItems; ++i) w[i] = j0 + i * kThreads < L ? weights[at + i * kThreads] : 0.f;
        if (warp < G) {
            const float2 ml = max_sum(s0, warp, L);
            if (lane == 0) s_ml[warp] = ml;
        }
        __syncthreads();
        constexpr int kStep = kThreads * kItems;
        for (int it = 0; it < loops; ++it) {
            const int j = j0 + it * kStep, next = j + kStep;
            float y[kItems][G], v[kItems];
            const bool more = it + 1 < loops && next - tid < L;
            if (more) {
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    v[i] = 0.f;
#pragma unroll
                    for (int h = 0; h < G; ++h) y[i][h] = -INFINITY;
                    if (next + i * kThreads < L) {
                        load_scores<G>(sc + (size_t)((it + 1) * kStep + i * kThreads) * G, y[i]);
                        v[i] = weights[at + (it + 1) * kStep + i * kThreads];
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float2 ml = s_ml[h];
#pragma unroll
                for (int i = 0; i < kItems; ++i) acc[i] = fmaf(fast_exp2(x[i][h] - ml.x), ml.y, h ? acc[i] : 0.f);
            }
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (j + i * kThreads < L) weights_out[at + it * kStep + i * kThreads] = w[i] + acc[i];
            if (!more) break;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                w[i] = v[i];
#pragma unroll
                for (int h = 0; h < G; ++h) x[i][h] = y[i][h];
            }
        }
    } else {
        int longest = 0;
        for (int m0 = 0; m0 < queries_per_row; m0 += kMembers) {
            const int nm = min(kMembers, queries_per_row - m0);
            float x[kItems][G];
            load(s0 + m0, clamped_len(p, s0 + m0), x);
            if (m0) __syncthreads();  // the previous sequences' values are read
            for (int mh = warp; mh < nm * G; mh += kThreads / 32) {
                const int s = s0 + m0 + mh / G, h = mh % G;
                const int L = clamped_len(p, s);
                const float2 ml = max_sum(s, h, L);
                if (lane == 0) {
                    s_ml[mh] = ml;
                    if (h == 0) s_len[mh / G] = L;
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int m = 0; m < nm; ++m) {
                longest = max(longest, s_len[m]);
                float y[kItems][G];
                const bool more = m + 1 < nm;
                if (more) load(s0 + m0 + m + 1, s_len[m + 1], y);
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float2 ml = s_ml[m * G + h];
#pragma unroll
                    for (int i = 0; i < kItems; ++i) acc[i] = fmaf(fast_exp2(x[i][h] - ml.x), ml.y, acc[i]);
                }
                if (more) {
#pragma unroll
                    for (int i = 0; i < kItems; ++i)
#pragma unroll
                        for (int h = 0; h < G; ++h) x[i][h] = y[i][h];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i)
            if (j0 + i * kThreads < longest) weights_out[at + i * kThreads] = weights[at + i * kThreads] + acc[i];
    }
}

template <typename T, int D, int G>
int launch_merge_t(const DecodeParams &p, const float *weights, float *weights_out, int width, int queries_per_row,
                   bool one_table, cudaStream_t stream) {
    const long long rows = (long long)(p.num_seqs / queries_per_row) * p.num_kv_heads;
    constexpr int kMost = 2;
    const bool few = rows * ((p.max_context_len + kMost * kThreads - 1) / (kMost * kThreads)) < 2 * sm_count();
    const int chunk = few ? kThreads : kMost * kThreads;
    int chunks = std::max(1, (p.max_context_len + chunk - 1) / chunk);
    // with many chunks a CTA takes several of a row's, the next one's loads ahead
    // (8 or 12 CTAs an SM measured best at 8 and at 4 heads)
    constexpr int kPerSm = G == 8 ? 8 : 12;
    const long long share = std::max(1LL, rows * chunks / (kPerSm * sm_count()));
    const int loops = queries_per_row > 1 ? 1 : (int)std::min<long long>(share, std::min(chunks, G == 8 ? 8 : 16));
    chunks = (chunks + loops - 1) / loops;
    const long long pairs = (long long)p.num_seqs * p.num_heads;
    const int per_cta = p.slots >= kWideMerge ? 1 : kThreads / 32;
    const long long merge = p.max_partitions > 1 ? (pairs + per_cta - 1) / per_cta : 0;
    const long long total = merge + rows * chunks + (one_table ? p.num_seqs : 0);
    if (total > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    auto kern = queries_per_row > 1
                    ? (few ? weights_merge_kernel<T, D, G, 1, true> : weights_merge_kernel<T, D, G, kMost, true>)
                    : (few ? weights_merge_kernel<T, D, G, 1, false> : weights_merge_kernel<T, D, G, kMost, false>);
    return launch_pdl(kern, dim3((unsigned)total), dim3(kThreads), 0, stream, p, weights,
                      weights_out, width, queries_per_row, loops, chunks, (int)merge, (int)(rows * chunks)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <typename T>
int launch_merge_dtype(int head_dim, int group, const DecodeParams &p, const float *weights, float *weights_out,
                       int width, int queries_per_row, bool one_table, cudaStream_t stream) {
#define PA_MERGE_CASE(DD, GG)                \
    if (head_dim == DD && group == GG)       \
        return launch_merge_t<T, DD, GG>(p, weights, weights_out, width, queries_per_row, one_table, stream);
    PA_MERGE_CASE(64, 1) PA_MERGE_CASE(64, 2) PA_MERGE_CASE(64, 4) PA_MERGE_CASE(64, 8)
    PA_MERGE_CASE(128, 1) PA_MERGE_CASE(128, 2) PA_MERGE_CASE(128, 4) PA_MERGE_CASE(128, 8)
#undef PA_MERGE_CASE
    return PA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_decode_scores(pa_dtype dt, int head_dim, int block_size, int group, const DecodeParams &p,
                         cudaStream_t stream) {
    const int rc = launch_decode_tc_scores(dt, head_dim, block_size, group, p, stream);
    if (rc != PA_ERR_UNSUPPORTED) return rc;
    return dt == PA_BF16 ? launch_decode_scores_bf16(head_dim, block_size, group, p, stream)
                         : launch_decode_scores_f16(head_dim, block_size, group, p, stream);
}

// Groups of 8 (the tensor-core decode): a unit costs some 5 us apart from its
// tokens (its set-up, its partial and that one's merge), a token 24 ns of a CTA's
// share of HBM, and on average half a unit per CTA slot is lost to the last
// round; with N tokens a slot the sum N / pt * 5 us + pt / 2 * 24 ns is least at
// pt = sqrt(417 N).  Lengths are on the device: three quarters of the longest
// each.  One sequence of 62000 tokens, 64/8 heads: 54 us at 512 (48 at 1024) against
// 60 at pa_decode's 256; three of 16384 to 65536 116 (1024) against 134; eight 285
// (2048) against 288 (1024).  Smaller groups keep pa_decode's choice (within 10% of the
// best everywhere it was tried).
int weights_partition_tokens(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                             int max_context_len) {
    if (head_dim != 128 || !decode_tc_group(num_heads / num_kv_heads))
        return auto_partition_tokens(num_seqs, num_heads, num_kv_heads, block_size, max_context_len);
    const double per_slot = 0.75 * num_seqs * max_context_len * num_kv_heads / (2.0 * sm_count());
    const double best = std::sqrt(417.0 * per_slot);
    int pt = 256;  // a multiple of every block size
    while (pt < 4096 && best > pt * 1.41421356) pt *= 2;
    return pt;
}

int launch_weights_merge(pa_dtype dt, int head_dim, int group, const DecodeParams &p, const float *weights,
                         float *weights_out, int width, int queries_per_row, bool one_table, cudaStream_t stream) {
    return dt == PA_BF16 ? launch_merge_dtype<__nv_bfloat16>(head_dim, group, p, weights, weights_out, width,
                                                             queries_per_row, one_table, stream)
                         : launch_merge_dtype<__half>(head_dim, group, p, weights, weights_out, width, queries_per_row,
                                                      one_table, stream);
}

}  // namespace pa

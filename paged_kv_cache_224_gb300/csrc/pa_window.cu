// pa_decode_weights for several query positions over one cache: the schedule of
// the tensor-core pass (pa_window.cuh), and what follows it.
//
// One kernel follows, with three kinds of CTA:
//   merge    one warp per (sequence, head): the log-sum-exp merge of its pieces,
//            and rows that a NaN or infinity behind their mask reached anew;
//   totals   one CTA per (row of totals, kv head, 128 tokens): a token's weight
//            is sum_r 2^(score_r - M_r) / l_r over the row's query rows
//            (positions x heads) that see it.  A warp takes 32 tokens, a lane
//            every 32nd query row: its loads are lines of 32 rows' scores of a
//            key, and the lanes' sums for 32 tokens change places in 31
//            shuffles, in a fixed order;
//   check    one CTA per sequence: its length, and that its table row is the
//            one its row of totals is attended over.
#include <algorithm>

#include "pa_window.cuh"

namespace pa {
namespace {
using namespace wnd;

constexpr int kTotThreads = 128;  // tokens of a totals CTA, 32 to a warp
constexpr int kBatch = 128;       // query rows whose maxima and sums are held at a time

struct WindowSchedule {
    long long tiles;
    int row_tiles, n, ctas;
};
WindowSchedule window_schedule(int rows, int queries_per_row, int group, int num_kv_heads, int max_context_len) {
    WindowSchedule s;
    s.row_tiles = (int)(((long long)queries_per_row * group + kUnitRows - 1) / kUnitRows);
    s.n = std::max(1, (int)(((long long)max_context_len + kNK - 1) / kNK));
    s.tiles = (long long)rows * num_kv_heads * s.row_tiles * s.n;
    s.ctas = (int)std::min<long long>(sm_count(), s.tiles);
    return s;
}

struct MergeParams {
    int queries_per_row, head_group, row_tiles, n;
    int full_tiles, full_ctas;              // of a launch of kPrefillMaxSeqs rows
    int last_first, last_tiles, last_ctas;  // the last launch: its first row, tiles and CTAs
    const float *weights;
    float *weights_out;
    int width, chunks, merge_ctas, total_ctas;
};

// Pieces of the unit of query row (row i of totals, kv head, row gr of positions x heads).
__device__ __forceinline__ int pieces_of(const DecodeParams &p, const MergeParams &mp, int i, int kvh, int gr) {
    const bool last = i >= mp.last_first;
    const int il = last ? i - mp.last_first : i % kPrefillMaxSeqs;
    const long long W = last ? mp.last_tiles : mp.full_tiles, N = last ? mp.last_ctas : mp.full_ctas;
    const int x = ((il * p.num_kv_heads + kvh) * mp.row_tiles + gr / kUnitRows) * mp.n;
    return cta_of(x + mp.n - 1, W, N) - cta_of(x, W, N) + 1;
}

__device__ __forceinline__ int clamped_len(const DecodeParams &p, int s) {
    return max(0, min(p.context_lens[s], (int)min((long long)p.max_context_len,
                                                  (long long)p.max_blocks_per_seq * p.block_size)));
}

template <typename T>
__global__ void __launch_bounds__(kTotThreads)
    window_merge_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ MergeParams mp) {
    __shared__ float2 s_ml[kBatch];  // (maximum, 1 / sum) of a query row
    __shared__ int s_len[kBatch];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = mp.head_group, w = mp.queries_per_row;
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x < mp.total_ctas) {
        // ---------------------------------------------------------------- totals
        const int chunk = blockIdx.x % mp.chunks, rh = blockIdx.x / mp.chunks;
        const int i = rh / p.num_kv_heads, kvh = rh - i * p.num_kv_heads;
        const int j0 = chunk * kTotThreads + warp * 32;  // the warp's first token
        const int rows = w * G, planes = (rows + 31) / 32;
        const int j = j0 + lane;
        const size_t at = (size_t)rh * mp.width + j;
        const float was = j < p.max_context_len ? mp.weights[at] : 0.f;
        float sum[32];  // per token, over this lane's query rows
#pragma unroll
        for (int k = 0; k < 32; ++k) sum[k] = 0.f;
        int longest = 0;
        for (int r0 = 0; r0 < rows; r0 += kBatch) {
            const int nr = min(kBatch, rows - r0);
            // the first 32 rows' scores (inside the tile-rounded buffer whatever the lengths are)
            const float *sc = p.scores + (((size_t)rh * planes + r0 / 32) * p.score_stride + j0) * 32 + lane;
            float x[32];
            auto fetch = [&](int b) {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = b * 32 + lane < nr ? __ldcs(sc + (size_t)b * p.score_stride * 32 + k * 32) : 0.f;
            };
            fetch(0);
            if (r0) __syncthreads();  // the previous rows' values are read
            if (tid < nr) {
                const int gr = r0 + tid, s = i * w + gr / G;
                const float2 *ml = p.ws_ml + ((size_t)s * p.num_heads + kvh * G + gr % G) * p.slots;
                const int np = pieces_of(p, mp, i, kvh, gr);
                const int L = clamped_len(p, s);
                float M = -INFINITY, l = 0.f;
#pragma unroll 8
                for (int k = 0; k < np; ++k) M = fmaxf(M, ml[k].x);
                if (M != -INFINITY) {
#pragma unroll 8
                    for (int k = 0; k < np; ++k) l = fmaf(fast_exp2(ml[k].x - M), ml[k].y, l);
                }
                // no key attended: 2^(-inf) = 0 for every one of them
                s_ml[tid] = M == -INFINITY ? make_float2(0.f, 0.f) : make_float2(M, 1.f / l);
                s_len[tid] = L;
            }
            __syncthreads();
            for (int b = 0; b * 32 < nr; ++b) {
                if (b) fetch(b);
                const int r = b * 32 + lane;
                const float2 ml = r < nr ? s_ml[r] : make_float2(0.f, 0.f);
                const int left = (r < nr ? s_len[r] : 0) - j0;  // of the warp's tokens, those this row sees
                longest = max(longest, left);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (k < left) sum[k] = fmaf(fast_exp2(fmaf(x[k], p.scale_log2, -ml.x)), ml.y, sum[k]);
            }
        }
        // the lanes' 32 sums: halves change places until lane k holds token k's
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            const bool up = lane & m;
#pragma unroll
            for (int k = 0; k < m; ++k) {
                const float keep = up ? sum[k + m] : sum[k], send = up ? sum[k] : sum[k + m];
                sum[k] = keep + __shfl_xor_sync(kFull, send, m);
            }
        }
        longest = __reduce_max_sync(kFull, longest);
        if (lane < longest) mp.weights_out[at] = was + sum[0];
        return;
    }
    const int b = blockIdx.x - mp.total_ctas;
    if (b >= mp.merge_ctas) {
        // ---------------------------------------------------------------- check
        const int s = b - mp.merge_ctas;
        const int L = clamped_len(p, s);
        if (tid == 0 && L != p.context_lens[s]) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
        const int32_t *row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const int32_t *lead = p.block_tables + (size_t)(s - s % w) * p.max_blocks_per_seq;
        bool same = true;
        for (int k = tid; k < (L + p.block_size - 1) / p.block_size; k += kTotThreads) same = same && row[k] == lead[k];
        if (!same) flag_error(p.d_err, PA_DEVERR_PREFIX);
        return;
    }
    // -------------------------------------------------------------------- merge
    constexpr int VPL = kD / 32;  // values per lane
    const int pair = b * (kTotThreads / 32) + warp;
    if (pair >= p.num_seqs * p.num_heads) return;
    const int s = pair / p.num_heads, hq = pair - s * p.num_heads;
    const int np = pieces_of(p, mp, s / w, hq / G, s % w * G + hq % G);
    const size_t base = (size_t)pair * p.slots;
    float M = -INFINITY;
    for (int k = lane; k < np; k += 32) M = fmaxf(M, p.ws_ml[base + k].x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, m));
    float lsum = 0.f, o[VPL];
#pragma unroll
    for (int d = 0; d < VPL; ++d) o[d] = 0.f;
#pragma unroll 4
    for (int k = 0; k < np; ++k) {
        const float2 ml = p.ws_ml[base + k];
        if (ml.x == -INFINITY) continue;  // an empty piece has no accumulator
        const float e = fast_exp2(ml.x - M);
        lsum = fmaf(e, ml.y, lsum);
        const float4 x = *reinterpret_cast<const float4 *>(p.ws_acc + (base + k) * kD + lane * VPL);
        o[0] = fmaf(e, x.x, o[0]); o[1] = fmaf(e, x.y, o[1]);
        o[2] = fmaf(e, x.z, o[2]); o[3] = fmaf(e, x.w, o[3]);
    }
    // In the MMAs every row meets every key, with weight 0 where it does not see
    // it, and 0 * NaN or infinity is NaN: a row that is not finite is added up
    // again from its kept scores, over its own keys alone.
    if (M != -INFINITY && __any_sync(kFull, !(isfinite(o[0]) && isfinite(o[1]) && isfinite(o[2]) && isfinite(o[3])))) {
#pragma unroll
        for (int d = 0; d < VPL; ++d) o[d] = 0.f;
        const int kvh = hq / G, gr = s % w * G + hq % G, bs = p.block_size;
        const int L = clamped_len(p, s);
        const int32_t *table = p.block_tables + (size_t)(s - s % w) * p.max_blocks_per_seq;
        const float *sc = p.scores + (((size_t)(s / w * p.num_kv_heads + kvh) * ((w * G + 31) / 32) + gr / 32) * p.score_stride) * 32 +
                          gr % 32;
#pragma unroll 8
        for (int j = 0; j < L; ++j) {
            const int b = table[j / bs];
            if (b < 0 || b >= p.num_blocks) continue;
            const float e = fast_exp2(fmaf(sc[(size_t)j * 32], p.scale_log2, -M));
            float v[VPL];
            const uint2 raw = *reinterpret_cast<const uint2 *>(
                static_cast<const T *>(p.v_cache) + (((size_t)b * p.num_kv_heads + kvh) * bs + j % bs) * kD + lane * VPL);
            Elem<T>::unpack2(raw.x, v[0], v[1]);
            Elem<T>::unpack2(raw.y, v[2], v[3]);
#pragma unroll
            for (int d = 0; d < VPL; ++d) o[d] = fmaf(e, v[d], o[d]);
        }
    }
    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
    uint2 u;
    u.x = Elem<T>::pack2(o[0] * inv, o[1] * inv);
    u.y = Elem<T>::pack2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (size_t)pair * kD + lane * VPL) = u;
}

}  // namespace

bool window_supported(int head_dim, int block_size, int group, int queries_per_row) {
    return head_dim == kD && block_size >= 16 && queries_per_row >= 4 && (long long)queries_per_row * group >= 16;
}

// Whether a supported window is attended together.  One position after the other
// reads the cache once each (from L2, mostly, after the first); together a unit has
// the set-up and the tiles of 128 keys of the prefill's CTA.  Measured on a GB300, 8
// kv heads, bf16, caches of half to all of L tokens, together / apart in us, by the
// number of caches (1, 16, 256):
//   8 heads a kv head, tensor-core decode:
//     4 positions  L 256: 13/12  24/24  339/229    8192: 26/25  203/163  2987/2388
//     8 positions  L 256: 14/17  28/41  414/455    8192: 27/39  235/287  (64: 890/1137)
//   4 heads:
//     4 positions  L 512: 12/11  31/25  452/244    2048: 15/15  72/76  987/859    8192: 25/30  201/237  2946/3231
//     8 positions  L 64: 13/10  17/19  220/161     512: 13/14  33/45  488/486     8192: 26/52  204/437  3002/6335
//     16 positions L 64: 14/15  20/33  284/330     8192: 28/94  237/836
//   2 heads:
//     8 positions  L 512: 12/11  31/35  452/353    1024: 14/13  45/64  636/646    8192: 25/40  200/313  2935/4607
//   1 head:
//     16 positions L 64: 13/11  16/22  198/219     8192: 25/59  200/477  2931/7377
bool window_preferred(int group, int queries_per_row, int max_context_len) {
    if (group == 8) return queries_per_row >= 8;
    return queries_per_row >= 16 || max_context_len >= (queries_per_row >= 8 ? 2048 / group : 4096);
}

int window_pieces(int rows, int queries_per_row, int group, int num_kv_heads, int max_context_len) {
    // a unit's first and last pieces, and whole ranges of at least q tiles between them
    auto most = [&](int r) {
        const WindowSchedule s = window_schedule(r, queries_per_row, group, num_kv_heads, max_context_len);
        return s.n > 1 ? (int)std::min<long long>(s.ctas, 2 + (s.n - 2) / (s.tiles / s.ctas)) : 1;
    };
    const int last = most((rows - 1) % kPrefillMaxSeqs + 1);
    return rows > kPrefillMaxSeqs ? std::max(last, most(kPrefillMaxSeqs)) : last;
}

int launch_window(pa_dtype dt, int block_size, int group, const DecodeParams &d, int queries_per_row,
                  const float *weights, float *weights_out, int width, cudaStream_t stream) {
    // TMA row coordinates are 32-bit
    if ((long long)d.num_blocks * d.num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    const int rows = d.num_seqs / queries_per_row;
    PrefillParams p{};
    p.query = d.query;
    p.k_cache = d.k_cache;
    p.v_cache = d.v_cache;
    p.d_err = d.d_err;
    p.num_heads = d.num_heads;
    p.num_kv_heads = d.num_kv_heads;
    p.num_blocks = d.num_blocks;
    p.scale_log2 = d.scale_log2;
    p.query_rows = d.num_seqs;
    p.part_o = d.ws_acc;
    p.part_ml = d.ws_ml;
    p.part_slots = d.slots;
    p.context_lens = d.context_lens;
    p.len_cap = (int)std::min<long long>(d.max_context_len, (long long)d.max_blocks_per_seq * d.block_size);
    p.scores = d.scores;
    p.score_stride = d.score_stride;
    for (int i0 = 0; i0 < rows; i0 += kPrefillMaxSeqs) {
        p.num_seqs = std::min(kPrefillMaxSeqs, rows - i0);
        p.row_base = i0;
        for (int i = 0; i < p.num_seqs; ++i) {
            PrefillSeq &q = p.seqs[i];
            q.row_start = (i0 + i) * queries_per_row;
            q.block_table = d.block_tables + (size_t)q.row_start * d.max_blocks_per_seq;
            q.prefix_len = std::max(d.max_context_len, 1) - 1;
            q.chunk_len = queries_per_row;
        }
        long long units = 0;
        int rc = prefill_schedule<true>(p, group, &units);
        if (rc != PA_OK) return rc;
        const WindowSchedule s = window_schedule(p.num_seqs, queries_per_row, group, d.num_kv_heads, d.max_context_len);
        rc = dt == PA_BF16 ? launch_window_bf16(block_size, group, p, (unsigned)s.ctas, stream)
                           : launch_window_f16(block_size, group, p, (unsigned)s.ctas, stream);
        if (rc != PA_OK) return rc;
    }
    MergeParams mp{};
    const int last = (rows - 1) % kPrefillMaxSeqs + 1;
    const WindowSchedule f = window_schedule(kPrefillMaxSeqs, queries_per_row, group, d.num_kv_heads, d.max_context_len);
    const WindowSchedule l = window_schedule(last, queries_per_row, group, d.num_kv_heads, d.max_context_len);
    mp.queries_per_row = queries_per_row;
    mp.head_group = group;
    mp.row_tiles = l.row_tiles;
    mp.n = l.n;
    mp.full_tiles = rows > kPrefillMaxSeqs ? (int)f.tiles : 1;
    mp.full_ctas = rows > kPrefillMaxSeqs ? f.ctas : 1;
    mp.last_first = rows - last;
    mp.last_tiles = (int)l.tiles;
    mp.last_ctas = l.ctas;
    mp.weights = weights;
    mp.weights_out = weights_out;
    mp.width = width;
    mp.chunks = (d.max_context_len + kTotThreads - 1) / kTotThreads;
    const long long totals = (long long)rows * d.num_kv_heads * mp.chunks;
    const long long merge = ((long long)d.num_seqs * d.num_heads + kTotThreads / 32 - 1) / (kTotThreads / 32);
    if (totals + merge + d.num_seqs > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    mp.total_ctas = (int)totals;
    mp.merge_ctas = (int)merge;
    const dim3 grid((unsigned)(totals + merge + d.num_seqs)), block(kTotThreads);
    const cudaError_t e = dt == PA_BF16 ? launch_pdl(window_merge_kernel<__nv_bfloat16>, grid, block, 0, stream, d, mp)
                                        : launch_pdl(window_merge_kernel<__half>, grid, block, 0, stream, d, mp);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

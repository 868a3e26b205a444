// Decode attention for batches that share a long prefix
// (pa_decode_common_prefix): the schedule of the prefix pass (pa_prefix.cuh)
// and the merge of its partials with those of the sequences' own tokens.
//
// With x = the keys of the prefix and of the sequence's own tokens, cut into
// pieces, a piece's partial is (acc, m, l) = (sum 2^(s_j - m) V_j, max s_j,
// sum 2^(s_j - m)), and out = sum 2^(m_i - M) acc_i / sum 2^(m_i - M) l_i over
// all of them, M the largest m_i.
#include <algorithm>

#include "pa_prefix.cuh"

namespace pa {
namespace {
using namespace pfx;

constexpr int kMergeWarps = 4;

// Schedule of one launch of `groups` groups (at most kPrefillMaxSeqs).
struct PrefixSchedule {
    long long tiles;  // key tiles of all units
    int row_tiles;    // units per (group, kv head)
    int n;            // key tiles per unit
    int ctas;
};
PrefixSchedule prefix_schedule(int groups, int group_size, int prefix_tokens, int group, int num_kv_heads) {
    PrefixSchedule s;
    s.row_tiles = (int)(((long long)group_size * group + kUnitRows - 1) / kUnitRows);
    s.n = (prefix_tokens + kNK - 1) / kNK;
    s.tiles = (long long)groups * num_kv_heads * s.row_tiles * s.n;
    s.ctas = (int)std::min<long long>(sm_count(), s.tiles);
    return s;
}

// Where the merge finds a row's prefix partials.
struct MergeParams {
    int group_size, row_tiles, n, head_group;
    int full_tiles, full_ctas;  // of a launch of kPrefillMaxSeqs groups
    int last_first, last_tiles, last_ctas;  // the last launch: its first group, tiles and CTAs
    int prefix_blocks;
};

// CTAs 0 .. merge_ctas-1: one warp per (sequence, head).  The others compare
// a sequence's prefix table entries with its group's first sequence's.
template <typename T>
__global__ void __launch_bounds__(kMergeWarps * 32)
    prefix_merge_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ MergeParams mp, int merge_ctas) {
    constexpr int VPL = kD / 32;  // values per lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= merge_ctas) {
        const int s = blockIdx.x - merge_ctas;
        const int32_t *row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const int32_t *lead = p.block_tables + (size_t)(s - s % mp.group_size) * p.max_blocks_per_seq;
        bool same = true;
        for (int j = threadIdx.x; j < mp.prefix_blocks; j += blockDim.x) same = same && row[j] == lead[j];
        if (!same) flag_error(p.d_err, PA_DEVERR_PREFIX);
        return;
    }
    const int pair = blockIdx.x * kMergeWarps + warp;
    if (pair >= p.num_seqs * p.num_heads) return;
    const int s = pair / p.num_heads, hq = pair - s * p.num_heads;
    const int kvh = hq / mp.head_group;
    const int g = s / mp.group_size, k = s - g * mp.group_size;
    // the unit of this row, and the CTAs its tiles went to
    const bool last = g >= mp.last_first;
    const int gl = last ? g - mp.last_first : g % kPrefillMaxSeqs;
    const long long W = last ? mp.last_tiles : mp.full_tiles, N = last ? mp.last_ctas : mp.full_ctas;
    const int r = (k * mp.head_group + hq % mp.head_group) / kUnitRows;
    const int x = ((gl * p.num_kv_heads + kvh) * mp.row_tiles + r) * mp.n;
    const int pre = cta_of(x + mp.n - 1, W, N) - cta_of(x, W, N) + 1;
    // the sequence's own partitions, clamped like the decode kernels
    const int cap = (int)min((long long)p.max_context_len, (long long)p.max_blocks_per_seq * p.block_size) - p.len_offset;
    const int L = max(0, min(p.context_lens[s] - p.len_offset, cap));
    const int own = (L + p.partition_tokens - 1) / p.partition_tokens;
    const int total = pre + own;
    const size_t base = (size_t)pair * p.slots;
    auto slot = [&](int i) { return base + (i < pre ? i : p.part_base + i - pre); };
    float M = -INFINITY;
    for (int i = lane; i < total; i += 32) M = fmaxf(M, p.ws_ml[slot(i)].x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, m));
    float lsum = 0.f, o[VPL];
#pragma unroll
    for (int d = 0; d < VPL; ++d) o[d] = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
        for (int i = 0; i < total; ++i) {
            const size_t sl = slot(i);
            const float2 ml = p.ws_ml[sl];
            const float w = fast_exp2(ml.x - M);
            lsum = fmaf(w, ml.y, lsum);
            const float4 a = *reinterpret_cast<const float4 *>(p.ws_acc + sl * kD + lane * VPL);
            o[0] = fmaf(w, a.x, o[0]); o[1] = fmaf(w, a.y, o[1]);
            o[2] = fmaf(w, a.z, o[2]); o[3] = fmaf(w, a.w, o[3]);
        }
    }
    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
    uint2 u;
    u.x = Elem<T>::pack2(o[0] * inv, o[1] * inv);
    u.y = Elem<T>::pack2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (size_t)pair * kD + lane * VPL) = u;
}

}  // namespace

int prefix_pieces(int groups, int group_size, int prefix_tokens, int group, int num_kv_heads) {
    int most = 1;
    // the full launches' schedule and the last one's
    for (int g : {std::min(groups, kPrefillMaxSeqs), (groups - 1) % kPrefillMaxSeqs + 1}) {
        const PrefixSchedule s = prefix_schedule(g, group_size, prefix_tokens, group, num_kv_heads);
        // a unit's first and last pieces, and whole ranges of at least q tiles between them
        const long long q = s.tiles / s.ctas;
        if (s.n > 1) most = std::max<int>(most, (int)std::min<long long>(s.ctas, 2 + (s.n - 2) / q));
    }
    return most;
}

int launch_prefix(pa_dtype dt, int block_size, int group, const PrefixParams &pp, float scale_log2,
                  cudaStream_t stream) {
    const DecodeParams &d = pp.d;
    // TMA row coordinates are 32-bit
    if ((long long)d.num_blocks * d.num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    PrefillParams p{};
    p.query = d.query;
    p.k_cache = d.k_cache;
    p.v_cache = d.v_cache;
    p.d_err = d.d_err;
    p.num_heads = d.num_heads;
    p.num_kv_heads = d.num_kv_heads;
    p.num_blocks = d.num_blocks;
    p.scale_log2 = scale_log2;
    p.query_rows = d.num_seqs;
    p.part_o = d.ws_acc;
    p.part_ml = d.ws_ml;
    p.part_slots = d.slots;
    for (int g0 = 0; g0 < pp.groups; g0 += kPrefillMaxSeqs) {
        p.num_seqs = std::min(kPrefillMaxSeqs, pp.groups - g0);
        for (int i = 0; i < p.num_seqs; ++i) {
            PrefillSeq &q = p.seqs[i];
            q.row_start = (g0 + i) * pp.group_size;
            q.block_table = d.block_tables + (size_t)q.row_start * d.max_blocks_per_seq;
            q.prefix_len = pp.prefix_tokens - 1;
            q.chunk_len = pp.group_size;
        }
        long long units = 0;
        int rc = prefill_schedule<true>(p, group, &units);
        if (rc != PA_OK) return rc;
        const PrefixSchedule s = prefix_schedule(p.num_seqs, pp.group_size, pp.prefix_tokens, group, d.num_kv_heads);
        rc = dt == PA_BF16 ? launch_prefix_bf16(block_size, group, p, (unsigned)s.ctas, stream)
                           : launch_prefix_f16(block_size, group, p, (unsigned)s.ctas, stream);
        if (rc != PA_OK) return rc;
    }
    return PA_OK;
}

int launch_prefix_merge(pa_dtype dt, int group, const PrefixParams &pp, cudaStream_t stream) {
    const DecodeParams &d = pp.d;
    MergeParams mp{};
    mp.group_size = pp.group_size;
    mp.head_group = group;
    mp.prefix_blocks = pp.prefix_tokens / d.block_size;
    const int last = (pp.groups - 1) % kPrefillMaxSeqs + 1;
    const PrefixSchedule f = prefix_schedule(kPrefillMaxSeqs, pp.group_size, pp.prefix_tokens, group, d.num_kv_heads);
    const PrefixSchedule l = prefix_schedule(last, pp.group_size, pp.prefix_tokens, group, d.num_kv_heads);
    mp.row_tiles = l.row_tiles;
    mp.n = l.n;
    mp.full_tiles = pp.groups > kPrefillMaxSeqs ? (int)f.tiles : 1;
    mp.full_ctas = pp.groups > kPrefillMaxSeqs ? f.ctas : 1;
    mp.last_first = pp.groups - last;
    mp.last_tiles = (int)l.tiles;
    mp.last_ctas = l.ctas;
    const long long pairs = (long long)d.num_seqs * d.num_heads;
    const long long merge = (pairs + kMergeWarps - 1) / kMergeWarps;
    if (merge + d.num_seqs > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(merge + d.num_seqs)), block(kMergeWarps * 32);
    const cudaError_t e = dt == PA_BF16
                              ? launch_pdl(prefix_merge_kernel<__nv_bfloat16>, grid, block, 0, stream, d, mp, (int)merge)
                              : launch_pdl(prefix_merge_kernel<__half>, grid, block, 0, stream, d, mp, (int)merge);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

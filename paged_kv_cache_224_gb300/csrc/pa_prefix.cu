// Decode attention for batches that share a long prefix
// (pa_decode_common_prefix): the schedule of the step (pa_prefix.cuh) and the
// merge of its partials.
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

// Prefix CTAs of a launch, the rest decoding from the start, by a time model.
// A prefix CTA takes about 5 us to its first tile, 1.8 us for a 128-key tile of
// 256 rows (2.4 with the weights in two values), and 4 us for the end of each
// segment, so counts that divide the units or that the units divide, where no CTA
// has pieces of two, are better than others.  A decode instance, two to a CTA,
// takes about 6 us for a unit beside its keys (the chain of its number, length,
// table entries and first keys, its last product and partial) and then 60 GB/s,
// all together at most 6.4 TB/s.  A CTA whose prefix tiles are done decodes.  The
// count is even (a prefix CTA that shares its SM pair with a decoding one runs a
// third longer).  The constants are fitted to sweeps of 8 to 152 CTAs over 19
// shapes on a GB300: the choice is within 2.5% of a sweep's best, 7% in one.  CTAs
// and us, of the choice, of that best and of all 152:
//   groups x size after prefix, own tokens up to, heads    choice      best       152
//   1 x 256 after 8192,  512, 64/8                          84: 122     96: 122   131
//   1 x 256 after 1024, 4096, 64/8                           6: 321     32: 318   338
//   1 x 128 after 4096, 1024, 64/8                          48: 70      40: 69     82
//   1 x 64 after 4096,   256, 32/8                          48: 27      40: 25     37
//   32 x 8 after 1008,   512, 32/32                        128: 337    128: 337   387
//   64 x 4 after 512,    512, 32/8                         128: 115    128: 116   135
//   2 x 12 after 992,    200, 16/16                         64: 21      64: 21     28
//   1 x 8 after 8192,    256, 8/8                          128: 22     128: 22     27
int split_ctas(long long tiles, int unit_tiles, bool two_values, double units, double unit_bytes) {
    const int sms = sm_count();
    const double t_tile = two_values ? 2.4e-6 : 1.8e-6, t_unit = 6e-6 + unit_bytes / 60e9;
    const long long prefix_units = tiles / unit_tiles;
    auto rate = [&](int ctas) {  // units per second
        const double r = 2.0 * ctas / t_unit;
        return unit_bytes > 0 ? std::min(r, 6.4e12 / unit_bytes) : r;
    };
    int best = 2;
    double best_t = 1e30;
    for (int n = 2; n <= sms; n += 2) {
        const long long q = (tiles + n - 1) / n;
        const bool even = prefix_units % n == 0 || n % prefix_units == 0;
        const double segments = (double)((q + unit_tiles - 1) / unit_tiles) + (even ? 0.0 : 1.0);
        const double tp = 5e-6 + q * t_tile + segments * 4e-6;
        const double done = rate(sms - n) * tp;
        const double t = units <= done ? tp : tp + std::max(t_unit, (units - done) / rate(sms));
        if (t < best_t) {
            best_t = t;
            best = n;
        }
    }
    return best;
}

PrefixSchedule prefix_schedule(int groups, int group_size, int prefix_tokens, int group, int num_kv_heads,
                               double units, double unit_bytes) {
    PrefixSchedule s;
    s.row_tiles = (int)(((long long)group_size * group + kUnitRows - 1) / kUnitRows);
    s.n = (prefix_tokens + kNK - 1) / kNK;
    s.tiles = (long long)groups * num_kv_heads * s.row_tiles * s.n;
    s.ctas = (int)std::min<long long>(split_ctas(s.tiles, s.n, prefix_two_values(group_size, group), units, unit_bytes), s.tiles);
    return s;
}

// Where the merge finds a row's prefix partials.
struct MergeParams {
    int group_size, row_tiles, n, head_group;
    int full_tiles, full_ctas;  // of a launch of kPrefillMaxSeqs groups
    int last_first, last_tiles, last_ctas;  // the last launch: its first group, tiles and CTAs
    int prefix_blocks;
};

// CTAs 0 .. merge_ctas-1: one warp per (sequence, head).  The others check a
// sequence each: its prefix table entries against its group's first sequence's,
// and its length, which nothing else looks at where no own tokens are allowed.
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
        if (threadIdx.x == 0) {
            const int L = p.context_lens[s];
            const long long room = (long long)p.max_blocks_per_seq * p.block_size;
            if (L < p.len_offset || L > min((long long)p.max_context_len, room)) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
        }
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
    // (a 32-bit division where the numbers allow it: a third of the 64-bit one's time)
    const int pre = W * N < (1LL << 31)
                        ? (int)(((unsigned)(x + mp.n) * (unsigned)N - 1u) / (unsigned)W -
                                ((unsigned)(x + 1) * (unsigned)N - 1u) / (unsigned)W) + 1
                        : cta_of(x + mp.n - 1, W, N) - cta_of(x, W, N) + 1;
    // The prefix partials do not depend on the sequence's length: they are on
    // their way while it is fetched, and the first of its own while their
    // maxima are compared.
    constexpr int kAhead = 4;
    const size_t base = (size_t)pair * p.slots;
    auto acc_of = [&](size_t sl) { return *reinterpret_cast<const float4 *>(p.ws_acc + sl * kD + lane * VPL); };
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float2 none = make_float2(-INFINITY, 0.f);
    float4 a[kAhead], b[kAhead / 2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) a[i] = i < pre ? acc_of(base + i) : zero;
    const float2 ml_pre = lane < pre ? p.ws_ml[base + lane] : none;
    // the sequence's own partitions, clamped like the decode kernels
    const int cap = (int)min((long long)p.max_context_len, (long long)p.max_blocks_per_seq * p.block_size) - p.len_offset;
    const int L = max(0, min(p.context_lens[s] - p.len_offset, cap));
    const int own = (L + p.partition_tokens - 1) / p.partition_tokens;
    const size_t own_base = base + p.part_base;
#pragma unroll
    for (int i = 0; i < kAhead / 2; ++i) b[i] = i < own ? acc_of(own_base + i) : zero;
    const float2 ml_own = lane < own ? p.ws_ml[own_base + lane] : none;
    float M = fmaxf(ml_pre.x, ml_own.x);
    for (int i = lane + 32; i < pre; i += 32) M = fmaxf(M, p.ws_ml[base + i].x);
    for (int i = lane + 32; i < own; i += 32) M = fmaxf(M, p.ws_ml[own_base + i].x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, m));
    float lsum = 0.f, o[VPL];
#pragma unroll
    for (int d = 0; d < VPL; ++d) o[d] = 0.f;
    auto add = [&](float2 ml, float4 x) {
        const float w = fast_exp2(ml.x - M);
        lsum = fmaf(w, ml.y, lsum);
        o[0] = fmaf(w, x.x, o[0]); o[1] = fmaf(w, x.y, o[1]);
        o[2] = fmaf(w, x.z, o[2]); o[3] = fmaf(w, x.w, o[3]);
    };
    auto lane_ml = [&](const float2 &ml, int i) {
        return make_float2(__shfl_sync(kFull, ml.x, i), __shfl_sync(kFull, ml.y, i));
    };
    if (M != -INFINITY) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) add(lane_ml(ml_pre, i), a[i]);  // (past the last: weight 0)
#pragma unroll 4
        for (int i = kAhead; i < pre; ++i) add(p.ws_ml[base + i], acc_of(base + i));
#pragma unroll
        for (int i = 0; i < kAhead / 2; ++i) add(lane_ml(ml_own, i), b[i]);
#pragma unroll 4
        for (int i = kAhead / 2; i < own; ++i) add(p.ws_ml[own_base + i], acc_of(own_base + i));
    }
    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
    uint2 u;
    u.x = Elem<T>::pack2(o[0] * inv, o[1] * inv);
    u.y = Elem<T>::pack2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (size_t)pair * kD + lane * VPL) = u;
}

}  // namespace

PrefixSchedules prefix_schedules(int groups, int group_size, int prefix_tokens, int group, int num_kv_heads,
                                 int longest_own, int partitions, int num_seqs) {
    PrefixSchedules x{};
    x.last_groups = (groups - 1) % kPrefillMaxSeqs + 1;
    if (groups > kPrefillMaxSeqs)
        x.full = prefix_schedule(kPrefillMaxSeqs, group_size, prefix_tokens, group, num_kv_heads, 0.0, 0.0);
    // the own tokens' lengths are on the device: half of the longest each
    const double bytes = 0.5 * longest_own * (2 * kD * 2) * num_kv_heads * num_seqs;
    const double units = longest_own > 0 ? (double)num_seqs * num_kv_heads * std::max(1.0, 0.5 * partitions) : 0.0;
    x.last = prefix_schedule(x.last_groups, group_size, prefix_tokens, group, num_kv_heads, units,
                             units > 0 ? bytes / units : 0.0);
    return x;
}

int prefix_pieces(int groups, const PrefixSchedules &x) {
    // a unit's first and last pieces, and whole ranges of at least q tiles between them
    auto most = [](const PrefixSchedule &s) {
        const long long q = s.tiles / s.ctas;
        return s.n > 1 ? (int)std::min<long long>(s.ctas, 2 + (s.n - 2) / q) : 1;
    };
    return groups > kPrefillMaxSeqs ? std::max(most(x.full), most(x.last)) : most(x.last);
}

int prefix_partition_tokens(int num_seqs, int num_kv_heads, int block_size, int longest_own) {
    const long long want = 4LL * 2 * sm_count(), have = (long long)num_seqs * num_kv_heads;
    const long long parts = std::max(1LL, want / have);
    const long long pt = std::max<long long>(256, (std::max(longest_own, 1) + parts - 1) / parts);
    return (int)((pt + block_size - 1) / block_size * block_size);
}

int launch_prefix(pa_dtype dt, int block_size, int group, const PrefixParams &pp, cudaStream_t stream) {
    const DecodeParams &d = pp.d;
    // TMA row coordinates are 32-bit
    if ((long long)d.num_blocks * d.num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    const bool any_own = d.max_context_len > pp.prefix_tokens;
    const long long units = any_own ? (long long)d.max_partitions * d.num_seqs * d.num_kv_heads : 0;
    if (units > 0x3fffffffLL) return PA_ERR_UNSUPPORTED;
    const PrefixSchedules &x = pp.sched;
    PrefixLaunch pl{};
    PrefillParams &p = pl.pp;
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
    pl.dp = d;
    pl.decode_next = pp.queue;
    for (int g0 = 0; g0 < pp.groups; g0 += kPrefillMaxSeqs) {
        const bool last = g0 + kPrefillMaxSeqs >= pp.groups;
        p.num_seqs = last ? x.last_groups : kPrefillMaxSeqs;
        for (int i = 0; i < p.num_seqs; ++i) {
            PrefillSeq &q = p.seqs[i];
            q.row_start = (g0 + i) * pp.group_size;
            q.block_table = d.block_tables + (size_t)q.row_start * d.max_blocks_per_seq;
            q.prefix_len = pp.prefix_tokens - 1;
            q.chunk_len = pp.group_size;
        }
        long long rows_units = 0;
        int rc = prefill_schedule<true>(p, group, &rows_units);
        if (rc != PA_OK) return rc;
        pl.prefix_ctas = last ? x.last.ctas : x.full.ctas;
        pl.decode_units = last ? (int)units : 0;
        const unsigned grid = last && any_own ? (unsigned)sm_count() : (unsigned)pl.prefix_ctas;
        rc = dt == PA_BF16 ? launch_prefix_bf16(block_size, group, pl, grid, stream)
                           : launch_prefix_f16(block_size, group, pl, grid, stream);
        if (rc != PA_OK) return rc;
    }
    return PA_OK;
}

int launch_prefix_merge(pa_dtype dt, int group, const PrefixParams &pp, cudaStream_t stream) {
    const DecodeParams &d = pp.d;
    const PrefixSchedules &x = pp.sched;
    MergeParams mp{};
    mp.group_size = pp.group_size;
    mp.head_group = group;
    mp.prefix_blocks = pp.prefix_tokens / d.block_size;
    mp.row_tiles = x.last.row_tiles;
    mp.n = x.last.n;
    mp.full_tiles = pp.groups > kPrefillMaxSeqs ? (int)x.full.tiles : 1;
    mp.full_ctas = pp.groups > kPrefillMaxSeqs ? x.full.ctas : 1;
    mp.last_first = pp.groups - x.last_groups;
    mp.last_tiles = (int)x.last.tiles;
    mp.last_ctas = x.last.ctas;
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

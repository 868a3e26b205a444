// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, kv head) with L cached tokens: when L > keep, the tokens kept
// are the first `sink`, the last `recent`, and of those between the
// keep - sink - recent with the largest totals, the lower index first among
// equals; otherwise all L.  They move, in order, to rows 0 .. n-1 of the
// sequence's new blocks, and their totals to entries 0 .. n-1 of its new row.
// The old blocks are only read: others may share them.
//
// Three launches:
//   mark    each new block's table entry writes its index into owner[block];
//   select  one CTA, or a cluster of 2 to 8, per (sequence, kv head): the
//           threshold total by radix selection (four histograms of 8 bits over
//           an order-preserving integer image of the fp32 totals), then one
//           pass in index order that emits the kept indices and their totals.
//           The totals' images stay in registers (up to 4096 or 8192 a CTA), so
//           that the totals are read twice, to rank them and, from L2, to emit
//           them; rows of more than 65536 read them again in every pass.  A
//           cluster's CTAs read each other's histograms and counts through
//           distributed shared memory.
//           Beside them one CTA per sequence looks for new blocks named twice
//           or still read, and strikes them from owner[];
//   copy    HBM-bound: 16-byte vectors of the kept rows, K and V, to the new
//           blocks that owner[] still grants.
// 64 sequences of 8 kv heads, 1025..4096 tokens to 1024, head_dim 128: 104 us,
// 5.3 TB/s (80% of the copy rate), 79 of them the copy (6.8 TB/s); 2 of 65536
// to 16384: 71 us, 39 of them the copy.  The selection is bound by instruction
// issue with many rows and by its barriers with few.  Selecting and copying in
// one kernel, so that a row's copy runs under other rows' selections, was
// slower (106 and 78 us: a CTA or cluster per row shares the rows out worse
// than a CTA per 256 of them).
//
// Few blocks (kOneCheck): the CTA that checks marks them too, all of them by
// itself, and the first launch falls away (3 sequences of 40..200 tokens to 48:
// 6.6 us and 14.5 us of host time with it, 6.2 and 12.2 without).
//
// owner[] needs no clearing: an entry e counts for block b only if the new
// table's entry e names b, so a stale value proves nothing by itself.
#include <cooperative_groups.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {
namespace cg = cooperative_groups;

constexpr int kStruck = -1;

// Length of sequence s, clamped to what its table, its row of totals and the
// caller's bound hold; *bad tells whether it had to be.
__device__ __forceinline__ int evict_len(const EvictParams &p, int s, bool *bad) {
    const long long room = (long long)p.max_blocks * p.block_size;
    const int cap = (int)min((long long)min(p.max_context_len, p.width), room);
    const int L = p.context_lens[s];
    *bad = L < 0 || L > cap;
    return L < 0 ? 0 : min(L, cap);
}

__device__ __forceinline__ int blocks_of(int tokens, int bs) { return (tokens + bs - 1) / bs; }

// The sequence's new blocks, by one CTA.
__device__ __forceinline__ void mark_blocks(const EvictParams &p, int s) {
    bool bad;
    const int n = min(evict_len(p, s, &bad), p.keep);
    const int nb = blocks_of(n, p.block_size);
    for (int j = threadIdx.x; j < nb; j += blockDim.x) {
        const int b = p.new_block_tables[(size_t)s * p.new_max_blocks + j];
        if (b >= 0 && b < p.num_blocks) p.owner[b] = s * p.new_max_blocks + j;
        else flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
    }
}

__global__ void __launch_bounds__(128) evict_mark_kernel(const __grid_constant__ EvictParams p) {
    pdl_wait();
    pdl_trigger();
    mark_blocks(p, blockIdx.x);
}

// One CTA per sequence, beside the selecting ones: its new length, and the new
// blocks that cannot be written.
__device__ __forceinline__ void check_blocks(const EvictParams &p, int s) {
    bool bad;
    const int L = evict_len(p, s, &bad);
    const int n = min(L, p.keep);
    if (threadIdx.x == 0) {
        if (bad) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
        p.new_context_lens[s] = n;
    }
    // a new block that two entries name belongs to neither
    for (int j = threadIdx.x; j < blocks_of(n, p.block_size); j += blockDim.x) {
        const int e = s * p.new_max_blocks + j, b = p.new_block_tables[e];
        if (b >= 0 && b < p.num_blocks && p.owner[b] != e) {
            p.owner[b] = kStruck;
            flag_error(p.d_err, PA_DEVERR_COPY_PAIR);
        }
    }
    // nor does one that this sequence's table reads
    for (int j = threadIdx.x; j < blocks_of(L, p.block_size); j += blockDim.x) {
        const int b = p.block_tables[(size_t)s * p.max_blocks + j];
        if (b < 0 || b >= p.num_blocks) {
            flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
            continue;
        }
        const int e = p.owner[b];
        if (e < 0 || e >= p.num_seqs * p.new_max_blocks || p.new_block_tables[e] != b) continue;
        const int es = e / p.new_max_blocks;
        bool eb;
        if (e - es * p.new_max_blocks < blocks_of(min(evict_len(p, es, &eb), p.keep), p.block_size)) {
            p.owner[b] = kStruck;
            flag_error(p.d_err, PA_DEVERR_COPY_PAIR);
        }
    }
}

// Totals as unsigned integers of the same order; NaN sorts below everything,
// and the two zeros are one value.
__device__ __forceinline__ unsigned order_key(float x) {
    if (x != x) return 0u;
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A row's tokens go to its CL CTAs of kSelThreads threads in rounds of kSelItems
// tokens a thread (one round, unless the row is longer than that); in a round
// CTA `rank` takes a contiguous segment, its warps contiguous segments of that,
// a warp's lanes neighbours.
template <int CL, int kSelThreads, int kSelItems>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kSelWarps = kSelThreads / 32;
    constexpr int kSelCap = kSelThreads * kSelItems;
    __shared__ unsigned s_hist[4][256];
    __shared__ unsigned s_sum[256];
    __shared__ uint2 s_warp[kSelWarps];
    __shared__ uint2 s_cta[2];      // this CTA's counts of a round (alternating), read by the others
    __shared__ unsigned s_pick[3];  // the digit, how many of its keys are to be taken, and how many there are
    const int rank = CL > 1 ? blockIdx.x % CL : 0;
    const int row = blockIdx.x / CL;
    const int s = row / p.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto all_sync = [] {
        if constexpr (CL > 1) cg::this_cluster().sync();
        else __syncthreads();
    };
    for (int i = tid; i < 4 * 256; i += kSelThreads) (&s_hist[0][0])[i] = 0u;
    __syncthreads();
    pdl_wait();  // the totals and lengths (and the marks) are complete and visible
    pdl_trigger();
    if (row >= p.num_seqs * p.num_kv_heads) {  // clusters that do not select (and so never sync)
        const int seq = blockIdx.x - p.num_seqs * p.num_kv_heads * CL;
        if (p.one_check) {
            if (seq > 0) return;
            for (int i = 0; i < p.num_seqs; ++i) mark_blocks(p, i);
            __syncthreads();
            for (int i = 0; i < p.num_seqs; ++i) check_blocks(p, i);
        } else if (seq < p.num_seqs) {
            check_blocks(p, seq);
        }
        return;
    }
    bool bad;
    const int L = evict_len(p, s, &bad);
    const int n = min(L, p.keep);
    const float *w = p.weights + (size_t)row * p.width;
    float *nw = p.new_weights + (size_t)row * p.width;
    int *kept = p.kept + (size_t)row * p.keep;

    const int rounds = max(1, (L + CL * kSelCap - 1) / (CL * kSelCap));
    // tokens of a warp in a full round: a multiple of 32
    const int wseg = rounds > 1 ? kSelItems * 32 : ((L + CL * kSelWarps - 1) / (CL * kSelWarps) + 31) / 32 * 32;
    const int first = (rank * kSelWarps + warp) * wseg + lane;  // in round 0, item 0
    const int round_len = CL * kSelWarps * wseg;
    const int lo = min(p.sink, L), hi = max(lo, L - p.recent);  // the tokens that are ranked
    const bool cut = L > p.keep;

    // Loads first, without conditions on j (a clamped index instead), so that
    // all of them are in flight at once.
    auto fetch = [&](int r, float (&x)[kSelItems]) {
#pragma unroll
        for (int i = 0; i < kSelItems; ++i)
            if (i * 32 < wseg) x[i] = w[min(r * round_len + first + i * 32, L - 1)];
    };
    unsigned key[kSelItems];
    auto load = [&](int r) {
        float x[kSelItems];
        fetch(r, x);
#pragma unroll
        for (int i = 0; i < kSelItems; ++i)
            if (i * 32 < wseg) key[i] = order_key(x[i]);
    };
    if (L > 0) load(0);  // (an empty row has no segments either)

    // ---- threshold: the `want` largest of the tokens [lo, hi)
    unsigned thr = 0u, eq_take = 0u;  // keys above thr are kept, and the first eq_take equal to it
    unsigned want = (unsigned)(p.keep - p.sink - p.recent);
    if (cut && want == 0) thr = 0xffffffffu;  // no key is above it, and none equal to it is taken
    if (cut && want > 0) {
        unsigned prefix = 0u;
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int r = 0; r < rounds; ++r) {
                if (rounds > 1) load(r);
#pragma unroll
                for (int i = 0; i < kSelItems; ++i) {
                    if (i * 32 >= wseg) break;
                    const int j = r * round_len + first + i * 32;
                    const bool in = j >= lo && j < hi && (pass == 0 || (key[i] >> (shift + 8)) == prefix);
                    const unsigned act = __ballot_sync(kFull, in);
                    if (!act) continue;
                    const unsigned digit = (key[i] >> shift) & 255u;
                    // totals are often all alike (no attention yet): then one add for the warp
                    const unsigned one = __shfl_sync(kFull, digit, __ffs(act) - 1);
                    if (__all_sync(kFull, !in || digit == one)) {
                        if (lane == 0) atomicAdd(&s_hist[pass][one], (unsigned)__popc(act));
                    } else if (in) {
                        atomicAdd(&s_hist[pass][digit], 1u);
                    }
                }
            }
            all_sync();
            if constexpr (CL > 1) {
                if (tid < 256) {
                    unsigned sum = 0u;
#pragma unroll
                    for (int c = 0; c < CL; ++c) sum += *cg::this_cluster().map_shared_rank(&s_hist[pass][tid], c);
                    s_sum[tid] = sum;
                }
                __syncthreads();
            }
            // digit of the want-th largest: counts from the top, by one warp, 8 digits a lane
            if (warp == 0) {
                unsigned c[8], sum = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = (CL > 1 ? s_sum : s_hist[pass])[255 - (lane * 8 + i)];
                    sum += c[i];
                }
                unsigned before = sum;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const unsigned up = __shfl_up_sync(kFull, before, m);
                    if (lane >= m) before += up;
                }
                before -= sum;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < want && want <= before + c[i]) {
                        s_pick[0] = 255u - (unsigned)(lane * 8 + i);
                        s_pick[1] = want - before;
                        s_pick[2] = c[i];
                    }
                    before += c[i];
                }
            }
            __syncthreads();
            prefix = (prefix << 8) | s_pick[0];
            want = s_pick[1];
            if (want == s_pick[2]) {
                // all keys that begin with these digits are taken: no more digits needed
                prefix <<= shift;
                thr = prefix ? prefix - 1u : 0u;
                eq_take = prefix ? 0u : 0xffffffffu;
                break;
            }
            thr = prefix;
            eq_take = want;
        }
    }

    // ---- emit in index order.  A token's place is the count of sure ones
    // before it plus that of those at the threshold, at most eq_take.
    uint2 base = make_uint2(0u, 0u);  // (sure, at the threshold) in earlier rounds
    for (int r = 0; r < rounds && L > 0; ++r) {
        float x[kSelItems];
        fetch(r, x);  // the totals to move, while the counts are put together
        if (rounds > 1) load(r);
        // the warp's tokens of item i that are kept for sure, and those at the threshold
        auto ballots = [&](int i, unsigned &sure, unsigned &at) {
            const int j = r * round_len + first + i * 32;
            const bool ranked = cut && j >= lo && j < hi;
            sure = __ballot_sync(kFull, j < L && (!ranked || key[i] > thr));
            at = __ballot_sync(kFull, j < L && ranked && key[i] == thr);
        };
        uint2 mine = make_uint2(0u, 0u);
#pragma unroll
        for (int i = 0; i < kSelItems; ++i) {
            if (i * 32 >= wseg) break;
            unsigned sure, at;
            ballots(i, sure, at);
            mine.x += __popc(sure);
            mine.y += __popc(at);
        }
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        uint2 before = base, total = make_uint2(0u, 0u);
#pragma unroll
        for (int q = 0; q < kSelWarps; ++q) {
            const uint2 v = s_warp[q];
            if (q < warp) before.x += v.x, before.y += v.y;
            total.x += v.x, total.y += v.y;
        }
        if constexpr (CL > 1) {
            if (tid == 0) s_cta[r & 1] = total;
            cg::this_cluster().sync();
            uint2 round = make_uint2(0u, 0u);
#pragma unroll
            for (int c = 0; c < CL; ++c) {
                const uint2 v = *cg::this_cluster().map_shared_rank(&s_cta[r & 1], c);
                if (c < rank) before.x += v.x, before.y += v.y;
                round.x += v.x, round.y += v.y;
            }
            total = round;
        } else {
            __syncthreads();  // s_warp is read
        }
        const unsigned below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < kSelItems; ++i) {
            if (i * 32 >= wseg) break;
            unsigned sure, at;
            ballots(i, sure, at);
            const unsigned eq = before.y + __popc(at & below);
            const unsigned pos = before.x + __popc(sure & below) + min(eq, eq_take);
            if ((sure >> lane & 1u) || ((at >> lane & 1u) && eq < eq_take)) {
                kept[pos] = r * round_len + first + i * 32;
                nw[pos] = x[i];
            }
            before.x += __popc(sure);
            before.y += __popc(at);
        }
        base.x += total.x;
        base.y += total.y;
    }
    for (int j = n + rank * kSelThreads + tid; j < p.keep; j += CL * kSelThreads) kept[j] = -1;
    for (int j = n + rank * kSelThreads + tid; j < p.width; j += CL * kSelThreads) nw[j] = 0.f;
    if constexpr (CL > 1) cg::this_cluster().sync();  // nobody leaves while its counts are being read
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = kCopyThreads;  // rows of one (sequence, kv head) per CTA

// Finding a row takes four loads, each waiting for the one before (length, kept
// index, table entries, owner); so a thread finds one row, all rows of the CTA
// at once, and then the CTA moves them, LPR lanes (16 bytes each) per row, four
// rows' K and V of each lane in flight.
template <int LPR>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p, int chunks) {
    constexpr int kRowsPass = kCopyThreads / LPR;
    constexpr int kPasses = kCopyRows / kRowsPass;
    constexpr int kFly = 4;
    static_assert(kPasses % kFly == 0, "passes in steps of kFly");
    __shared__ longlong2 s_row[kCopyRows];  // (from, to) in rows of the pool; from -1: no copy
    const int chunk = blockIdx.x % chunks;
    const int sh = blockIdx.x / chunks;
    const int s = sh / p.num_kv_heads, h = sh - s * p.num_kv_heads;
    pdl_wait();
    pdl_trigger();
    bool bad;
    const int n = min(evict_len(p, s, &bad), p.keep);
    const int r0 = chunk * kCopyRows;
    if (r0 >= n) return;
    const int bs = p.block_size, shift = 31 - __clz(bs);  // a power of two
    {
        const int r = r0 + threadIdx.x;
        longlong2 x = make_longlong2(-1, 0);
        if (r < n) {
            const int j = p.kept[(size_t)sh * p.keep + r];
            const int nb = p.new_block_tables[(size_t)s * p.new_max_blocks + (r >> shift)];
            const int b = p.block_tables[(size_t)s * p.max_blocks + (j >> shift)];
            if (b >= 0 && b < p.num_blocks && nb >= 0 && nb < p.num_blocks &&
                p.owner[nb] == s * p.new_max_blocks + (r >> shift)) {
                x.x = ((long long)b * p.num_kv_heads + h) * bs + (j & (bs - 1));
                x.y = ((long long)nb * p.num_kv_heads + h) * bs + (r & (bs - 1));
            }
        }
        s_row[threadIdx.x] = x;
    }
    __syncthreads();
    const int c = threadIdx.x % LPR, first = threadIdx.x / LPR;
    const int passes = (min(n - r0, kCopyRows) + kRowsPass - 1) / kRowsPass;
    const uint4 *ks = static_cast<const uint4 *>(p.k_cache), *vs = static_cast<const uint4 *>(p.v_cache);
    uint4 *kd = static_cast<uint4 *>(p.k_cache), *vd = static_cast<uint4 *>(p.v_cache);
    for (int p0 = 0; p0 < passes; p0 += kFly) {
        longlong2 x[kFly];
        uint4 k[kFly], v[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            x[i] = s_row[(p0 + i) * kRowsPass + first];
            if (x[i].x >= 0) {
                k[i] = ks[x[i].x * LPR + c];
                v[i] = vs[x[i].x * LPR + c];
            }
        }
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            if (x[i].x >= 0) {
                kd[x[i].y * LPR + c] = k[i];
                vd[x[i].y * LPR + c] = v[i];
            }
        }
    }
}

// Most table entries, and sequences, that one CTA marks and checks by itself
// (a sequence takes it some 2 us of dependent loads, beside the selection's 6).
constexpr int kOneCheckBlocks = 1024, kOneCheckSeqs = 4;

constexpr int kNarrow = 256, kNarrowItems = 16;
constexpr int kWide = 512, kWideItems = 16;

template <int CL, int kThreads, int kItems>
int launch_select(const EvictParams &p, long long rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // the checking CTAs beside them, in whole clusters
    const int checks = p.one_check ? 1 : p.num_seqs;
    cfg.gridDim = dim3((unsigned)(rows * CL + (checks + CL - 1) / CL * CL));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<CL, kThreads, kItems>, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_evict(const EvictParams &p_in, cudaStream_t stream) {
    EvictParams p = p_in;
    p.one_check = p.num_seqs <= kOneCheckSeqs &&
                  (long long)p.num_seqs * (p.max_blocks + p.new_max_blocks) <= kOneCheckBlocks;
    if (!p.one_check &&
        launch_pdl(evict_mark_kernel, dim3(p.num_seqs), dim3(128), 0, stream, p) != cudaSuccess)
        return PA_ERR_CUDA;
    const long long rows = (long long)p.num_seqs * p.num_kv_heads;
    const int most = std::min(p.keep, std::min(p.max_context_len, p.width));
    const int chunks = std::max(1, (most + kCopyRows - 1) / kCopyRows);
    if (rows * chunks > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    // CTAs per row: as many as hold it in registers, and more while the rows
    // leave SMs idle and each CTA still has 2048 tokens.  Rows that need more
    // than eight CTAs of 256 threads get CTAs of 512.
    const int longest = std::min(p.max_context_len, p.width);
    int cl = 1;
    while (cl < 8 && ((long long)cl * kNarrow * kNarrowItems < longest ||
                      (rows * cl * 2 <= sm_count() && longest >= 2 * cl * 2048)))
        cl *= 2;
    if (rows * cl + p.num_seqs + cl > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const bool wide = (long long)cl * kNarrow * kNarrowItems < longest;
    const int rc = wide      ? launch_select<8, kWide, kWideItems>(p, rows, stream)
                   : cl == 1 ? launch_select<1, kNarrow, kNarrowItems>(p, rows, stream)
                   : cl == 2 ? launch_select<2, kNarrow, kNarrowItems>(p, rows, stream)
                   : cl == 4 ? launch_select<4, kNarrow, kNarrowItems>(p, rows, stream)
                             : launch_select<8, kNarrow, kNarrowItems>(p, rows, stream);
    if (rc != PA_OK) return rc;
    const dim3 grid((unsigned)(rows * chunks)), block(kCopyThreads);
    cudaError_t e;
    switch (p.head_dim) {
        case 64: e = launch_pdl(evict_copy_kernel<8>, grid, block, 0, stream, p, chunks); break;
        case 128: e = launch_pdl(evict_copy_kernel<16>, grid, block, 0, stream, p, chunks); break;
        default: return PA_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

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
//   select  one CTA per (sequence, kv head): the threshold total by radix
//           selection (four histograms of 8 bits over an order-preserving
//           integer image of the fp32 totals), then one pass in index order
//           that emits the kept indices and their totals.  The CTAs of kv head
//           0 also look for new blocks named twice or still read, and strike
//           them from owner[];
//   copy    HBM-bound: 16-byte vectors of the kept rows, K and V, to the new
//           blocks that owner[] still grants.
// owner[] needs no clearing: an entry e counts for block b only if the new
// table's entry e names b, so a stale value proves nothing by itself.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

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

__global__ void __launch_bounds__(128) evict_mark_kernel(const __grid_constant__ EvictParams p) {
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x;
    bool bad;
    const int n = min(evict_len(p, s, &bad), p.keep);
    const int nb = blocks_of(n, p.block_size);
    for (int j = threadIdx.x; j < nb; j += blockDim.x) {
        const int b = p.new_block_tables[(size_t)s * p.new_max_blocks + j];
        if (b >= 0 && b < p.num_blocks) p.owner[b] = s * p.new_max_blocks + j;
        else flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
    }
}

// Totals as unsigned integers of the same order; NaN sorts below everything,
// and the two zeros are one value.
__device__ __forceinline__ unsigned order_key(float x) {
    if (x != x) return 0u;
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelItems = 4;  // tokens per thread and chunk of the emitting pass

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ unsigned s_hist[256];
    __shared__ unsigned s_warp[kSelWarps];
    __shared__ unsigned s_pick[2];  // the digit, and how many are still to be taken below it
    const int h = blockIdx.x % p.num_kv_heads, s = blockIdx.x / p.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    bool bad;
    const int L = evict_len(p, s, &bad);
    const int n = min(L, p.keep);
    const size_t row = ((size_t)s * p.num_kv_heads + h);
    const float *w = p.weights + row * p.width;
    float *nw = p.new_weights + row * p.width;
    int *kept = p.kept + row * p.keep;

    if (h == 0) {
        if (tid == 0) {
            if (bad) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
            p.new_context_lens[s] = n;
        }
        // a new block that two entries name belongs to neither
        for (int j = tid; j < blocks_of(n, p.block_size); j += kSelThreads) {
            const int e = s * p.new_max_blocks + j, b = p.new_block_tables[e];
            if (b >= 0 && b < p.num_blocks && p.owner[b] != e) {
                p.owner[b] = kStruck;
                flag_error(p.d_err, PA_DEVERR_COPY_PAIR);
            }
        }
        // nor does one that this sequence's table reads
        for (int j = tid; j < blocks_of(L, p.block_size); j += kSelThreads) {
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

    // ---- threshold: the `want` largest of the tokens [lo, hi)
    unsigned thr = 0u, eq_take = 0u;  // keys above thr are kept, and the first eq_take equal to it
    const int lo = min(p.sink, L), hi = max(lo, L - p.recent);
    const bool cut = L > p.keep;
    if (cut) {
        unsigned want = (unsigned)(p.keep - p.sink - p.recent);
        if (want == 0) {
            thr = 0xffffffffu;  // no key is above it, and none equal to it is taken
        } else {
            unsigned prefix = 0u;
            for (int shift = 24; shift >= 0; shift -= 8) {
                if (tid < 256) s_hist[tid] = 0u;
                __syncthreads();
                for (int j = lo + tid; j < hi; j += kSelThreads) {
                    const unsigned k = order_key(w[j]);
                    if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
                }
                __syncthreads();
                // digit of the want-th largest: counts from the top, by one warp, 8 digits a lane
                if (warp == 0) {
                    unsigned c[8], sum = 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        c[i] = s_hist[255 - (lane * 8 + i)];
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
                        }
                        before += c[i];
                    }
                }
                __syncthreads();
                prefix = (prefix << 8) | s_pick[0];
                want = s_pick[1];
            }
            thr = prefix;
            eq_take = want;
        }
    }

    // ---- emit in index order.  Of a token's predecessors, the sure ones (low
    // half of a packed count) and those at the threshold (high half) give its
    // place: sure + min(equal, eq_take).
    unsigned base_sure = 0u, base_eq = 0u;
    for (int j0 = 0; j0 < L; j0 += kSelThreads * kSelItems) {
        unsigned cls[kSelItems], mine = 0u;  // 1: kept, 1 << 16: at the threshold
        float x[kSelItems];
#pragma unroll
        for (int i = 0; i < kSelItems; ++i) {
            const int j = j0 + tid * kSelItems + i;
            cls[i] = 0u;
            x[i] = 0.f;
            if (j < L) {
                x[i] = w[j];
                const unsigned k = order_key(x[i]);
                if (!cut || j < lo || j >= hi || k > thr) cls[i] = 1u;
                else if (k == thr) cls[i] = 1u << 16;
            }
            mine += cls[i];
        }
        unsigned scan = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const unsigned up = __shfl_up_sync(kFull, scan, m);
            if (lane >= m) scan += up;
        }
        __syncthreads();  // the previous chunk's totals are read
        if (lane == 31) s_warp[warp] = scan;
        __syncthreads();
        unsigned before = scan - mine, total = 0u;
#pragma unroll
        for (int q = 0; q < kSelWarps; ++q) {
            const unsigned v = s_warp[q];
            if (q < warp) before += v;
            total += v;
        }
        unsigned sure = base_sure + (before & 0xffffu), eq = base_eq + (before >> 16);
#pragma unroll
        for (int i = 0; i < kSelItems; ++i) {
            const bool at = cls[i] >> 16;
            if (cls[i] == 1u || (at && eq < eq_take)) {
                const unsigned pos = sure + min(eq, eq_take);
                kept[pos] = j0 + tid * kSelItems + i;
                nw[pos] = x[i];
            }
            sure += cls[i] & 1u;
            eq += at;
        }
        base_sure += total & 0xffffu;
        base_eq += total >> 16;
    }
    for (int j = n + tid; j < p.keep; j += kSelThreads) kept[j] = -1;
    for (int j = n + tid; j < p.width; j += kSelThreads) nw[j] = 0.f;
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;  // rows of one (sequence, kv head) per CTA

// LPR lanes (16 bytes each) per row.
template <int LPR>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p, int chunks) {
    constexpr int kRowsPass = kCopyThreads / LPR;
    constexpr int kPasses = kCopyRows / kRowsPass > 0 ? kCopyRows / kRowsPass : 1;
    const int chunk = blockIdx.x % chunks;
    const int sh = blockIdx.x / chunks;
    const int s = sh / p.num_kv_heads, h = sh - s * p.num_kv_heads;
    pdl_wait();
    pdl_trigger();
    bool bad;
    const int n = min(evict_len(p, s, &bad), p.keep);
    const int r0 = chunk * kCopyRows;
    if (r0 >= n) return;
    const int bs = p.block_size;
    const int c = threadIdx.x % LPR;
    const int32_t *kept = p.kept + (size_t)sh * p.keep;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks;
    const int32_t *new_table = p.new_block_tables + (size_t)s * p.new_max_blocks;
    const uint4 *ks = static_cast<const uint4 *>(p.k_cache), *vs = static_cast<const uint4 *>(p.v_cache);
    uint4 *kd = static_cast<uint4 *>(p.k_cache), *vd = static_cast<uint4 *>(p.v_cache);
    long long src[kPasses], dst[kPasses];  // 16-byte units; src -1: no copy
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = r0 + i * kRowsPass + threadIdx.x / LPR;
        src[i] = -1;
        dst[i] = 0;
        if (r < n) {
            const int j = kept[r];
            const int nj = r / bs, b = table[j / bs], nb = new_table[nj];
            const bool ok = b >= 0 && b < p.num_blocks && nb >= 0 && nb < p.num_blocks;
            if (ok && p.owner[nb] == s * p.new_max_blocks + nj) {
                src[i] = (((long long)b * p.num_kv_heads + h) * bs + j % bs) * LPR + c;
                dst[i] = (((long long)nb * p.num_kv_heads + h) * bs + r % bs) * LPR + c;
            }
        }
    }
    uint4 k[kPasses], v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (src[i] >= 0) {
            k[i] = ks[src[i]];
            v[i] = vs[src[i]];
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (src[i] >= 0) {
            kd[dst[i]] = k[i];
            vd[dst[i]] = v[i];
        }
    }
}

}  // namespace

int launch_evict(const EvictParams &p, cudaStream_t stream) {
    if (launch_pdl(evict_mark_kernel, dim3(p.num_seqs), dim3(128), 0, stream, p) != cudaSuccess) return PA_ERR_CUDA;
    const long long rows = (long long)p.num_seqs * p.num_kv_heads;
    const int most = std::min(p.keep, std::min(p.max_context_len, p.width));
    const int chunks = std::max(1, (most + kCopyRows - 1) / kCopyRows);
    if (rows * chunks > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    if (launch_pdl(evict_select_kernel, dim3((unsigned)rows), dim3(kSelThreads), 0, stream, p) != cudaSuccess)
        return PA_ERR_CUDA;
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

// Decode attention over a prefix that many sequences share, on the tensor
// cores: the kernel and its launch templates, instantiated per dtype in
// pa_prefix_bf16.cu and pa_prefix_f16.cu; the host side is in pa_prefix.cu.
//
// One launch of one CTA per SM.  CTAs 0 .. prefix_ctas-1 first attend the
// groups' queries over their prefixes (the chunked prefill's CTA code with
// kPrefix): a group's query rows -- its sequences times the G heads of one kv
// head -- are the rows of 256-row units, so every K/V tile brought into shared
// memory serves 256 rows and the prefix is read from HBM once per group.  Every
// CTA then runs two decode instances (pa_decode_tc.cuh) over the sequences' own
// tokens, units drawn from a queue the grid shares.  The two halves bind on
// different things, the tensor pipe and HBM, and so run side by side; both
// leave unnormalised partials for the merge (pa_prefix.cu).  Scores, maxima,
// sums, accumulators and partials are fp32.  The softmax weights are MMA operands
// of 16 bits: the own tokens' go in as two values, and so do the prefix's for
// groups of up to 128 rows (kTwoP; 2 x 12 sequences after 992 tokens, 16 heads:
// 22.7 us against 21.8 rounded once).  Larger groups round the prefix's once, the
// prefill's choice: two values took the case below from 127 to 171 us, and over a
// prefix's keys, 16 at least, one rounding each averages out (bf16, 8192 keys:
// at most 2.3e-3 off where two values are 1.7e-3 off, the result's own rounding).
//
// 256 sequences after 8192 shared tokens, own tokens up to 512, 64/8 heads,
// bf16: 127 us, 557 TFLOP/s and 2.5 TB/s at once (two launches, prefix and own
// tokens one after the other: 153).  Of a decode instance's 5 to 8 us per
// sequence and kv head 1.2 us per 128-key tile are work; the rest is the chain
// of its length, queries, last product and partial.
#pragma once

#include "pa_decode_tc.cuh"
#include "pa_prefill.cuh"

namespace pa {
namespace pfx {
using namespace pf;

constexpr int kStepThreads = kThreads + 32;  // twelve warps: two decode instances
constexpr int kDecodeSlots = tcd::kSlotsStandalone;
constexpr uint32_t kDecodeInst1 = (tcd::TcLayout<kDecodeSlots>::kSmemUsed + 1023u) & ~1023u;
constexpr uint32_t kHolder = kOffBar + 248;  // TMEM base of a decode-only CTA (past the prefix pass's barriers)
static_assert(kStepThreads == 2 * tcd::kThreads, "two decode instances");
static_assert(kDecodeInst1 + tcd::TcLayout<kDecodeSlots>::kSmemUsed <= (uint32_t)kOffBar,
              "both decode instances fit below the prefix pass's barriers");
static_assert((2 * kSlots + 2 + 2 * kQT) * 8 + 4 + 4 * kQT <= 248, "the holder is past the prefix pass's barriers");
static_assert(2 * tcd::kTmemCols <= kTmemCols, "both instances' columns in the prefix pass's allocation");

// Have a tensor map fetched before the first copy that needs it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

template <typename T, int BS, int G, bool kTwoP>
__global__ void __launch_bounds__(kStepThreads, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixLaunch pl, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
    const bool prefix = (int)blockIdx.x < pl.prefix_ctas;
    const int warp = threadIdx.x >> 5, inst = (int)threadIdx.x / tcd::kThreads;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    volatile uint32_t *holder =
        reinterpret_cast<volatile uint32_t *>(smem_raw + (((raw + 1023u) & ~1023u) - raw) + kHolder);
    if (threadIdx.x == 0) {
        prefetch_map(&tmk);
        prefetch_map(&tmv);
        prefetch_map(&tmq);
    }
    uint32_t tmem = 0;
    if (prefix)  // ends with a CTA barrier: every warp is past the pass's use of shared memory and TMEM
        tmem = prefill_cta<T, BS, G, true, true, false, kTwoP>(pl.pp, tmk, tmv, tmq, (int)blockIdx.x, pl.prefix_ctas);
    tcd::TcRun r;
    tcd::tc_init<kDecodeSlots>(r, inst * kDecodeInst1, inst * 6, kBarL + 1 + inst);
    if (!prefix && warp == 1) tcd::tc_alloc(holder, 2 * tcd::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!prefix) tmem = *holder;
    r.tmem = tmem + inst * tcd::kTmemCols;
    tcd::tc_queue_loop<T, BS, G, kDecodeSlots>(pl.dp, &tmk, &tmv, r, pl.decode_next, pl.decode_units,
                                               2 * (int)gridDim.x);
    tcd::tc_drain<kDecodeSlots>(r);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tcd::tc_dealloc(tmem, prefix ? (uint32_t)kTmemCols : 2 * tcd::kTmemCols);
}

template <typename T, int BS, int G, bool kTwoP>
int launch_prefix_t(const PrefixLaunch &pl, unsigned grid, cudaStream_t stream) {
    auto kern = prefix_tc_kernel<T, BS, G, kTwoP>;
    static std::atomic<uint64_t> attr_done{0};
    if (ensure_smem_attr(kern, kSmemAlloc, attr_done) != PA_OK) return PA_ERR_CUDA;
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap tmk, tmv, tmq;
    if (!make_pool_map(&tmk, pl.pp.k_cache, pl.pp, BS, bf16) || !make_pool_map(&tmv, pl.pp.v_cache, pl.pp, BS, bf16) ||
        !make_query_map(&tmq, pl.pp, G, bf16))
        return PA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = kSmemAlloc;
    cfg.stream = stream;  // plain stream order: its CTAs fill every SM, and start no sooner when launched early
    return cudaLaunchKernelEx(&cfg, kern, pl, tmk, tmv, tmq) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T>
int launch_prefix_dtype(int block_size, int group, const PrefixLaunch &pl, unsigned grid, cudaStream_t stream) {
#define PA_PFX_CASE(BB, GG) \
    if (block_size == BB && group == GG)                                             \
        return prefix_two_values(pl.pp.seqs[0].chunk_len, GG)                        \
                   ? launch_prefix_t<T, BB, GG, true>(pl, grid, stream)              \
                   : launch_prefix_t<T, BB, GG, false>(pl, grid, stream);
#define PA_PFX_GROUPS(BB) PA_PFX_CASE(BB, 1) PA_PFX_CASE(BB, 2) PA_PFX_CASE(BB, 4) PA_PFX_CASE(BB, 8)
    PA_PFX_GROUPS(16)
    PA_PFX_GROUPS(32)
    PA_PFX_GROUPS(64)
    PA_PFX_GROUPS(128)
#undef PA_PFX_GROUPS
#undef PA_PFX_CASE
    return PA_ERR_UNSUPPORTED;
}

}  // namespace pfx
}  // namespace pa

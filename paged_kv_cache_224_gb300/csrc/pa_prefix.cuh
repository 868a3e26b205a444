// Decode attention over a prefix that many sequences share, on the tensor
// cores: the kernel instances of one dtype (the CTA's code is the chunked
// prefill's, pa_prefill.cuh, with kPrefix).
//
// The group's query rows -- its sequences times the G heads of one kv head --
// are the rows of 256-row units, so every K/V tile brought into shared memory
// serves 256 rows, and the prefix is read from HBM once per group: with few
// rows the pass is bound by HBM, with many by the tensor pipe.
#pragma once

#include "pa_prefill.cuh"

namespace pa {
namespace pfx {
using namespace pf;

template <typename T, int BS, int G>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
    pdl_wait();  // the kernel before this one on the stream (e.g. the cache write) has finished
    prefill_cta<T, BS, G, false, true>(p, tmk, tmv, tmq, (int)blockIdx.x, (int)gridDim.x);
}

template <typename T, int BS, int G>
int launch_prefix_t(const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    auto kern = prefix_tc_kernel<T, BS, G>;
    static std::atomic<uint64_t> attr_done{0};
    if (ensure_smem_attr(kern, kSmemAlloc, attr_done) != PA_OK) return PA_ERR_CUDA;
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap tmk, tmv, tmq;
    if (!make_pool_map(&tmk, p.k_cache, p, BS, bf16) || !make_pool_map(&tmv, p.v_cache, p, BS, bf16) ||
        !make_query_map(&tmq, p, G, bf16))
        return PA_ERR_CUDA;
    return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemAlloc, stream, p, tmk, tmv, tmq) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

template <typename T>
int launch_prefix_dtype(int block_size, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
#define PA_PFX_CASE(BB, GG) \
    if (block_size == BB && group == GG) return launch_prefix_t<T, BB, GG>(p, grid, stream);
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

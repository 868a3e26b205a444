// Several query positions over one paged cache, scores kept: the kernel and its
// launch templates, instantiated per dtype in pa_window_bf16.cu and
// pa_window_f16.cu; the host side and what follows are in pa_window.cu.
//
// The CTA's code is the chunked prefill's (pa_prefill.cuh, kPrefix and kWindow):
// the rows of a unit are the query positions times the G heads of one kv head,
// up to 256 of them against every K/V tile, where the decode kernels would read
// the whole cache once per position.  Softmax weights go to their product with V
// as two 16-bit values (kTwoP): rounded once, over two to four keys, they would
// put outputs past what a position alone keeps to.  The totals take them in fp32
// from the kept scores.  16 positions of 4 heads over 8191 tokens, 8 kv heads,
// f16: 32 us (28 with weights rounded once, 98 position by position), of which a
// CTA's 3 to 4 key tiles take some 2.5 us each and its first copies, its partial
// and the totals the rest: bound by latency at this size.
#pragma once

#include "pa_prefill.cuh"

namespace pa {
namespace wnd {
using namespace pf;

template <typename T, int BS, int G>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
    pdl_wait();  // the kernel before this one on the stream (e.g. the cache write) has finished
    prefill_cta<T, BS, G, false, true, true, true>(p, tmk, tmv, tmq, (int)blockIdx.x, (int)gridDim.x);
}

template <typename T, int BS, int G>
int launch_window_t(const PrefillParams &p, unsigned grid, cudaStream_t stream) {
    auto kern = window_tc_kernel<T, BS, G>;
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
int launch_window_dtype(int block_size, int group, const PrefillParams &p, unsigned grid, cudaStream_t stream) {
#define PA_WND_CASE(BB, GG) \
    if (block_size == BB && group == GG) return launch_window_t<T, BB, GG>(p, grid, stream);
#define PA_WND_GROUPS(BB) PA_WND_CASE(BB, 1) PA_WND_CASE(BB, 2) PA_WND_CASE(BB, 4) PA_WND_CASE(BB, 8)
    PA_WND_GROUPS(16)
    PA_WND_GROUPS(32)
    PA_WND_GROUPS(64)
    PA_WND_GROUPS(128)
#undef PA_WND_GROUPS
#undef PA_WND_CASE
    return PA_ERR_UNSUPPORTED;
}

}  // namespace wnd
}  // namespace pa

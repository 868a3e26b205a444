// Paged decode attention over an 8-bit cache on the tensor cores (tcgen05,
// kind::f8f6f4), head_dim 128.
//
// The mathematics is that of pa_fp8_decode.cu: weights over z_j = s_j + ev_j, sums
// of 2^(z_j - M) codes of v_j, and of 2^(z_j - M) 2^(-ev_j).  The codes go to the
// MMAs as they lie in memory, with keys as the M dimension:
//   S^T[128 keys][N] = K[128 keys][128 dims] . Q^T
//   O^T[128 dims][N] += V^T[128 dims][128 keys] . P^T    (V read in place, MN-major)
// An 8-bit operand on the other side would leave a query or a weight 3 or 4 bits, so
// each goes in as several rows of N, every one the rounded residual of those before
// times a power of two: queries as three e4m3 rows (12 bits, what fp16 has and more
// than bf16 has: scores are as exact as fp32 sums), weights as four e5m2 rows (12
// bits; e5m2 for its range, so that what a key 2^-30 below the largest adds still
// counts: a long context may hold very many of them).  N is padded to 16 by the
// MMA anyway (32 for eight heads).
#include "pa_fp8_decode_tc.cuh"

namespace pa {
namespace {

using namespace tc8;

constexpr int kSlots = 6;  // ring slots of 16 KB; two CTAs to an SM

template <typename T, int BS, int G>
__global__ void __launch_bounds__(kThreads, 2)
    decode_fp8_tc_kernel(const __grid_constant__ Fp8DecodeParams p, const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv) {
    using L = Lay<G, kSlots>;
    extern __shared__ unsigned char smem_raw[];
    pdl_wait();     // the kernel before this one on the stream (e.g. the cache write) has finished
    pdl_trigger();  // the reduce may be scheduled once every CTA of this grid has started
    const Unit u = unit_of(p.d, (int)blockIdx.x, BS, threadIdx.x == 0);
    if (u.skip) return;
    if (u.ntiles == 0) {
        empty_unit<T, G>(p.d, u, (int)threadIdx.x);
        return;
    }
    const uint32_t raw = smem_addr(smem_raw), sb = (raw + 1023u) & ~1023u;  // swizzle atoms start on 1 KB
    unsigned char *smem = smem_raw + (sb - raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
    volatile uint32_t *holder = reinterpret_cast<volatile uint32_t *>(bars + 2 * kSlots + 7);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kSlots; ++i) mbar_init(&bars[i], 1);
        mbar_init(&bars[2 * kSlots], 128);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars[2 * kSlots + 1 + b], 1);
            mbar_init(&bars[2 * kSlots + 3 + b], 128);
            mbar_init(&bars[2 * kSlots + 5 + b], 1);
        }
        fence_barrier_init();
    }
    if (threadIdx.x >> 5 == 1) tcd::tc_alloc(holder, L::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    run_unit<T, BS, G, kSlots>(p, &tmk, &tmv, u, smem, sb, tmem);
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x >> 5 == 1) tcd::tc_dealloc(tmem, L::kCols);
}

// The pool as rows of 128 codes: a block of a kv head is one box of block_size rows.
bool make_rows_map(CUtensorMap *map, const void *pool, const DecodeParams &p, int bs) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {kD, (cuuint64_t)p.num_blocks * p.num_kv_heads * bs};
    const cuuint64_t strides[1] = {kD};
    const cuuint32_t box[2] = {kD, (cuuint32_t)bs};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int BS, int G>
int launch_t(const Fp8DecodeParams &p, cudaStream_t stream) {
    auto kern = decode_fp8_tc_kernel<T, BS, G>;
    constexpr int smem = Lay<G, kSlots>::kAlloc;
    static std::atomic<uint64_t> attr_done{0};
    if (ensure_smem_attr(kern, smem, attr_done) != PA_OK) return PA_ERR_CUDA;
    CUtensorMap tmk, tmv;
    if (!make_rows_map(&tmk, p.d.k_cache, p.d, BS) || !make_rows_map(&tmv, p.d.v_cache, p.d, BS)) return PA_ERR_UNSUPPORTED;
    const long long units = (long long)p.d.max_partitions * p.d.num_seqs * p.d.num_kv_heads;
    if (units > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    return launch_pdl(kern, dim3((unsigned)units), dim3(kThreads), smem, stream, p, tmk, tmv) == cudaSuccess ? PA_OK
                                                                                                             : PA_ERR_CUDA;
}

template <typename T, int G>
int launch_block(int bs, const Fp8DecodeParams &p, cudaStream_t stream) {
    switch (bs) {
        case 8: return launch_t<T, 8, G>(p, stream);
        case 16: return launch_t<T, 16, G>(p, stream);
        case 32: return launch_t<T, 32, G>(p, stream);
        case 64: return launch_t<T, 64, G>(p, stream);
        default: return launch_t<T, 128, G>(p, stream);
    }
}

template <typename T>
int launch_group(int bs, int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    return group == 1   ? launch_block<T, 1>(bs, p, stream)
           : group == 2 ? launch_block<T, 2>(bs, p, stream)
           : group == 4 ? launch_block<T, 4>(bs, p, stream)
                        : launch_block<T, 8>(bs, p, stream);
}

}  // namespace

int launch_decode_fp8_tc(pa_dtype dt, int block_size, int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    // TMA rows are 32-bit coordinates
    if ((long long)p.d.num_blocks * p.d.num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    return dt == PA_BF16 ? launch_group<__nv_bfloat16>(block_size, group, p, stream)
                         : launch_group<__half>(block_size, group, p, stream);
}

}  // namespace pa

// Paged decode attention over an 8-bit cache.
//
// With k_j = code * 2^(ek_j), v_j = code * 2^(ev_j) of key j's block, and scores in
// log2 units (scale * log2(e) in the query), the sum that is kept runs over
//     z_j = s_j + ev_j,   o = sum_j 2^(z_j - M) * (codes of v_j),
//     l = sum_j 2^(z_j - M) * 2^(-ev_j),   M the running maximum of z,
// and out = o / l: the values' scales only move the exponents, and however far the
// scales of two blocks are apart, no term of o is larger than its codes.
//
// A CTA takes one unit (sequence, kv head, partition) for up to four of the kv head's
// query heads; D / 16 adjacent lanes hold a key's row, 16 codes each.
#include <type_traits>

#include "pa_fp8.cuh"
#include "pa_internal.h"

namespace pa {

int launch_decode_reduce_bf16(int head_dim, const DecodeParams &p, cudaStream_t stream);
int launch_decode_reduce_f16(int head_dim, const DecodeParams &p, cudaStream_t stream);

namespace {

constexpr int kWarps = 4;

template <typename T, int D, int GH>
__global__ void __launch_bounds__(kWarps * 32) decode_fp8_kernel(const __grid_constant__ Fp8DecodeParams fp) {
    constexpr int kLanes = D / 16, kKeys = 32 / kLanes;  // lanes of a key, keys of a warp
    const DecodeParams &p = fp.d;
    __shared__ float s_acc[kWarps][GH][D];
    __shared__ float2 s_ml[kWarps][GH];
    pdl_wait();     // the kernel before this one on the stream (e.g. the cache write) has finished
    pdl_trigger();  // the reduce may be scheduled once every CTA of this grid has started
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int subs = p.grp_inner / GH;
    const int sub = blockIdx.x % subs, unit = blockIdx.x / subs;
    const int per_part = p.num_seqs * p.num_kv_heads;
    const int part = unit / per_part, rem = unit - part * per_part;
    const int s = rem / p.num_kv_heads, kvh = rem - s * p.num_kv_heads;
    int L = p.context_lens[s];
    const int Lcap = min(p.max_context_len, p.max_blocks_per_seq * p.block_size);
    if (L < 0 || L > Lcap) {
        if (tid == 0 && part == 0 && kvh == 0 && sub == 0) flag_error(p.d_err, PA_DEVERR_CONTEXT_RANGE);
        L = L < 0 ? 0 : Lcap;
    }
    const int nparts = L > 0 ? (L + p.partition_tokens - 1) / p.partition_tokens : 1;
    if (part >= nparts) return;
    const int tok0 = part * p.partition_tokens, tok1 = min(L, tok0 + p.partition_tokens);
    const int c = lane % kLanes;
    const size_t row0 = (size_t)s * p.num_heads + (size_t)kvh * p.grp_inner + sub * GH;

    float q[GH][16];
#pragma unroll
    for (int h = 0; h < GH; ++h) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) + (row0 + h) * D + c * 16);
        float a[8], b[8];
        unpack8<T>(src[0], a);
        unpack8<T>(src[1], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[h][i] = a[i] * p.scale_log2;
            q[h][8 + i] = b[i] * p.scale_log2;
        }
    }
    float acc[GH][16], m[GH], l[GH];
#pragma unroll
    for (int h = 0; h < GH; ++h) {
        m[h] = kEmptyMax;
        l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[h][i] = 0.f;
    }
    const int32_t *table = p.block_tables + (size_t)s * p.table_stride;
    // every lane of the warp goes through the same steps; a key past the end has no block
    for (int j0 = tok0 + warp * kKeys; j0 < tok1; j0 += kWarps * kKeys) {
        const int j = j0 + lane / kLanes;
        const int slot = j / p.block_size;
        int blk = j < tok1 ? table[slot] : -1;
        if (j < tok1 && (blk < 0 || blk >= p.num_blocks)) {
            flag_error(p.d_err, PA_DEVERR_BLOCK_RANGE);
            blk = -1;
        }
        uint4 ku = make_uint4(0, 0, 0, 0), vu = ku;
        float ks = 0.f, ev = 0.f;
        if (blk >= 0) {
            const size_t tile = (size_t)blk * p.num_kv_heads + kvh;
            const size_t at = (tile * p.block_size + (j - slot * p.block_size)) * D + c * 16;
            ku = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.k_cache) + at);
            vu = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.v_cache) + at);
            ks = scale_of(fp.k_scales[tile]);
            ev = log_scale_of(fp.v_scales[tile]);
        }
        float f[16], dot[GH];
        values16(ku, f);
#pragma unroll
        for (int h = 0; h < GH; ++h) {
            dot[h] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) dot[h] = fmaf(q[h][i], f[i], dot[h]);
#pragma unroll
            for (int x = kLanes / 2; x > 0; x >>= 1) dot[h] += __shfl_xor_sync(kFull, dot[h], x);
        }
        if (blk >= 0) {
            values16(vu, f);
            const float per = scale_of(ev == ev ? (unsigned)max(127 - (int)ev, 0) : 255u);  // 2^(-ev)
#pragma unroll
            for (int h = 0; h < GH; ++h) {
                const float z = fmaf(dot[h], ks, ev);
                const float mn = fmaxf(m[h], z);
                const float alpha = fast_exp2(m[h] - mn), w = fast_exp2(z - mn);
                m[h] = mn;
                l[h] = fmaf(l[h], alpha, w * per);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[h][i] = fmaf(acc[h][i], alpha, w * f[i]);
            }
        }
    }
    // the warp's keys, then the warps
#pragma unroll
    for (int h = 0; h < GH; ++h) {
#pragma unroll
        for (int x = kLanes; x < 32; x <<= 1) {
            const float mo = __shfl_xor_sync(kFull, m[h], x), lo = __shfl_xor_sync(kFull, l[h], x);
            const float mn = fmaxf(m[h], mo), a = fast_exp2(m[h] - mn), b = fast_exp2(mo - mn);
            m[h] = mn;
            l[h] = l[h] * a + lo * b;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[h][i] = acc[h][i] * a + __shfl_xor_sync(kFull, acc[h][i], x) * b;
        }
        if (lane < kLanes) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s_acc[warp][h][c * 16 + i] = acc[h][i];
            if (lane == 0) s_ml[warp][h] = make_float2(m[h], l[h]);
        }
    }
    __syncthreads();
    const bool direct = nparts == 1;
    for (int i = tid; i < GH * D; i += kWarps * 32) {
        const int h = i / D, d = i - h * D;
        float M = kEmptyMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][h].x);
        float lsum = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = fast_exp2(s_ml[w][h].x - M);
            lsum = fmaf(a, s_ml[w][h].y, lsum);
            o = fmaf(a, s_acc[w][h][d], o);
        }
        const size_t row = row0 + h;
        if (direct) {
            static_cast<T *>(p.out)[row * D + d] = (T)(lsum != 0.f ? o / lsum : 0.f);
        } else {
            const size_t at = row * p.slots + part;
            p.ws_acc[at * D + d] = o;
            if (d == 0) p.ws_ml[at] = make_float2(M, lsum);
        }
    }
}

template <typename T, int D, int GH>
cudaError_t decode_t(const Fp8DecodeParams &p, cudaStream_t stream) {
    const long long ctas = (long long)p.d.max_partitions * p.d.num_seqs * p.d.num_kv_heads * (p.d.grp_inner / GH);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(decode_fp8_kernel<T, D, GH>, dim3((unsigned)ctas), dim3(kWarps * 32), 0, stream, p);
}

template <typename T, int D>
cudaError_t decode_d(int group, const Fp8DecodeParams &p, cudaStream_t stream) {
    return group == 1 ? decode_t<T, D, 1>(p, stream) : group == 2 ? decode_t<T, D, 2>(p, stream) : decode_t<T, D, 4>(p, stream);
}

}  // namespace

int fp8_partition_tokens(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                         int max_context_len) {
    (void)head_dim;
    return auto_partition_tokens(num_seqs, num_heads, num_kv_heads, block_size, max_context_len);
}

int launch_decode_fp8(pa_dtype dt, int head_dim, int block_size, int group, const Fp8DecodeParams &p,
                      cudaStream_t stream) {
    int rc = head_dim == 128 ? launch_decode_fp8_tc(dt, block_size, group, p, stream) : PA_ERR_UNSUPPORTED;
    if (rc != PA_OK && rc != PA_ERR_UNSUPPORTED) return rc;
    cudaError_t e = cudaSuccess;
    if (rc == PA_OK) ;
    else if (dt == PA_BF16) e = head_dim == 128 ? decode_d<__nv_bfloat16, 128>(group, p, stream) : decode_d<__nv_bfloat16, 64>(group, p, stream);
    else e = head_dim == 128 ? decode_d<__half, 128>(group, p, stream) : decode_d<__half, 64>(group, p, stream);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    if (p.d.max_partitions == 1) return PA_OK;
    return dt == PA_BF16 ? launch_decode_reduce_bf16(head_dim, p.d, stream) : launch_decode_reduce_f16(head_dim, p.d, stream);
}

}  // namespace pa

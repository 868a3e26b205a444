// Rotary positions with several axes, fused with the cache write.
//
// Pair i of a head (dimensions (i, i + R/2), or (2i, 2i + 1) when interleaved;
// R = rot_dim) turns by the angle positions[axis(i)][t] * inv_freq[i]:
//     (a, b) -> (a cos - b sin, b cos + a sin),
// in fp32, rounded once; dimensions past R and the values pass unchanged.
// Queries go to query_out, keys and values straight into their cache slots.
//
// Angles.  fp32 has no digits left for the fraction of a turn once a position
// passes a few thousand, so the turn count is kept in fixed point: inv_freq /
// 2 pi, reduced to [-1/2, 1/2] in fp64, becomes a 64-bit fraction of a turn,
// and position * fraction modulo 2^64 -- one wrapping integer product -- is
// the angle modulo a whole turn, with nothing lost to the position's size.
// Its top 32 bits go to sincospi: the angle is within 2^-25 turns' worth of
// fp32 rounding plus |position| * 2^-55 turns of the exact product.
//
// HBM-bound: every row is read and written once.  One CTA per token; its
// cosines and sines are computed once, one pair per thread, into shared memory
// and serve every head.  A thread moves units of two 16-byte vectors (8 pairs),
// and a thread's place in the head is the same for every head it takes, so it
// reads its 8 cosines and sines once.
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <typename T>
__global__ void __launch_bounds__(1024) rotary_kernel(const __grid_constant__ RotaryParams p) {
    // cosines of pairs 8c .. 8c+3, 8c+4 .. 8c+7, then the sines alike, [4][unit c]: a warp's reads are consecutive
    __shared__ float4 s_cs[4][kRotaryMaxDim / 16];
    __shared__ long long s_dst;  // element offset of kv head 0's row in the caches, -1: not written
    const int t = blockIdx.x;
    const int tid = threadIdx.x;
    const int upr = p.head_dim / 16;  // units of a head; the first rot_dim / 16 are turned
    const int nrot = p.rot_dim / 16;
    const int c = tid % upr;
    const int row0 = tid / upr, rows_step = blockDim.x / upr;
    const int rows = p.num_heads + 2 * p.num_kv_heads;
    const bool turned = c < nrot;
    // element offsets of the unit's two vectors inside a head
    const int e0 = turned ? (p.interleaved ? c * 16 : c * 8) : c * 16;
    const int e1 = turned && !p.interleaved ? p.rot_dim / 2 + c * 8 : e0 + 8;

    pdl_wait();
    pdl_trigger();  // what follows may be placed; it waits for these writes
    auto src_of = [&](int row) {
        const T *base;
        if (row < p.num_heads) base = static_cast<const T *>(p.query) + t * p.query_stride + (long long)row * p.head_dim;
        else if (row < p.num_heads + p.num_kv_heads)
            base = static_cast<const T *>(p.key) + t * p.key_stride + (long long)(row - p.num_heads) * p.head_dim;
        else
            base = static_cast<const T *>(p.value) + t * p.value_stride +
                   (long long)(row - p.num_heads - p.num_kv_heads) * p.head_dim;
        return base;
    };
    // the first row's vectors are on their way while the angles are computed
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    int row = row0 < rows_step ? row0 : rows;  // threads past the last whole row of units take none
    if (row < rows) {
        const T *s = src_of(row);
        va = ldg_stream(s + e0);
        vb = ldg_stream(s + e1);
    }
    for (int i = tid; i < p.rot_dim / 2; i += blockDim.x) {
        const float f = p.inv_freq[i];
        const int pos = p.positions[(long long)p.pair_axis[i] * p.num_tokens + t];
        double turns = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= rint(turns);
        const long long frac = __double2ll_rn(turns * 18446744073709551616.0);  // of a turn, in 2^-64
        const unsigned long long ang = (unsigned long long)frac * (unsigned long long)(long long)pos;
        const int top = (int)(unsigned)((ang + 0x80000000ull) >> 32);
        float sn, cs;
        sincospif((float)top * 4.656612873077393e-10f, &sn, &cs);  // top * 2^-31 half turns
        if (!isfinite(f)) sn = cs = __int_as_float(0x7fc00000);
        float *q = reinterpret_cast<float *>(s_cs);
        constexpr int plane = kRotaryMaxDim / 16 * 4;
        const int u = i >> 3, k = (i >> 2) & 1;
        q[k * plane + u * 4 + (i & 3)] = cs;
        q[(2 + k) * plane + u * 4 + (i & 3)] = sn;
    }
    if (tid == 0) {
        const long long slot = p.slots[t];
        long long dst = -1;
        if (slot >= (long long)p.num_blocks * p.block_size) {
            flag_error(p.d_err, PA_DEVERR_SLOT_RANGE);
        } else if (slot >= 0) {
            const long long blk = slot / p.block_size;
            dst = (blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size)) * p.head_dim;
        }
        s_dst = dst;
    }
    __syncthreads();
    const long long dst = s_dst;
    float cs[8], sn[8];
    if (turned) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 x = s_cs[k][c], y = s_cs[2 + k][c];
            cs[4 * k] = x.x, cs[4 * k + 1] = x.y, cs[4 * k + 2] = x.z, cs[4 * k + 3] = x.w;
            sn[4 * k] = y.x, sn[4 * k + 1] = y.y, sn[4 * k + 2] = y.z, sn[4 * k + 3] = y.w;
        }
    }
    while (row < rows) {
        const int next = row + rows_step;
        uint4 na = va, nb = vb;
        if (next < rows) {
            const T *s = src_of(next);
            na = ldg_stream(s + e0);
            nb = ldg_stream(s + e1);
        }
        if (turned && row < p.num_heads + p.num_kv_heads) {
            float a[8], b[8];
            unpack8<T>(va, a);
            unpack8<T>(vb, b);
            if (p.interleaved) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = a[2 * k], y = a[2 * k + 1], z = b[2 * k], w = b[2 * k + 1];
                    a[2 * k] = fmaf(x, cs[k], -(y * sn[k]));
                    a[2 * k + 1] = fmaf(y, cs[k], x * sn[k]);
                    b[2 * k] = fmaf(z, cs[4 + k], -(w * sn[4 + k]));
                    b[2 * k + 1] = fmaf(w, cs[4 + k], z * sn[4 + k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float x = a[k], y = b[k];
                    a[k] = fmaf(x, cs[k], -(y * sn[k]));
                    b[k] = fmaf(y, cs[k], x * sn[k]);
                }
            }
            va = pack8<T>(a);
            vb = pack8<T>(b);
        }
        T *out = nullptr;
        if (row < p.num_heads) {
            out = static_cast<T *>(p.query_out) + t * p.query_out_stride + (long long)row * p.head_dim;
        } else if (dst >= 0) {
            const bool is_v = row >= p.num_heads + p.num_kv_heads;
            const long long h = row - p.num_heads - (is_v ? p.num_kv_heads : 0);
            out = static_cast<T *>(is_v ? p.v_cache : p.k_cache) + dst + h * p.block_size * p.head_dim;
        }
        if (out) {
            // values have no turned units: their two vectors lie side by side all the same, e0 and e1 cover the row
            *reinterpret_cast<uint4 *>(out + e0) = va;
            *reinterpret_cast<uint4 *>(out + e1) = vb;
        }
        va = na;
        vb = nb;
        row = next;
    }
}

}  // namespace

int launch_rotary(pa_dtype dt, const RotaryParams &p, cudaStream_t stream) {
    // enough threads that a token's units take one pass, up to 640
    const int units = (p.num_heads + 2 * p.num_kv_heads) * (p.head_dim / 16);
    const int threads = std::min(640, std::max(64, (units + 31) / 32 * 32));
    cudaError_t e;
    if (dt == PA_BF16) e = launch_pdl(rotary_kernel<__nv_bfloat16>, dim3(p.num_tokens), dim3(threads), 0, stream, p);
    else e = launch_pdl(rotary_kernel<__half>, dim3(p.num_tokens), dim3(threads), 0, stream, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

// Norms of queries and keys head by head, the rotation and the cache write in one pass.
//
//   y[d] = x[d] / sqrt(mean(x^2) + eps) * w[d], then the pairs of y turned as in
// pa_rotary.cu, all in fp32, one rounding.  (Heads beyond 2^59 or below 2^-50, whose squares
// fp32 does not hold, brought to the middle by a power of two took every call with them: a
// look at each row's sum 58.4 -> 60.0 us, the 8-bit write 64.3 -> 66.3.)  (Queries alone where the keys go to
// an 8-bit cache.)
//
// HBM-bound, every row is read and written once, but only just: four rows of 128 values
// cost a warp some 220 instructions, so what can be kept out of the loop is.  A warp has
// one token (or, in short calls, every n-th part of its rows), its cosines, sines and
// weights in registers, and walks its rows with constant steps, four loads of each lane
// on their way at once.  Warps wait for nothing but their own loads.
// 8192 tokens of 64/8 heads of 128, bf16: 58.4 us, 5.75 TB/s (85% of the copy rate).  The
// rotary kernel's form, a CTA per token with one row ahead, took 69; windows of four
// tokens dealt out to groups of lanes with three rows ahead 76 (346 instructions, most
// of them for addresses); three rows at a time and more warps 64; tokens parted among
// twice as many warps 72 (each part computes the angles anew); pair axes read from
// constant memory, every lane its own, 59.4.
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rotary.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;  // rows that a lane has under way

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, 5) norm_rotary_kernel(const __grid_constant__ RotaryParams p, int parts) {
    constexpr int kPlane = kRotaryMaxDim / 16;
    // cosines of pairs 8c .. 8c+3, 8c+4 .. 8c+7, then the sines alike, so that a warp's reads are consecutive
    __shared__ float4 s_cs[kWarps][4][kPlane];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = p.head_dim, upr = D / 16, half = p.rot_dim / 2, lanes = norm_lanes(upr);
    const int c = lane % lanes, sub = lane / lanes, per_warp = 32 / lanes;
    const bool busy = c < upr, turned = c < p.rot_dim / 16;
    const int e0 = turned && !kInterleaved ? c * 8 : c * 16;
    const int e1 = turned && !kInterleaved ? half + c * 8 : e0 + 8;
    const float per_dim = 1.f / (float)D;
    const long long item = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(item / parts), part = (int)(item - (long long)t * parts);

    pdl_wait();
    pdl_trigger();  // what follows may be placed; it waits for these writes
    if (t >= p.num_tokens) return;

    float cs[8], sn[8];
    if (half > 0) {
        float *q = reinterpret_cast<float *>(s_cs[warp]);
        for (int i = lane; i < half; i += 32) {
            const float f = p.inv_freq[i];
            float x, y;
            turn_sincos(turn_fraction(f), p.positions[(p.one_axis ? 0LL : (long long)p.pair_axis[i] * p.num_tokens) + t], y, x);
            if (!isfinite(f)) x = y = __int_as_float(0x7fc00000);
            const int at = (i >> 2 & 1) * kPlane * 4 + (i >> 3) * 4 + (i & 3);
            q[at] = x;
            q[2 * kPlane * 4 + at] = y;
        }
        __syncwarp();
        if (turned) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = s_cs[warp][i][c], y = s_cs[warp][2 + i][c];
                cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
                sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
            }
        }
    }
    // `heads` rows from src on, a head's row every D elements there and every out_step in
    // out; without norm weights (the values) they pass as they are
    auto rows = [&](const T *src, T *out, long long out_step, int heads, const void *norm) {
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (norm && busy) {
            w0 = *reinterpret_cast<const uint4 *>(static_cast<const T *>(norm) + e0);
            w1 = *reinterpret_cast<const uint4 *>(static_cast<const T *>(norm) + e1);
        }
        const int first = part * per_warp + sub, step = parts * per_warp;
        for (int r0 = first; r0 - sub < heads; r0 += kRows * step) {  // (the same for all lanes)
            uint4 va[kRows], vb[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = r0 + i * step;
                va[i] = vb[i] = make_uint4(0, 0, 0, 0);
                if (r < heads && busy) {
                    va[i] = ldg_stream(src + r * D + e0);
                    vb[i] = ldg_stream(src + r * D + e1);
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = r0 + i * step;
                if (r - sub >= heads) break;
                if (norm) {
                    float a[8], b[8];
                    unpack8<T>(va[i], a);
                    unpack8<T>(vb[i], b);
                    norm_unit<T>(a, b, lanes, per_dim, p.eps, w0, w1);
                    if (turned) turn_unit<kInterleaved>(a, b, cs, sn);
                    va[i] = pack8<T>(a);
                    vb[i] = pack8<T>(b);
                }
                if (out && r < heads && busy) {
                    *reinterpret_cast<uint4 *>(out + r * out_step + e0) = va[i];
                    *reinterpret_cast<uint4 *>(out + r * out_step + e1) = vb[i];
                }
            }
        }
    };
    rows(static_cast<const T *>(p.query) + t * p.query_stride, static_cast<T *>(p.query_out) + t * p.query_out_stride, D,
         p.num_heads, p.query_norm);
    if (p.num_kv_heads > 0) {
        const long long dst = cache_row(p, p.slots[t]);
        if (dst < 0) return;
        const long long step = (long long)p.block_size * D;
        rows(static_cast<const T *>(p.key) + t * p.key_stride, static_cast<T *>(p.k_cache) + dst, step, p.num_kv_heads,
             p.key_norm);
        rows(static_cast<const T *>(p.value) + t * p.value_stride, static_cast<T *>(p.v_cache) + dst, step, p.num_kv_heads,
             nullptr);
    }
}

template <typename T, bool kInterleaved>
int launch_t(const RotaryParams &p, cudaStream_t stream) {
    // A token's rows are parted among warps until there are about four times as many
    // warps as the GPU holds, or a part is down to one warp's rows at a time: enough to
    // even out the last ones, and each part computes the token's angles anew.
    const int per_warp = 32 / norm_lanes(p.head_dim / 16);
    const int most = std::max(1, (std::max(p.num_heads, p.num_kv_heads) + per_warp - 1) / per_warp);
    const long long want = 4LL * 24 * sm_count();
    const int parts = (int)std::min<long long>(most, std::max(1LL, want / p.num_tokens));
    const long long ctas = ((long long)p.num_tokens * parts + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    return launch_pdl(norm_rotary_kernel<T, kInterleaved>, dim3((unsigned)ctas), dim3(kWarps * 32), 0, stream, p, parts) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

int launch_norm_rotary(pa_dtype dt, const RotaryParams &p, cudaStream_t stream) {
    if (dt == PA_BF16) return p.interleaved ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
    return p.interleaved ? launch_t<__half, true>(p, stream) : launch_t<__half, false>(p, stream);
}

}  // namespace pa

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
// 2 pi modulo 1 becomes a 64-bit fraction of a turn, and position * fraction
// modulo 2^64 -- one wrapping integer product -- is the angle modulo a whole
// turn, with nothing lost to the position's size.  Its top 32 bits go to
// sincospi: the angle is within 2^-25 turns' worth of fp32 rounding plus
// |position| * 2^-64 turns of the exact product, whatever inv_freq is.  (An fp64
// product for the fraction is off by up to 2^-54 of the turns a position makes,
// too much far out for frequencies above 1, and slower: 8192 tokens take 57 us by
// one, 59.6 by two that add up, 55.5 by the integers.)
//
// HBM-bound: every row is read and written once.  A CTA walks tokens
// blockIdx.x, + gridDim.x, ...; a token's cosines and sines are computed once,
// one pair per thread, into one of two shared buffers and serve every head,
// and while its rows move, the next token's first vectors are on their way and
// its angles are computed.  A thread moves units of two 16-byte vectors (8
// pairs); its place in the head is the same for every head it takes, so it
// reads its 8 cosines and sines once per token, and pair i's turns per
// position stay in one thread's register throughout.  8192 tokens of 64/8 heads
// of 128, bf16: 55.5 us, 6.0 TB/s (90% of the copy rate).  With the fp64 product,
// one CTA per token, which does that and the first loads of every token anew, took
// 147 us, blocks of 640 threads, two to an SM, 64.
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

// A token's kv head 0 row: element offset in the caches, or -1 for none.
__device__ __forceinline__ long long cache_row(const RotaryParams &p, long long slot) {
    if (slot < 0) return -1;
    if (slot >= (long long)p.num_blocks * p.block_size) {
        flag_error(p.d_err, PA_DEVERR_SLOT_RANGE);
        return -1;
    }
    // most pools have fewer than 2^32 slots, and a 32-bit division costs a third
    const long long blk = (slot >> 32) ? slot / p.block_size : (long long)((unsigned)slot / (unsigned)p.block_size);
    return (blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size)) * p.head_dim;
}

// f / (2 pi) modulo 1, in 2^-64, to half a unit, for finite f.  With f = m 2^e
// (m of 24 bits) only the bits of 1 / (2 pi) from e places after the binary point
// on count modulo 1, and 96 of them are enough (Payne and Hanek's reduction,
// 1983): three 32-bit products, no fp64.
__device__ __forceinline__ long long turn_fraction(float f) {
    // 160 zeros, for e < 0, and 1 / (2 pi) to 224 bits
    static constexpr unsigned kBits[12] = {0u, 0u, 0u, 0u, 0u, 0x28be60dbu, 0x9391054au, 0x7f09d5f4u, 0x7d4d3770u,
                                           0x36d8a566u, 0x4f10e410u, 0x7f9458eau};
    const unsigned u = __float_as_uint(f), ex = u >> 23 & 255u;
    const unsigned m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int at = (int)min(max(ex, 1u), 254u) - 150 + 160;  // the first bit that counts, 11 .. 264
    const int k = at >> 5, s = at & 31;
    const unsigned w0 = kBits[k], w1 = kBits[k + 1], w2 = kBits[k + 2], w3 = kBits[k + 3];
    const unsigned hi = __funnelshift_l(w1, w0, s), mid = __funnelshift_l(w2, w1, s), lo = __funnelshift_l(w3, w2, s);
    const unsigned long long low = (unsigned long long)m * lo;
    const unsigned long long frac = ((unsigned long long)(m * hi) << 32) + (unsigned long long)m * mid + (low >> 32) +
                                    (low >> 31 & 1u);
    return (long long)((u >> 31) ? 0ull - frac : frac);
}

constexpr int kMaxThreads = 320;

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kMaxThreads, 4) rotary_kernel(const __grid_constant__ RotaryParams p) {
    // [2 tokens]: cosines of pairs 8c .. 8c+3, 8c+4 .. 8c+7, then the sines
    // alike, [4][unit c], so that a warp's reads are consecutive
    __shared__ float4 s_cs[2][4][kRotaryMaxDim / 16];
    __shared__ long long s_dst[2];
    const int tid = threadIdx.x;
    const int upr = p.head_dim / 16;  // units of a head; the first rot_dim / 16 are turned
    const int half = p.rot_dim / 2;
    const int c = tid % upr;
    const int row0 = tid / upr, rows_step = blockDim.x / upr;
    const int rows_qk = p.num_heads + p.num_kv_heads, rows = rows_qk + p.num_kv_heads;
    const bool turned = c < p.rot_dim / 16;
    // element offsets of the unit's two vectors inside a head (the values' too: e0 and e1 cover the row either way)
    const int e0 = turned && !kInterleaved ? c * 8 : c * 16;
    const int e1 = turned && !kInterleaved ? half + c * 8 : e0 + 8;
    const bool active = row0 < rows_step;  // threads past the last whole row of units move nothing

    pdl_wait();
    pdl_trigger();  // what follows may be placed; it waits for these writes

    // threads [0, half) of the block's upper end turn pair `mine`, the last
    // warp's first lane looks the slot up: not the threads with most rows
    const int mine = (int)blockDim.x - 1 - tid;
    long long frac = 0, frac2 = 0;  // turns per position in 2^-64, of pair `mine` (and mine + blockDim.x)
    bool finite = true, finite2 = true;
    auto turns_of = [&](int i, bool &ok) {
        const float f = p.inv_freq[i];
        ok = isfinite(f);
        return turn_fraction(f);
    };
    if (mine < half) frac = turns_of(mine, finite);
    if (mine + (int)blockDim.x < half) frac2 = turns_of(mine + blockDim.x, finite2);
    auto angle = [&](int i, long long fr, bool ok, int pos, int buf) {
        const unsigned long long ang = (unsigned long long)fr * (unsigned long long)(long long)pos;
        const int top = (int)(unsigned)((ang + 0x80000000ull) >> 32);
        float sn, cs;
        sincospif((float)top * 4.656612873077393e-10f, &sn, &cs);  // top * 2^-31 half turns
        if (!ok) sn = cs = __int_as_float(0x7fc00000);
        float *q = reinterpret_cast<float *>(s_cs[buf]);
        constexpr int plane = kRotaryMaxDim / 16 * 4;
        const int u = i >> 3, k = (i >> 2) & 1;
        q[k * plane + u * 4 + (i & 3)] = cs;
        q[(2 + k) * plane + u * 4 + (i & 3)] = sn;
    };
    auto prepare = [&](int t, int buf) {
        if (mine < half)
            angle(mine, frac, finite, p.positions[(long long)p.pair_axis[mine] * p.num_tokens + t], buf);
        if (mine + (int)blockDim.x < half)
            angle(mine + blockDim.x, frac2, finite2,
                  p.positions[(long long)p.pair_axis[mine + blockDim.x] * p.num_tokens + t], buf);
        if (tid == 0) s_dst[buf] = cache_row(p, p.slots[t]);
    };
    auto src_of = [&](int t, int row) {
        if (row < p.num_heads) return static_cast<const T *>(p.query) + t * p.query_stride + row * p.head_dim;
        if (row < rows_qk) return static_cast<const T *>(p.key) + t * p.key_stride + (row - p.num_heads) * p.head_dim;
        return static_cast<const T *>(p.value) + t * p.value_stride + (row - rows_qk) * p.head_dim;
    };

    int t = blockIdx.x, buf = 0;
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    if (active && row0 < rows) {
        const T *s = src_of(t, row0);
        va = ldg_stream(s + e0);
        vb = ldg_stream(s + e1);
    }
    prepare(t, 0);
    __syncthreads();
    for (; t < p.num_tokens; t += gridDim.x, buf ^= 1) {
        const int t_next = t + gridDim.x;
        if (active) {
            const long long dst = s_dst[buf];
            float cs[8], sn[8];
            if (turned) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 x = s_cs[buf][k][c], y = s_cs[buf][2 + k][c];
                    cs[4 * k] = x.x, cs[4 * k + 1] = x.y, cs[4 * k + 2] = x.z, cs[4 * k + 3] = x.w;
                    sn[4 * k] = y.x, sn[4 * k + 1] = y.y, sn[4 * k + 2] = y.z, sn[4 * k + 3] = y.w;
                }
            }
            for (int row = row0; row < rows; row += rows_step) {
                // the next unit's vectors, of this token or the next
                const bool more = row + rows_step < rows;
                uint4 na = va, nb = vb;
                if (more || t_next < p.num_tokens) {
                    const T *s = more ? src_of(t, row + rows_step) : src_of(t_next, row0);
                    na = ldg_stream(s + e0);
                    nb = ldg_stream(s + e1);
                }
                if (turned && row < rows_qk) {
                    float a[8], b[8];
                    unpack8<T>(va, a);
                    unpack8<T>(vb, b);
                    if (kInterleaved) {
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
                    out = static_cast<T *>(p.query_out) + t * p.query_out_stride + row * p.head_dim;
                } else if (dst >= 0) {
                    const bool is_v = row >= rows_qk;
                    const long long h = row - (is_v ? rows_qk : p.num_heads);
                    out = static_cast<T *>(is_v ? p.v_cache : p.k_cache) + dst + h * p.block_size * p.head_dim;
                }
                if (out) {
                    *reinterpret_cast<uint4 *>(out + e0) = va;
                    *reinterpret_cast<uint4 *>(out + e1) = vb;
                }
                va = na;
                vb = nb;
            }
        }
        if (t_next < p.num_tokens) prepare(t_next, buf ^ 1);
        __syncthreads();  // the next token's angles are written, and this one's read
    }
}

template <typename T, bool kInterleaved>
int launch_t(const RotaryParams &p, int threads, cudaStream_t stream) {
    auto kern = rotary_kernel<T, kInterleaved>;
    static std::atomic<int> resident[kMaxThreads / 32 + 1];  // CTAs an SM holds, by block size; asked for once
    int n = resident[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) != cudaSuccess || n < 1) return PA_ERR_CUDA;
        resident[threads / 32].store(n, std::memory_order_relaxed);
    }
    const int grid = std::min(p.num_tokens, sm_count() * n);
    return launch_pdl(kern, dim3(grid), dim3(threads), 0, stream, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_rotary(pa_dtype dt, const RotaryParams &p, cudaStream_t stream) {
    // A token's units take one pass of up to kMaxThreads threads; the grid
    // is one wave of resident CTAs, which walk the tokens.
    const int units = (p.num_heads + 2 * p.num_kv_heads) * (p.head_dim / 16);
    const int passes = (units + kMaxThreads - 1) / kMaxThreads;
    const int threads = std::max(64, ((units + passes - 1) / passes + 31) / 32 * 32);
    if (dt == PA_BF16) return p.interleaved ? launch_t<__nv_bfloat16, true>(p, threads, stream)
                                             : launch_t<__nv_bfloat16, false>(p, threads, stream);
    return p.interleaved ? launch_t<__half, true>(p, threads, stream) : launch_t<__half, false>(p, threads, stream);
}

}  // namespace pa

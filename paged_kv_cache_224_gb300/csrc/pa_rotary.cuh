// What the rotary kernels share: streaming loads, the turns a position makes, and
// how a head's units lie over the lanes.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

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

// sine and cosine of `pos` positions' angle, `fr` = turn_fraction(inv_freq): the
// product modulo 2^64 is the angle modulo a whole turn.
__device__ __forceinline__ void turn_sincos(long long fr, int pos, float &sn, float &cs) {
    const unsigned long long ang = (unsigned long long)fr * (unsigned long long)(long long)pos;
    const int top = (int)(unsigned)((ang + 0x80000000ull) >> 32);
    sincospif((float)top * 4.656612873077393e-10f, &sn, &cs);  // top * 2^-31 half turns
}

// Lanes that a head's units take when they add up its squares.
__host__ __device__ constexpr int norm_lanes(int units) {
    return units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : 16;
}

// Turn the pairs of a unit (two vectors of a head) by its cosines and sines.
template <bool kInterleaved>
__device__ __forceinline__ void turn_unit(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
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
}

// 1 / sqrt(x), within 2^-22.9 of itself.
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Divide a head, held by `lanes` adjacent lanes, by its root mean square and multiply it
// by its weights (w0, w1: those of the unit's two vectors).
template <typename T>
__device__ __forceinline__ void norm_unit(float (&a)[8], float (&b)[8], int lanes, float per_dim, float eps, const uint4 &w0,
                                          const uint4 &w1) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        s0 = fmaf(a[k], a[k], s0);
        s1 = fmaf(b[k], b[k], s1);
    }
    float sum = s0 + s1;
    for (int m = lanes >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(kFull, sum, m);
    const float r = rsqrt_approx(fmaf(sum, per_dim, eps));
    float w[8];
    unpack8<T>(w0, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = a[k] * r * w[k];
    unpack8<T>(w1, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = b[k] * r * w[k];
}

}  // namespace pa

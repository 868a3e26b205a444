// What the rotary kernels share: streaming loads, the turns a position makes, and
// how a head's units lie over the lanes.
#pragma once

#include "pa_device.cuh"

namespace pa {

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
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

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

}  // namespace pa

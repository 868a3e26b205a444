// 8-bit caches: e4m3 codes and their power-of-two scales.
//
// A block of one kv head holds block_size rows of codes and one scale 2^e, kept
// as the byte e + 127 (e8m0).  Between two scales a row is moved by a power of
// two, which costs no precision as long as its codes stay out of the subnormals:
// that is why the scale is a power of two and not amax / 448.
#pragma once

#include <cuda_fp8.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kScaleLowest = -64;    // exponent of the smallest scale that is written
constexpr float kF16Top = 61440.f;   // largest code times a power of two that fp16 holds (1.875 * 2^15)
constexpr float kEmptyMax = -3.0e38f;  // running maximum of a partial without keys: finite, so that a merge of such partials is zeros

// 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float scale_of(unsigned byte) {
    return __uint_as_float(byte == 255u ? 0x7fc00000u : byte ? byte << 23 : 0x00400000u);
}
// byte - 127, the scale's logarithm; 255 is NaN.
__device__ __forceinline__ float log_scale_of(unsigned byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : (float)((int)byte - 127);
}

// The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), from kScaleLowest on;
// amax finite and >= 0.
__device__ __forceinline__ int scale_exponent(float amax) {
    const unsigned u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kScaleLowest ? kScaleLowest : e;
}

// What is held of a value: infinities, which e4m3 lacks, as NaN; for fp16 models
// nothing beyond kF16Top, so that whatever a code stands for is an fp16 value too.
template <typename T>
__device__ __forceinline__ float holdable(float x) {
    const bool finite = fabsf(x) <= 3.402823466e38f;
    if constexpr (std::is_same<T, __half>::value) x = fminf(fmaxf(x, -kF16Top), kF16Top);
    return finite ? x : __uint_as_float(0x7fc00000u);
}

// Bits of the largest magnitude that holdable() leaves as it is.
template <typename T>
__device__ __forceinline__ unsigned top_held() {
    return std::is_same<T, __half>::value ? 0x47700000u : 0x7f7fffffu;  // 61440, the largest float
}

// |x|, or 0 where it is not finite: what counts towards a scale.
__device__ __forceinline__ float counted(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

__device__ __forceinline__ unsigned codes2(float a, float b) {
    return (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
    return codes2(a, b) | codes2(c, d) << 16;
}
__device__ __forceinline__ float2 values2(unsigned two) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&r));
}
// The 16 values of a vector of codes.
__device__ __forceinline__ void values16(const uint4 &u, float (&f)[16]) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 a = values2(w[k] & 0xffffu), b = values2(w[k] >> 16);
        f[4 * k] = a.x, f[4 * k + 1] = a.y, f[4 * k + 2] = b.x, f[4 * k + 3] = b.y;
    }
}

// l 2^d for d <= 0 and a sum of weights l, in two halves: where scales of the values enter
// the maxima and are far apart, l may be as large as 2^d is small.
__device__ __forceinline__ float moved(float l, float d) {
    const float half = fast_exp2(0.5f * d);
    return l * half * half;
}

}  // namespace pa

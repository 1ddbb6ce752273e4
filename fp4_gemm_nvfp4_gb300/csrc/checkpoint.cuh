// checkpoint.cuh -- the 8-bit form in which activations are kept for the
// backward pass: one E4M3 code per value and one power-of-two scale 2^(b - 127)
// per 1x32 block, b the smallest byte from 10 up that takes the block's largest
// finite magnitude to at most 448 (E4M3's largest value).
//
// A power of two makes x / scale and code * scale exact, so the code's rounding
// (3 bits after the leading one: at most 2^-4 of the value) is the only one.
// From b = 10 on the smallest code, 2^-9, stands for 2^-126: every kept value is
// a normal FP32 and BF16 number.  At the other end 2^128 is none: what would
// round to it (magnitudes past 1.9375 * 2^127) is kept as 1.875 * 2^127.
// Infinities and NaN become E4M3's one NaN and
// do not take part in the block's maximum.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "device_common.cuh"

namespace nvfp4 {

constexpr int kCheckpointBlock = 32;
constexpr uint32_t kLeastScaleByte = 10;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// |x|, or 0 for an infinity or a NaN, as bits: these order like the values.
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
    const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
    return m < 0x7F800000u ? m : 0u;
}

// The scale byte of a block whose largest magnitude has these bits: 448 is
// 1.75 * 2^8, so a mantissa past 1.75 takes the next power.
__device__ __forceinline__ uint32_t checkpoint_scale(uint32_t amax_bits) {
    const uint32_t e = (amax_bits + 0x1FFFFFu) >> 23;
    return e < kLeastScaleByte + 8u ? kLeastScaleByte : e - 8u;
}
__device__ __forceinline__ float checkpoint_factor(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ float checkpoint_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// One value in units of its block's scale.  The conversion saturates an
// infinity to 448; a product with 0 makes it NaN.
__device__ __forceinline__ float checkpoint_scaled(float x, float inv) {
    float v = x * (finite_magnitude(x) == 0u ? 0.0f : inv);
    if (inv == 0x1p-120f && fabsf(v) > 240.0f) v = copysignf(240.0f, v);   // the type's end
    return v;
}

// Four values, times inv, as four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3_codes_x4(float a, float b, float c, float d, float inv) {
    uint16_t lo, hi;
    a = checkpoint_scaled(a, inv), b = checkpoint_scaled(b, inv);
    c = checkpoint_scaled(c, inv), d = checkpoint_scaled(d, inv);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Four codes, times factor.
__device__ __forceinline__ void e4m3_values_x4(uint32_t codes, float factor, float* v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h;   // two FP16, exact
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(codes >> (16 * i))));
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        v[2 * i] = lo * factor;
        v[2 * i + 1] = hi * factor;
    }
}

}  // namespace nvfp4

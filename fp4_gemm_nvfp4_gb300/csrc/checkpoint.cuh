// checkpoint.cuh -- the 8-bit form in which activations are kept for the
// backward pass: one E4M3 code per value and one power-of-two scale 2^(b - 127)
// per 1x32 block, b the smallest byte from 10 up that takes the block's largest
// finite magnitude to at most 448 (E4M3's largest value).
//
// A power of two makes x / scale and code * scale exact, so the code's rounding
// (3 bits after the leading one: at most 2^-4 of the value, or half the smallest
// code, 2^(b - 137), where that is more) is the only one.
// From b = 10 on the smallest code, 2^-9, stands for 2^-126: every kept value is
// a normal FP32 and BF16 number.  At the other end 2^128 is none: what would
// round to it (magnitudes past 1.9375 * 2^127) is kept as 1.875 * 2^127.
// Infinities and NaN become E4M3's one NaN and
// do not take part in the block's maximum.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "device_common.cuh"
#include "mma_common.cuh"

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

// Four values as four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3_codes_x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// One value in units of its block's scale where the block is not an ordinary
// one: the conversion would saturate an infinity to 448, so that it is made a
// NaN, and at the type's end codes stop at 240.
__device__ __forceinline__ float checkpoint_scaled(float x, float inv) {
    float v = x * (finite_magnitude(x) == 0u ? 0.0f : inv);
    if (inv == 0x1p-120f && fabsf(v) > 240.0f) v = copysignf(240.0f, v);
    return v;
}
// Whether a block with this largest magnitude, infinities and NaN counted, is
// not an ordinary one.
constexpr uint32_t kOrdinaryBelow = 0x7F000000u;   // 2^127

// Eight BF16 values, of which four lanes have a 1x32 block: its scale byte (all
// four lanes).  Magnitudes order like their bits, two at a time.  `special` is
// set where a block of the warp is not an ordinary one.
__device__ __forceinline__ uint32_t bf16_scale(const uint4& w, bool& special) {
    constexpr uint32_t kMagnitudes = 0x7FFF7FFFu;
    uint32_t m = __vmaxu2(__vmaxu2(w.x & kMagnitudes, w.y & kMagnitudes), __vmaxu2(w.z & kMagnitudes, w.w & kMagnitudes));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = max(m & 0xFFFF0000u, m << 16);
    special = __any_sync(0xFFFFFFFFu, m >= kOrdinaryBelow);
    if (special) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(finite_magnitude(bf16lo(u[i])), finite_magnitude(bf16hi(u[i]))));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    return checkpoint_scale(m);
}
// ... and a lane's codes.
__device__ __forceinline__ uint2 bf16_codes(const uint4& w, uint32_t b, bool special) {
    float v[8] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y), bf16lo(w.z), bf16hi(w.z), bf16lo(w.w), bf16hi(w.w)};
    const float inv = checkpoint_inverse(b);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = special ? checkpoint_scaled(v[k], inv) : v[k] * inv;
    return make_uint2(e4m3_codes_x4(v[0], v[1], v[2], v[3]), e4m3_codes_x4(v[4], v[5], v[6], v[7]));
}

// 32 FP32 values as the codes of one block; returns its scale byte.
__device__ __forceinline__ uint32_t fp32_codes(const uint32_t* v, uint32_t* codes) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(__uint_as_float(v[i]))));
    uint32_t bits = __float_as_uint(m) & 0x7FFFFFFFu;
    uint32_t b = checkpoint_scale(bits);
    if (bits < kOrdinaryBelow) {
        const float f = checkpoint_inverse(b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            codes[i] = e4m3_codes_x4(__uint_as_float(v[4 * i]) * f, __uint_as_float(v[4 * i + 1]) * f,
                                     __uint_as_float(v[4 * i + 2]) * f, __uint_as_float(v[4 * i + 3]) * f);
    } else {
        bits = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) bits = max(bits, finite_magnitude(__uint_as_float(v[i])));
        b = checkpoint_scale(bits);
        const float f = checkpoint_inverse(b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            codes[i] = e4m3_codes_x4(
                checkpoint_scaled(__uint_as_float(v[4 * i]), f), checkpoint_scaled(__uint_as_float(v[4 * i + 1]), f),
                checkpoint_scaled(__uint_as_float(v[4 * i + 2]), f), checkpoint_scaled(__uint_as_float(v[4 * i + 3]), f));
    }
    return b;
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
__device__ __forceinline__ void e4m3_pairs_x4(uint32_t codes, float factor, uint64_t* v) {
    float f[4];
    e4m3_values_x4(codes, factor, f);
    v[0] = pair(f[0], f[1]);
    v[1] = pair(f[2], f[3]);
}

}  // namespace nvfp4

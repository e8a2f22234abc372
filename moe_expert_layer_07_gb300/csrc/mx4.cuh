// MXFP4 arithmetic that several kernels share (defined in mx4.cu's header).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// Scale byte of a block from its largest magnitude's fp32 bits (as unsigned
// integers, magnitudes order like their values, infinities and NaN on top).
// A subnormal number's biased exponent is 0, below every exponent the clamp
// lets through.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    if (amax_bits == 0u) return 127u;
    return (uint32_t)max((int)(amax_bits >> 23) - 2, 0);
}

// The scale that a byte stands for: 2^(byte - 127); byte 0 is a subnormal
// number, byte 255 NaN.
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
    const uint32_t edge = byte == 0u || byte == 255u ? 0x00400000u : 0u;
    return __uint_as_float((byte << 23) | edge);
}

// 2^(127 - byte), the reciprocal of a finite block's scale (byte <= 252 there).
__device__ __forceinline__ float mx4_inv_scale(uint32_t byte) {
    return __uint_as_float((254u - byte) << 23);
}

// e2m1 codes of eight values times `inv` (element 0 in the lowest four bits).
__device__ __forceinline__ uint32_t mx4_codes8_scaled(const float (&v)[8], float inv) {
    uint32_t out;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(out)
        : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv),
          "f"(v[5] * inv), "f"(v[6] * inv), "f"(v[7] * inv));
    return out;
}
__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8], uint32_t byte) {
    return byte == 255u ? 0u : mx4_codes8_scaled(v, mx4_inv_scale(byte));
}

// Two e2m1 codes (a byte's low and high half) as fp16 values, exact: four
// words of two from one word of eight.
__device__ __forceinline__ void mx4_half8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=&r"(h[0]), "=&r"(h[1]), "=&r"(h[2]), "=&r"(h[3])
        : "r"(codes));
}
__device__ __forceinline__ void mx4_values8(uint32_t codes, float scale, float (&v)[8]) {
    uint32_t h[4];
    mx4_half8(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        v[2 * j] = f.x * scale;
        v[2 * j + 1] = f.y * scale;
    }
}

}  // namespace moe

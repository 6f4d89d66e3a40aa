// e4m3.cuh -- the 8-bit cache's numbers: e4m3 codes times a power of two for each block
// of tokens and kv head.
//
// A scale is a power of two in fp32; its exponent alone is read, held to 2^-64 .. 2^120, so that
// scales, their inverses and sums of weights times either stay finite whatever the bits
// are. Powers of two: code times scale is exact in bf16 and fp32, a scale that rises moves
// only the exponents of earlier codes (no bit is lost but below 2^-14 of the largest value that the
// new scale can hold), and a quotient by it needs no division. A scale of 32 bits a block costs 0.4 % of 16 x 64 codes.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace sc {

constexpr int kMinScaleExp = -64, kMaxScaleExp = 120;

// Two e4m3 codes (the halves' bytes in order) as f16, exactly; NaN codes give NaN.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
// Two values rounded to nearest, ties to even, up to +-448 (infinities too; NaN stays): lo in the
// low byte.
__device__ __forceinline__ uint32_t f32_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\t"
        "cvt.u32.u16 %0, h;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float f16_lo(uint32_t h) {
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.f32.f16 %0, lo;\n\t}"
        : "=f"(f)
        : "r"(h));
    return f;
}
__device__ __forceinline__ float f16_hi(uint32_t h) {
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.f32.f16 %0, hi;\n\t}"
        : "=f"(f)
        : "r"(h));
    return f;
}

// The scale that a word holds, as fp32 bits, and its inverse's.
__device__ __forceinline__ uint32_t scale_bits(uint32_t word) {
    const uint32_t e = word & 0x7F800000u;
    return min(max(e, (uint32_t)(127 + kMinScaleExp) << 23), (uint32_t)(127 + kMaxScaleExp) << 23);
}
__device__ __forceinline__ uint32_t inverse_bits(uint32_t scale) { return 0x7F000000u - scale; }

// Eight codes times their scale as bf16. The scale is a power of two, so that multiplying after
// the rounding to bf16 is exact too.
__device__ __forceinline__ uint4 e4m3_bf16x8(uint2 w, uint32_t scale) {
    const uint32_t s = scale >> 16 | (scale & 0xFFFF0000u);
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t four = e < 2 ? w.x : w.y;
        const uint32_t h = e & 1 ? e4m3x2_f16x2_hi(four) : e4m3x2_f16x2(four);
        out[e] = bf2_mul(pack_bf16(f16_lo(h), f16_hi(h)), s);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// The least scale with which a value of these fp32 bits (finite, not negative) fits: 448 is
// 1.75 x 2^8.
__device__ __forceinline__ uint32_t scale_for(uint32_t value) {
    const int e = (int)(value >> 23) - 127 - 8 + ((value & 0x7FFFFFu) > 0x600000u);
    return (uint32_t)(127 + min(max(e, kMinScaleExp), kMaxScaleExp)) << 23;
}

}  // namespace sc

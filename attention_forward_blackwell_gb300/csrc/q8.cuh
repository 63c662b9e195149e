// Caches held in 8 bits: what the kernels that write and read them share
// (cache_q8.cu, decode_q8.cu).
//
// A value is an e4m3 code times the scale of its block of keys and head.  The
// conversions of the machine do the rounding: e4m3 to fp16 is exact, and
// cvt.rn.satfinite rounds fp32 to the nearest code, ties to even.
#pragma once

#include <cstdint>

namespace fa {

// Two codes (the lower 16 bits) as fp16.
__device__ __forceinline__ uint32_t q8_halves(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
// The upper two of four codes.
__device__ __forceinline__ uint32_t q8_halves_up(uint32_t four) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(four));
    return r;
}
__device__ __forceinline__ float2 halves_to_floats(uint32_t h) {
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}
// Four codes as fp32, and four fp32 values rounded to codes.
__device__ __forceinline__ void q8_floats(uint32_t four, float (&x)[4]) {
    const float2 a = halves_to_floats(q8_halves(four)), b = halves_to_floats(q8_halves_up(four));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}
__device__ __forceinline__ uint32_t q8_codes(float x0, float x1, float x2, float x3) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
}

constexpr int kScaleLow = -54, kScaleHigh = 54;   // exponents of scales

// The smallest 2^e, kScaleLow <= e <= kScaleHigh, with 448 2^e no less than the
// root of `square`.  (448 2^e)^2 = 49/64 2^(18 + 2 e): compared with the square
// itself, part 2^power with part in [1/2, 1), nothing is rounded.  The limits keep
// the squares within fp32; a reach below 2^-63 counts as none.
__device__ __forceinline__ float q8_scale(float square) {
    const uint32_t bits = __float_as_uint(square);
    if (!(square >= 0x1p-126f)) return __uint_as_float((uint32_t)(127 + kScaleLow) << 23);
    const int y = (int)(bits >> 23) - 126 - 18;                            // power - 18
    const bool over = (bits & 0x7fffffu) > 0x440000u;                      // part > 49/64
    int e = (y + 1) >> 1;                                                  // (rounds down)
    if ((y & 1) == 0 && over) ++e;
    e = e < kScaleLow ? kScaleLow : (e > kScaleHigh ? kScaleHigh : e);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

}  // namespace fa

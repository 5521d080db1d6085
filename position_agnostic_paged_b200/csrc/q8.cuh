// q8.cuh -- e4m3 codes: conversions and the power-of-two scale rule of the 8-bit pool.
#pragma once

#include "common.cuh"

namespace lazy {

constexpr float kCodeMax = 448.f;          // largest e4m3 value: 1.75 * 2^8
constexpr float kScaleMin = 0x1p-126f;     // smallest scale a write makes

// Four codes (one register, lowest byte first) as two f16 pairs; every e4m3 value is an f16 value.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float &x0, float &x1) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
        : "=f"(x0), "=f"(x1)
        : "r"(h));
}
// Four values as codes, rounded to nearest even; values beyond +-448 (infinities too) become +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t f32_to_codes(float x0, float x1, float x2, float x3) {
    uint32_t w;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
        " mov.b32 %0, {a, b};\n}\n"
        : "=r"(w)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return w;
}
// Least power of two s >= 2^-126 with amax <= 448 s (amax finite, >= 0).
__device__ __forceinline__ float q8_scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    // amax = f 2^e with 1 <= f < 2: s = 2^(e - 8) if f <= 1.75, else 2^(e - 7)
    const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

}  // namespace lazy

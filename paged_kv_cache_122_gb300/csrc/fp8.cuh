// e4m3 values (1 sign, 4 exponent and 3 significand bits, largest 448, one NaN
// and no infinity) and the power-of-two scales of the 8-bit cache.
#pragma once

#include "common.cuh"

namespace pk {

constexpr float kScaleMin = 0x1p-64f, kScaleMax = 0x1p64f;   // scales the kernels accept

PK_DEV bool scale_ok(float s) { return s >= kScaleMin && s <= kScaleMax; }   // false for NaN

// Two floats to two e4m3 bytes (lo in the low byte), nearest even, values
// beyond 448 to +-448, NaN to NaN.
PK_DEV uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 bytes to two floats (exact; through fp16, whose range holds theirs).
PK_DEV void e4m3x2_to_float(uint32_t two, float &lo, float &hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(h));
}

PK_DEV uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | (e4m3x2(c, d) << 16); }

PK_DEV void e4m3x4_to_float(uint32_t w, float (&f)[4]) {
    e4m3x2_to_float(w & 0xffffu, f[0], f[1]);
    e4m3x2_to_float(w >> 16, f[2], f[3]);
}

// The smallest power of two s, 2^-64 <= s <= 2^64, with m2 <= (448 s)^2: with
// m2 = g 2^k, 1 <= g < 2, and 448^2 = 1.53125 * 2^17, that is the smallest e
// with 2 e >= k - 17 + (g > 1.53125).  Only the exponent of the sum of
// squares is looked at, so no square root rounds.
PK_DEV float needed_scale(float m2) {
    const uint32_t b = __float_as_uint(m2);
    const int k = static_cast<int>(b >> 23) - 127 + ((b & 0x7fffffu) > 4456448u);   // 0.53125 * 2^23
    const int e = min(64, max(-64, (k - 16) >> 1));
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace pk

// MXFP4 rounding shared by the quantiser and the 4-bit product: 32 values share
// an E8M0 scale byte X (scale 2^(X-127)), each becomes an E2M1 code (sign, two
// exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6).
#pragma once

#include "common.cuh"

namespace moe {

// Scale byte of a block whose largest magnitude is amax:
//   X - 127 = floor(log2 amax) - 2     (2: the exponent of E2M1's largest value)
// read off amax's exponent bits; at least 0 (amax below 2^-124 uses 2^-127).
// A block that holds a NaN or an infinity gets 255, the NaN scale: `bits` is
// the largest of the magnitudes' bit patterns, so both lead to exponent 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t bits) {
    const uint32_t ex = bits >> 23;
    return ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
}
// 2^(127 - X), exact for every X that mx_scale_byte gives a finite block (0..252).
__device__ __forceinline__ float mx_inv_scale(uint32_t X) { return __uint_as_float((254u - X) << 23); }
__device__ __forceinline__ float mx_scale(uint32_t X) {
    return X == 0u ? __uint_as_float(0x00400000u) : X == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(X << 23);
}

// Eight values times inv (exact: a power of two, results below 8) to eight E2M1
// codes, value i in bits 4i..4i+3.  The conversion rounds to nearest, ties to
// the even code, and takes magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float inv) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0] * inv), "f"(v[1] * inv), "f"(v[2] * inv), "f"(v[3] * inv), "f"(v[4] * inv), "f"(v[5] * inv),
          "f"(v[6] * inv), "f"(v[7] * inv));
    return w;
}

// The values of eight codes (packed as by mx_codes8) under scale s: exact in
// float, two significant bits times a power of two.
__device__ __forceinline__ void mx_values8(uint32_t w, float s, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = *(const __half2*)&h[i];
        v[2 * i] = __low2float(p) * s;
        v[2 * i + 1] = __high2float(p) * s;
    }
}

}  // namespace moe

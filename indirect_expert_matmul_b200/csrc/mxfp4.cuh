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

// Largest magnitude bit pattern of eight values, then of the four lanes (4i ..
// 4i+3) that hold one block of 32; `mask` names the lanes taking part.
__device__ __forceinline__ uint32_t mx_block_bits(const float (&v)[8], unsigned mask) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(mask, m, 1));
    return max(m, __shfl_xor_sync(mask, m, 2));
}

// Eight consecutive elements at p (16-byte aligned when VEC) as float.
template <bool VEC>
__device__ __forceinline__ void mx_load8(const void* p, int type, float (&e)[8]) {
    if (type == MOE_F32) {
        const float* f = (const float*)p;
        if (VEC) {
            const float4 a = __ldg((const float4*)f), b = __ldg((const float4*)f + 1);
            e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w;
            e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = __ldg(f + i);
        }
        return;
    }
    uint32_t w[4];
    if (VEC) {
        const uint4 v = __ldg((const uint4*)p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint16_t* h = (const uint16_t*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(h + 2 * i) | (uint32_t)__ldg(h + 2 * i + 1) << 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (type == MOE_BF16) {
            e[2 * i] = __uint_as_float(w[i] << 16);
            e[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            e[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xffffu)));
            e[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
        }
    }
}

}  // namespace moe

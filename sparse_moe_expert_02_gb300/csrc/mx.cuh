// Microscaled 4-bit floating point (MXFP4 of the OCP Microscaling Formats
// specification): blocks of 32 columns, one E8M0 scale 2^(s-127) a block,
// E2M1 elements (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a
// byte with the even column in the low half.
//
//   e = floor(log2(amax)) - 2 (2 = the exponent of E2M1's largest binade),
//       at least -127;  s = e + 127
//   code = E2M1 of v * 2^-e, round to nearest even, saturating
//
// A block of zeros takes s = 127 (scale 1); a block that holds an infinity
// or a NaN takes s = 255 (E8M0's NaN), and all of it reads back as NaN.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMxBlock = 32;  // columns that share a scale

// Scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const uint32_t ex = amax_bits >> 23;  // biased exponent: floor(log2) + 127 (0: below 2^-126)
    if (amax_bits == 0) return 127u;
    if (ex == 255u) return 255u;
    return ex > 2u ? ex - 2u : 0u;
}
// 2^-e, the factor that takes values to codes; s != 255.
__device__ __forceinline__ float mx_inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^(s-127); s = 0 is the subnormal 2^-127, s = 255 a NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
    return s == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(s ? s << 23 : 0x00400000u);
}
// Two values to one byte of codes, a in the low half.
__device__ __forceinline__ uint32_t mx_codes(float a, float b) {
    uint16_t r;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n mov.b16 %0, {t, 0};\n}\n" : "=h"(r) : "f"(a), "f"(b));
    return r;
}
// The four bytes of a word as eight code values, pairs of fp16 (exact).
__device__ __forceinline__ void mx_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

}  // namespace moe

// 4-bit codes as bf16, for the products with 4-bit weights.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

// Eight codes (a word, the first in the lowest four bits) as bf16 pairs of
// code - zero; z: 128 + zero in both halves.  bf16 counts in ones from 128 to
// 256, so 0x4300 + code is 128 + code, and the difference is exact.
__device__ __forceinline__ void int4_pairs(uint32_t w, __nv_bfloat162 z, uint32_t (&o)[4]) {
    const uint32_t h = w >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // byte j of w and of w >> 4: their low halves are codes 2j and 2j + 1
        const uint32_t v = (__byte_perm(w, h, (4 + j) << 8 | j) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*(const __nv_bfloat162*)&v, z);
        o[j] = *(const uint32_t*)&d;
    }
}
__device__ __forceinline__ __nv_bfloat162 int4_zero(int zero) {
    const uint32_t v = (0x4300u + (uint32_t)zero) * 0x10001u;
    return *(const __nv_bfloat162*)&v;
}

// Values from fp32 scales as bf16, rounded once.  code - zero times a scale may
// need 28 bits: rounded to 24 it can land on a tie of bf16 that it is not, and
// the rounding from there would go to the even side.  int4_value: 32 bits that
// round to the bf16 nearest to d s; the residual, exact, says on which side of
// the tie the product lies.  Asked for each value, the product of 2047 rows by
// 4096 x 4096 codes took 128 us instead of 68; asked only of scales of which
// some product lands there (one in some ten thousand), 71.
__device__ __forceinline__ float int4_value(float d, float s) {
    const float p = d * s;
    uint32_t b = __float_as_uint(p);
    if ((b & 0xFFFFu) == 0x8000u) {
        const float rest = fmaf(d, s, -p);
        if (rest != 0.0f) b += (rest > 0.0f) == (p > 0.0f) ? 1u : ~0u;
    }
    return __uint_as_float(b);
}
// (d and 2 d have the same digits, and powers of two round nothing)
__device__ __forceinline__ bool int4_on_ties(float s) {
    bool any = false;
#pragma unroll
    for (int d = 3; d < 16; d += 2) any |= (__float_as_uint((float)d * s) & 0xFFFFu) == 0x8000u;
    return any;
}

}  // namespace moe

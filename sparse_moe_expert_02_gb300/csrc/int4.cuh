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

}  // namespace moe

// Microscaled 4-bit floating point: quantise rows and read them back
// (moe_mx_quantize, moe_mx_dequantize; the format is in mx.cuh).
//
// Four lanes share a block of 32 columns, eight columns each: the block's
// amax is two shuffles away, a lane's codes are one 32-bit word, and a warp
// reads 512 bytes of bf16 and writes 128 bytes of codes in one piece.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

// Eight columns at col of a row of `cols` (columns past the end are zero).
template <bool VEC, typename T> __device__ __forceinline__ void load8(const T* row, int col, int cols, float* v) {
    if constexpr (VEC) {
        if constexpr (sizeof(T) == 2) {
            const uint4 q = __ldg((const uint4*)(row + col));
            const T* e = (const T*)&q;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 q = __ldg((const float4*)(row + col) + h);
                v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? to_f32(__ldg(row + col + i)) : 0.0f;
    }
}

template <bool VEC, typename T>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const T* __restrict__ x, int64_t ld, int64_t rows, int cols, int blocks,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const int64_t n = rows * blocks * 4;  // one unit: eight columns
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    // four lanes of a block run together, so whole quads leave the loop
    for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < n; u += step) {
        const int64_t blk = u >> 2, row = blk / blocks;
        const int col = (int)(blk - row * blocks) * kMxBlock + (int)(u & 3) * 8;
        float v[8];
        load8<VEC>(x + row * ld, col, cols, v);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        const uint32_t quad = 0xFu << (threadIdx.x & 28);
        m = max(m, __shfl_xor_sync(quad, m, 1));
        m = max(m, __shfl_xor_sync(quad, m, 2));
        const uint32_t sb = mx_scale_byte(m);
        const float f = sb == 255u ? 0.0f : mx_inv_scale(sb);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= mx_codes(v[2 * i] * f, v[2 * i + 1] * f) << (8 * i);
        if (sb == 255u) w = 0;
        *(uint32_t*)(q + blk * 16 + (u & 3) * 4) = w;
        if ((u & 3) == 0) s[blk] = (uint8_t)sb;
    }
}

template <bool VEC, typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t rows,
                                                            int cols, int blocks, T* __restrict__ out, int64_t ld) {
    const int64_t n = rows * blocks * 4;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < n; u += step) {
        const int64_t blk = u >> 2, row = blk / blocks;
        const int col = (int)(blk - row * blocks) * kMxBlock + (int)(u & 3) * 8;
        const float f = mx_scale(__ldg(s + blk));
        uint32_t h[4];
        mx_f16x2(__ldg((const uint32_t*)(q + blk * 16 + (u & 3) * 4)), h);
        T v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*(const __half2*)&h[i]);
            v[2 * i] = from_f32<T>(p.x * f);
            v[2 * i + 1] = from_f32<T>(p.y * f);
        }
        T* o = out + row * ld + col;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((uint4*)o)[i] = ((const uint4*)v)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < cols) o[i] = v[i];
        }
    }
}

unsigned grid_for(int64_t units) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(cdiv(units, 256), 152 * 8 * 4)); }

}  // namespace

cudaError_t launch_mx_quantize(const void* x, int x_elem, int64_t ld, int64_t rows, int cols, uint8_t* q, uint8_t* s,
                               cudaStream_t stream) {
    const int blocks = (int)cdiv(cols, kMxBlock);
    const unsigned grid = grid_for(rows * blocks * 4);
    const int eb = x_elem == kF32 ? 4 : 2;
    const bool vec = cols % kMxBlock == 0 && ((uintptr_t)x & 15) == 0 && (ld * eb) % 16 == 0;
#define MOE_Q(V, T) mx_quantize_kernel<V, T><<<grid, 256, 0, stream>>>((const T*)x, ld, rows, cols, blocks, q, s)
    if (x_elem == kF32) {
        if (vec) MOE_Q(true, float);
        else MOE_Q(false, float);
    } else {
        if (vec) MOE_Q(true, bf16);
        else MOE_Q(false, bf16);
    }
#undef MOE_Q
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int cols, void* out, int out_elem,
                                 int64_t ld, cudaStream_t stream) {
    const int blocks = (int)cdiv(cols, kMxBlock);
    const unsigned grid = grid_for(rows * blocks * 4);
    const int eb = out_elem == kF32 ? 4 : 2;
    const bool vec = cols % kMxBlock == 0 && ((uintptr_t)out & 15) == 0 && (ld * eb) % 16 == 0;
#define MOE_DQ(V, T) mx_dequantize_kernel<V, T><<<grid, 256, 0, stream>>>(q, s, rows, cols, blocks, (T*)out, ld)
    if (out_elem == kF32) {
        if (vec) MOE_DQ(true, float);
        else MOE_DQ(false, float);
    } else {
        if (vec) MOE_DQ(true, bf16);
        else MOE_DQ(false, bf16);
    }
#undef MOE_DQ
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe

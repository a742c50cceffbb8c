// Microscaled 4-bit floating point: quantise rows and read them back
// (moe_mx_quantize, moe_mx_dequantize; the format is in mx.cuh).
//
// Bound by HBM: 2 or 4 bytes in and 17/32 out per element, or the reverse.
// Aligned rows: four lanes share a block of 32 columns, eight columns each:
// the block's amax is two shuffles away, a lane's codes are one 32-bit word,
// and a warp reads 512 bytes of bf16 and writes 128 bytes of codes in one
// piece; a thread has two such units in flight (16384 x 4096 bf16, quantised
// and read back: 62 us, 5.4 TB/s; with one 94, with four 64).  Rows that lie
// one after the other are one long row, which saves a division per unit.
// Other rows (any alignment, a ragged last block): a warp takes a block, a
// column a lane, so that its loads and stores stay in one piece all the same.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

// Loads go past L1 (each byte is read once) and not through the read-only path:
// the kernels start while the one before them, which may write what they read,
// ends (common.cuh, programmatic dependent launch).
constexpr int kUnroll = 2;

// Eight columns as they lie in memory: their largest magnitude's bits, and
// their codes.
template <typename T> struct Eight;
template <> struct Eight<bf16> {
    uint4 q;
    __device__ __forceinline__ void load(const bf16* p) { q = __ldcg((const uint4*)p); }
    __device__ __forceinline__ uint32_t amax() const {  // two at a time, as 16-bit integers: NaNs count
        const uint32_t m = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu), __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
        return max(m << 16, m & 0xFFFF0000u);
    }
    __device__ __forceinline__ uint32_t codes(float f) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) c |= mx_codes(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f) << (8 * i);
        return c;
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcg((const float4*)p);
        b = __ldcg((const float4*)p + 1);
    }
    __device__ __forceinline__ uint32_t amax() const {
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ uint32_t codes(float f) const {
        return mx_codes(a.x * f, a.y * f) | mx_codes(a.z * f, a.w * f) << 8 | mx_codes(b.x * f, b.y * f) << 16 | mx_codes(b.z * f, b.w * f) << 24;
    }
};

// n units of eight columns (whole blocks: a multiple of four); per: units of a row.
template <typename T>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const T* __restrict__ x, int64_t ld, int64_t n, int64_t per,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    pdl_wait_then_release();
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const bool flat = n == per;
    for (int64_t w0 = (int64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~31); w0 < n; w0 += kUnroll * step) {
        // whole warps stay together; past the end a lane repeats the last unit of its place in a block
        const int64_t u0 = w0 + (threadIdx.x & 31);
        Eight<T> v[kUnroll];
        uint32_t m[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t u = min(u0 + j * step, n - 4 + (threadIdx.x & 3));
            const int64_t row = flat ? 0 : u / per;
            v[j].load(x + row * ld + (u - row * per) * 8);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) m[j] = v[j].amax();
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 1));
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 2));
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t u = u0 + j * step;
            const uint32_t sb = mx_scale_byte(m[j]);
            const uint32_t c = v[j].codes(mx_inv_scale(sb));  // (of a block with a NaN: not used)
            if (u < n) {
                *(uint32_t*)(q + u * 4) = sb == 255u ? 0u : c;
                if ((u & 3) == 0) s[u >> 2] = (uint8_t)sb;
            }
        }
    }
}

// h = silu(g) * u, quantised: units of eight columns of one long row.
__global__ void __launch_bounds__(256) mx_swiglu_kernel(const float* __restrict__ g, const float* __restrict__ u, int64_t n,
                                                        uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t w0 = (int64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~31); w0 < n; w0 += step) {
        const int64_t i = min(w0 + (threadIdx.x & 31), n - 4 + (threadIdx.x & 3));
        Eight<float> a, b;
        a.load(g + i * 8);
        b.load(u + i * 8);
        a.a = make_float4(swiglu(a.a.x, b.a.x), swiglu(a.a.y, b.a.y), swiglu(a.a.z, b.a.z), swiglu(a.a.w, b.a.w));
        a.b = make_float4(swiglu(a.b.x, b.b.x), swiglu(a.b.y, b.b.y), swiglu(a.b.z, b.b.z), swiglu(a.b.w, b.b.w));
        uint32_t m = a.amax();
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t sb = mx_scale_byte(m);
        const uint32_t c = a.codes(mx_inv_scale(sb));
        if (w0 + (threadIdx.x & 31) < n) {
            *(uint32_t*)(q + i * 4) = sb == 255u ? 0u : c;
            if ((i & 3) == 0) s[i >> 2] = (uint8_t)sb;
        }
    }
}

// n blocks, a warp each.
template <typename T>
__global__ void __launch_bounds__(256) mx_quantize_any_kernel(const T* __restrict__ x, int64_t ld, int64_t n, int cols, int blocks,
                                                              uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t b0 = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); b0 < n; b0 += kUnroll * step) {
        float v[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t b = b0 + j * step;
            v[j] = 0.0f;
            if (b < n) {
                const int64_t row = b / blocks;
                const int col = (int)(b - row * blocks) * kMxBlock + lane;
                if (col < cols) v[j] = to_f32(__ldcg(x + row * ld + col));
            }
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t b = b0 + j * step;
            if (b >= n) break;
            const uint32_t sb = mx_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7FFFFFFFu));
            const float a = sb == 255u ? 0.0f : v[j] * mx_inv_scale(sb);
            const uint32_t c = mx_codes(a, __shfl_down_sync(0xffffffffu, a, 1));
            if ((lane & 1) == 0) q[b * 16 + (lane >> 1)] = (uint8_t)c;
            if (lane == 0) s[b] = (uint8_t)sb;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* s, int64_t n,
                                                            int64_t per, T* __restrict__ out, int64_t ld) {
    pdl_wait_then_release();
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const bool flat = n == per;
    for (int64_t u0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u0 < n; u0 += kUnroll * step) {
        uint32_t w[kUnroll], sb[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t u = min(u0 + j * step, n - 1);
            w[j] = __ldcg((const uint32_t*)(q + u * 4));
            sb[j] = s[u >> 2];  // by way of L1: four warps share a sector
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t u = u0 + j * step;
            const float f = mx_scale(sb[j]);
            uint32_t h[4];
            mx_f16x2(w[j], h);
            alignas(16) T v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = __half22float2(*(const __half2*)&h[i]);
                v[2 * i] = from_f32<T>(p.x * f);
                v[2 * i + 1] = from_f32<T>(p.y * f);
            }
            if (u < n) {
                const int64_t row = flat ? 0 : u / per;
                T* o = out + row * ld + (u - row * per) * 8;
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((uint4*)o)[i] = ((const uint4*)v)[i];
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_any_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t n,
                                                                int cols, int blocks, T* __restrict__ out, int64_t ld) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t b0 = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); b0 < n; b0 += kUnroll * step) {
        uint32_t w[kUnroll], sb[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t b = b0 + j * step;
            if (b < n) {
                w[j] = __ldcg(q + b * 16 + (lane >> 1));
                sb[j] = __ldcg(s + b);
            }
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int64_t b = b0 + j * step;
            if (b >= n) break;
            uint32_t h[4];
            mx_f16x2(w[j], h);
            const float2 p = __half22float2(*(const __half2*)&h[0]);
            const int64_t row = b / blocks;
            const int col = (int)(b - row * blocks) * kMxBlock + lane;
            if (col < cols) out[row * ld + col] = from_f32<T>((lane & 1 ? p.y : p.x) * mx_scale(sb[j]));
        }
    }
}

// Blocks of 256 threads for `threads` units: up to eight a SM resident, a few rounds.
unsigned grid_for(int64_t threads) {
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(cdiv(threads, 256), 152 * 8 * 4));
}

struct Shape {
    bool vec;
    int blocks;
    int64_t units, per;  // vec: units of eight columns, and of a row (all of them: one long row)
    unsigned grid;
};
Shape shape_of(const void* p, int eb, int64_t ld, int64_t rows, int cols) {
    Shape h;
    h.blocks = (int)cdiv(cols, kMxBlock);
    h.vec = cols % kMxBlock == 0 && ((uintptr_t)p & 15) == 0 && (ld * eb) % 16 == 0;
    h.units = rows * h.blocks * 4;
    h.per = ld == cols || rows == 1 ? h.units : (int64_t)h.blocks * 4;
    h.grid = grid_for(h.vec ? h.units : rows * h.blocks * 32);
    return h;
}

}  // namespace

cudaError_t launch_mx_quantize(const void* x, int x_elem, int64_t ld, int64_t rows, int cols, uint8_t* q, uint8_t* s,
                               cudaStream_t stream) {
    cudaError_t e;
    const Shape h = shape_of(x, x_elem == kF32 ? 4 : 2, ld, rows, cols);
    const int64_t n = rows * h.blocks;
    if (x_elem == kF32) {
        if (h.vec) e = launch_kernel(mx_quantize_kernel<float>, dim3(h.grid), dim3(256), 0, stream, 1, (const float*)x, ld, h.units, h.per, q, s);
        else e = launch_kernel(mx_quantize_any_kernel<float>, dim3(h.grid), dim3(256), 0, stream, 1, (const float*)x, ld, n, cols, h.blocks, q, s);
    } else {
        if (h.vec) e = launch_kernel(mx_quantize_kernel<bf16>, dim3(h.grid), dim3(256), 0, stream, 1, (const bf16*)x, ld, h.units, h.per, q, s);
        else e = launch_kernel(mx_quantize_any_kernel<bf16>, dim3(h.grid), dim3(256), 0, stream, 1, (const bf16*)x, ld, n, cols, h.blocks, q, s);
    }
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_mx_swiglu(const float* g, const float* u, int64_t n, uint8_t* q, uint8_t* s, cudaStream_t stream) {
    mx_swiglu_kernel<<<grid_for(n / 8), 256, 0, stream>>>(g, u, n / 8, q, s);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int cols, void* out, int out_elem,
                                 int64_t ld, cudaStream_t stream) {
    cudaError_t e;
    const Shape h = shape_of(out, out_elem == kF32 ? 4 : 2, ld, rows, cols);
    const int64_t n = rows * h.blocks;
    if (out_elem == kF32) {
        if (h.vec) e = launch_kernel(mx_dequantize_kernel<float>, dim3(h.grid), dim3(256), 0, stream, 1, q, s, h.units, h.per, (float*)out, ld);
        else e = launch_kernel(mx_dequantize_any_kernel<float>, dim3(h.grid), dim3(256), 0, stream, 1, q, s, n, cols, h.blocks, (float*)out, ld);
    } else {
        if (h.vec) e = launch_kernel(mx_dequantize_kernel<bf16>, dim3(h.grid), dim3(256), 0, stream, 1, q, s, h.units, h.per, (bf16*)out, ld);
        else e = launch_kernel(mx_dequantize_any_kernel<bf16>, dim3(h.grid), dim3(256), 0, stream, 1, q, s, n, cols, h.blocks, (bf16*)out, ld);
    }
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

// 4-bit codes with a scale per group of columns: quantise rows and read them
// back (moe_int4_quantize, moe_int4_dequantize).
//   value = scale * (code - zero),  zero 8 where none is stored.
//
// Weights are prepared once, so the simplest form that keeps loads in one
// piece: a warp takes a group, a lane one to four of its columns.  Codes are
// the nearest to the exact quotient by the stored scale (ties to even): the
// rounded quotient's residuals to its neighbours, each one fused multiply-add
// and so exact in sign, decide.
//
// Measured, 65536 x 4096 in groups of 128 with zero points: quantising 715 to 740
// us (bf16 in: 100 at the copy's rate; a warp has one group, 128 loads of an
// element, on its way), reading back 124 to 132 as bf16 (100), 285 as fp32 (180).
#include <algorithm>

#include "common.cuh"
#include "int4.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Nearest integer to v / s for s > 0, ties to even, within [-16, 16].
__device__ __forceinline__ int nearest(float v, float s) {
    const float q = fminf(fmaxf(v / s, -16.0f), 16.0f);
    int n = __float2int_rn(q);
    // v against the midpoints on both sides of n (n +- 1/2 is exact, and so is the residual's sign)
    const float above = fmaf(-((float)n + 0.5f), s, v), below = fmaf(-((float)n - 0.5f), s, v);
    if (above > 0.0f || (above == 0.0f && (n & 1))) ++n;
    else if (below < 0.0f || (below == 0.0f && (n & 1))) --n;
    return n;
}

template <typename T, typename TS>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* x, int64_t ld, int64_t rows, int cols, int group, uint8_t* codes, TS* scales, uint8_t* zeros) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, nb = (cols + group - 1) / group;
    const int64_t units = rows * nb, step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const int64_t r = u / nb;
        const int c0 = (int)(u - r * nb) * group, n = min(group, cols - c0);  // n is even: cols is
        // a lane holds pairs of columns: 2 lane + 64 j
        float v[4];
        float lo = 0.0f, hi = 0.0f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 2 * lane + 64 * (j >> 1) + (j & 1);
            v[j] = c < n ? to_f32(x[r * ld + c0 + c]) : 0.0f;
            bad |= !(fabsf(v[j]) < __int_as_float(0x7F800000));
            lo = fminf(lo, v[j]);
            hi = fmaxf(hi, v[j]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        bad = __any_sync(0xffffffffu, bad);
        TS st = from_f32<TS>(bad ? __int_as_float(0x7FC00000) : zeros ? hi / 15.0f - lo / 15.0f : fmaxf(hi, -lo) / 7.0f);
        float s = to_f32(st);
        if (s == 0.0f) {  // zeros, or all below half of the smallest scale
            st = from_f32<TS>(1.0f);
            s = 1.0f;
        }
        int z = 8;
        if (zeros) z = bad ? 0 : min(max(nearest(-lo, s), 0), 15);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = 2 * lane + 64 * j;
            if (c >= n) continue;
            int q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) q[i] = bad ? 0 : min(max(nearest(v[2 * j + i], s) + z, 0), 15);
            codes[r * (cols / 2) + (c0 + c) / 2] = (uint8_t)(q[0] | q[1] << 4);
        }
        if (lane == 0) {
            scales[u] = st;
            if (zeros) zeros[u] = (uint8_t)z;
        }
    }
}

// A thread reads back sixteen columns (they lie in one group).
template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Int4 q, int64_t rows, int cols, T* out, int64_t ld, bool vec) {
    pdl_wait_then_release();
    const int per = cols / 16, nb = (cols + q.group - 1) / q.group;
    const int64_t units = rows * per, step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
        const int64_t r = u / per;
        const int c = (int)(u - r * per) * 16;
        const int64_t at = r * nb + c / q.group;
        const float s = q.scale_elem == kF32 ? ((const float*)q.scales)[at] : to_f32(((const bf16*)q.scales)[at]);
        const int z = q.zeros ? q.zeros[at] : 8;
        const uint2 w = *(const uint2*)(q.codes + u * 8);
        T* o = out + r * ld + c;
        __align__(16) T v[16];
        auto code = [&](int j) { return (float)((int)(((j < 8 ? w.x : w.y) >> (4 * (j & 7))) & 15u) - z); };
        if (sizeof(T) == 2 && q.scale_elem == kF32 && int4_on_ties(s)) {  // (with bf16 scales 13 bits hold a product)
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = from_f32<T>(int4_value(code(j), s));
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = from_f32<T>(code(j) * s);
        }
        if (vec) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); ++j) ((uint4*)o)[j] = ((const uint4*)v)[j];
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = v[j];
        }
    }
}

unsigned blocks_for(int64_t units, int num_sms) { return (unsigned)std::min<int64_t>(std::max<int64_t>(units, 1), 16 * num_sms); }

}  // namespace

cudaError_t launch_int4_quantize(const void* x, int x_elem, int64_t ld, int64_t rows, int cols, const Int4& q, int num_sms, cudaStream_t s) {
    const dim3 grid(blocks_for(cdiv(rows * cdiv(cols, q.group), kThreads / 32), num_sms)), block(kThreads);
    uint8_t *codes = const_cast<uint8_t*>(q.codes), *zeros = const_cast<uint8_t*>(q.zeros);
    cudaError_t e;
#define MOE_Q(T, TS) launch_kernel(quantize_kernel<T, TS>, grid, block, 0, s, 1, (const T*)x, ld, rows, cols, q.group, codes, (TS*)const_cast<void*>(q.scales), zeros)
    if (x_elem == kF32) e = q.scale_elem == kF32 ? MOE_Q(float, float) : MOE_Q(float, bf16);
    else e = q.scale_elem == kF32 ? MOE_Q(bf16, float) : MOE_Q(bf16, bf16);
#undef MOE_Q
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_int4_dequantize(const Int4& q, int64_t rows, int cols, void* out, int out_elem, int64_t ld, int num_sms, cudaStream_t s) {
    const dim3 grid(blocks_for(cdiv(rows * (cols / 16), kThreads), num_sms)), block(kThreads);
    const bool vec = ((uintptr_t)out & 15) == 0 && ld * (out_elem == kF32 ? 4 : 2) % 16 == 0;
    const cudaError_t e = out_elem == kF32 ? launch_kernel(dequantize_kernel<float>, grid, block, 0, s, 1, q, rows, cols, (float*)out, ld, vec)
                                           : launch_kernel(dequantize_kernel<bf16>, grid, block, 0, s, 1, q, rows, cols, (bf16*)out, ld, vec);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

// The whole layer for a few tokens (moe_forward_few).
//
// A warp per output value: logits, then (after the top-k) the activations of
// every (token, chosen expert) pair, then the outputs, each a dot product
// over one weight row, read straight from the expert's matrices: no
// permutation and no copies of x.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__device__ __forceinline__ float weight_at(const void* w, const void* scale, int dtype, int64_t row, int rows, int col, int cols) {
    const int64_t at = row * cols + col;
    if (dtype == MOE_F32) return __ldg((const float*)w + at);
    if (dtype == MOE_BF16) return __bfloat162float(__ldg((const bf16*)w + at));
    if (dtype == MOE_FP8_E4M3_B128) {
        const int64_t g = row / rows, r = row - g * rows;
        return e4m3_to_f32(__ldg((const uint8_t*)w + at)) *
               __ldg((const float*)scale + (g * (rows / 128) + r / 128) * (cols / 128) + col / 128);
    }
    uint32_t h[4];
    mx_f16x2((uint32_t)__ldg((const uint8_t*)w + at / 2), h);
    const float2 v = __half22float2(*(const __half2*)&h[0]);
    return ((col & 1) ? v.y : v.x) * mx_scale(__ldg((const uint8_t*)scale + at / kMxBlock));
}

__global__ void few_logits_kernel(const FewParams p) {
    const int e = blockIdx.x, t = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (t >= p.T) return;
    float s = 0.0f;
    for (int c = lane; c < p.D; c += 32) {
        const float x = p.dtype == MOE_F32 ? ((const float*)p.x)[(int64_t)t * p.D + c] : __bfloat162float(((const bf16*)p.x)[(int64_t)t * p.D + c]);
        const float w = p.dtype == MOE_F32 ? ((const float*)p.w_router)[(int64_t)e * p.D + c] : __bfloat162float(((const bf16*)p.w_router)[(int64_t)e * p.D + c]);
        s = fmaf(x, w, s);
    }
    s = warp_sum(s);
    if (lane == 0) p.logits[(int64_t)t * p.E + e] = s + (p.b_router ? p.b_router[e] : 0.0f);
}

// Rows as the expert products read them: fp32 of x (from_x) or of h in place.
__global__ void few_as_read_kernel(const FewParams p, float* v, int rows, int cols, int from_x) {
    const int g = p.dtype == MOE_FP8_E4M3_B128 ? 128 : 32;
    const int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (int64_t)rows * cols / g) return;
    float a[4] = {}, m = 0.0f;
    for (int j = 0; j < g / 32; ++j) {
        const int64_t at = i * g + j * 32 + lane;
        a[j] = !from_x ? v[at] : p.dtype == MOE_F32 ? ((const float*)p.x)[at] : __bfloat162float(((const bf16*)p.x)[at]);
        m = fmaxf(m, fabsf(a[j]));
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int j = 0; j < g / 32; ++j) {
        float r = a[j];
        if (p.dtype == MOE_FP8_E4M3_B128) {
            r = m > 0 ? e4m3_to_f32(f32_to_e4m3(r * (448.0f / m))) * (m / 448.0f) : 0.0f;
        } else if (p.dtype == MOE_MXFP4) {
            const uint32_t s = mx_scale_byte(__float_as_uint(m));
            uint32_t h[4];
            mx_f16x2(mx_codes(r * (s == 255 ? 0.0f : mx_inv_scale(s)), 0.0f), h);
            r = __half2float(((const __half*)h)[0]) * mx_scale(s);
        }
        v[i * g + j * 32 + lane] = r;
    }
}

__device__ __forceinline__ int expert_of(const FewParams& p, int t, int j) {
    if (j == p.k) return p.E;
    const int e = p.blob[t * p.k + j];
    return min(max(e, 0), p.E - 1);
}

__global__ void few_gateup_kernel(const FewParams p) {
    const int64_t u = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (u >= (int64_t)p.T * (p.k + 1) * p.I) return;
    const int pair = (int)(u / p.I), i = (int)(u % p.I), t = pair / (p.k + 1);
    const int64_t row = (int64_t)expert_of(p, t, pair % (p.k + 1)) * p.I + i;
    float a = 0.0f, b = 0.0f;
    for (int c = lane; c < p.D; c += 32) {
        const float x = p.xr[(int64_t)t * p.D + c];
        a = fmaf(weight_at(p.w_gate, p.s_gate, p.dtype, row, p.I, c, p.D), x, a);
        b = fmaf(weight_at(p.w_up, p.s_up, p.dtype, row, p.I, c, p.D), x, b);
    }
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) p.h[u] = swiglu(a, b);
}

template <typename OT>
__global__ void few_down_kernel(const FewParams p) {
    const int64_t u = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (u >= (int64_t)p.T * p.D) return;
    const int t = (int)(u / p.D), d = (int)(u % p.D);
    float out = 0.0f;
    for (int jj = 0; jj <= p.k; ++jj) {
        const int j = jj == 0 ? p.k : jj - 1;  // the shared expert first
        const int64_t row = (int64_t)expert_of(p, t, j) * p.D + d;
        float y = 0.0f;
        for (int c = lane; c < p.I; c += 32) {
            const float w = p.dtype == MOE_BF16 ? (p.down_f16 ? __half2float(((const f16*)p.w_down)[row * p.I + c])
                                                              : __bfloat162float(((const bf16*)p.w_down)[row * p.I + c]))
                                                : weight_at(p.w_down, p.s_down, p.dtype, row, p.D, c, p.I);
            y = fmaf(w, p.h[((int64_t)t * (p.k + 1) + j) * p.I + c], y);
        }
        const float g = j == p.k ? 1.0f : __int_as_float(p.blob[p.T * p.k + t * p.k + j]);
        out = fmaf(g, warp_sum(y), out);
    }
    if (lane == 0) ((OT*)p.out)[u] = from_f32<OT>(out);
}

}  // namespace

cudaError_t launch_few(const FewParams& p, cudaStream_t s) {
    few_logits_kernel<<<p.E, 32 * kFewMax, 0, s>>>(p);
    cudaError_t e = launch_topk(p.logits, 1, nullptr, nullptr, p.T, p.E, p.k, p.blob, p.err, s);
    if (e != cudaSuccess) return e;
    const int pairs = p.T * (p.k + 1);
    few_as_read_kernel<<<(unsigned)cdiv((int64_t)p.T * p.D / 32, 4), 128, 0, s>>>(p, p.xr, p.T, p.D, 1);
    few_gateup_kernel<<<(unsigned)cdiv((int64_t)pairs * p.I, 4), 128, 0, s>>>(p);
    if (p.dtype == MOE_FP8_E4M3_B128 || p.dtype == MOE_MXFP4)
        few_as_read_kernel<<<(unsigned)cdiv((int64_t)pairs * p.I / 32, 4), 128, 0, s>>>(p, p.h, pairs, p.I, 0);
    const unsigned grid = (unsigned)cdiv((int64_t)p.T * p.D, 4);
    if (p.out_elem == kF32) few_down_kernel<float><<<grid, 128, 0, s>>>(p);
    else few_down_kernel<bf16><<<grid, 128, 0, s>>>(p);
    count_launches(5);
    return cudaGetLastError();
}

}  // namespace moe

// The experts' activation and its gradient (moe_swiglu, moe_swiglu_grad):
//   h  = w s g u,                  s = 1 / (1 + e^-g)
//   du = w dh s g,   dg = w dh u s (1 + g (1 - s)),   dw = sum_i dh s g u
// for rows of I elements with an optional factor w per row.
//
// Bound by HBM: three tensors forward, five backward, each element once.
// A row belongs to a team of threads, a warp where there are rows enough and a
// block where there are not, which goes over it eight elements a thread at a
// time; dw is then a sum within the team, always in the same order.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// V elements of a row: 16-byte loads of V = 8 (two of them in fp32), or one.
template <typename T, int V> struct Pack {
    float v[V];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V == 1) {
            v[0] = to_f32(*p);
        } else if constexpr (sizeof(T) == 4) {
            const float4 a = __ldcg((const float4*)p), b = __ldcg((const float4*)p + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 q = __ldcg((const uint4*)p);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (V == 1) {
            *p = from_f32<T>(v[0]);
        } else if constexpr (sizeof(T) == 4) {
            ((float4*)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            ((float4*)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *(const uint32_t*)&h;
            }
            *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// s = 1 / (1 + e^-g) and 1 - s, both from e^-|g|, which neither overflows nor
// cancels (e^89 is past fp32's range, but -89 e^-89 is not).  FULL: to a few
// ulp, where h, dgate and dup stay in fp32; else by the hardware's exponential
// and reciprocal, some 2^-21 about zero, below a 2000th of a bf16 step.  dweight
// is fp32 all the same, but a sum of bf16 products: 1.3e-7 of its rms off 64 bits
// either way (1.1e-7 by tensor operations in 32 bits), and the full form takes 150
// us instead of 140 for 81920 x 1024, 21 instead of 17 for 4097 x 1000.
template <bool FULL> __device__ __forceinline__ void sigmoid(float g, float& s, float& rest) {
    const float e = FULL ? expf(-fabsf(g)) : __expf(-fabsf(g));
    const float r = FULL ? 1.0f / (1.0f + e) : __fdividef(1.0f, 1.0f + e);
    s = g < 0.0f ? e * r : r;
    rest = g < 0.0f ? r : e * r;
}

template <typename T, typename TO, int V>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const ActParams p, int team) {
    pdl_wait_then_release();
    constexpr bool kFull = sizeof(T) == 4 || sizeof(TO) == 4;
    const int per = kThreads / team, lane = threadIdx.x % team;
    const int64_t step = (int64_t)gridDim.x * per;
    for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / team; r < p.rows; r += step) {
        const T *g = (const T*)p.gate + r * p.ld_gate, *u = (const T*)p.up + r * p.ld_up;
        TO* o = (TO*)p.out + r * p.ld_out;
        const float w = p.weight ? p.weight[r] : 1.0f;
#pragma unroll 4
        for (int i = lane * V; i < p.I; i += team * V) {
            Pack<T, V> a, b;
            Pack<TO, V> h;
            a.load(g + i);
            b.load(u + i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float s, rest;
                sigmoid<kFull>(a.v[j], s, rest);
                h.v[j] = a.v[j] * s * b.v[j] * w;
            }
            h.store(o + i);
        }
    }
}

template <typename T, int V> __global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(const ActParams p, int team) {
    pdl_wait_then_release();
    constexpr bool kFull = sizeof(T) == 4;
    __shared__ float part[kThreads / 32];
    const int per = kThreads / team, lane = threadIdx.x % team;
    const int64_t step = (int64_t)gridDim.x * per;
    for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / team; r < p.rows; r += step) {
        const T *g = (const T*)p.gate + r * p.ld_gate, *u = (const T*)p.up + r * p.ld_up, *d = (const T*)p.dh + r * p.ld_dh;
        T *dg = (T*)p.dgate + r * p.ld_dgate, *du = (T*)p.dup + r * p.ld_dup;
        const float w = p.weight ? p.weight[r] : 1.0f;
        float sum = 0.0f;
#pragma unroll 4
        for (int i = lane * V; i < p.I; i += team * V) {
            Pack<T, V> a, b, c, x, y;
            a.load(g + i);
            b.load(u + i);
            c.load(d + i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float s, rest;
                sigmoid<kFull>(a.v[j], s, rest);
                const float silu = a.v[j] * s, du1 = c.v[j] * silu;
                sum = fmaf(du1, b.v[j], sum);
                x.v[j] = w * c.v[j] * b.v[j] * fmaf(silu, rest, s);
                y.v[j] = w * du1;
            }
            x.store(dg + i);
            y.store(du + i);
        }
        if (p.dweight) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (team == 32) {
                if (lane == 0) p.dweight[r] = sum;
            } else {  // the block is the team: its rows are the same for every thread
                if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
                __syncthreads();
                if (threadIdx.x == 0) {
                    float t = 0.0f;
                    for (int i = 0; i < kThreads / 32; ++i) t += part[i];
                    p.dweight[r] = t;
                }
                __syncthreads();
            }
        }
    }
}

bool whole(const void* p, int64_t ld, int elem) { return ((uintptr_t)p & 15) == 0 && ld * (elem == kF32 ? 4 : 2) % 16 == 0; }

// Threads of a row, and blocks.
int team_of(const ActParams& p, int num_sms) { return p.rows >= 8 * num_sms || p.I <= 256 ? 32 : kThreads; }
unsigned blocks_of(const ActParams& p, int team, int num_sms) {
    return (unsigned)std::min<int64_t>(cdiv(p.rows, kThreads / team), (int64_t)num_sms * 8);
}

}  // namespace

cudaError_t launch_swiglu(const ActParams& p, int num_sms, cudaStream_t s) {
    const int team = team_of(p, num_sms);
    const dim3 grid(blocks_of(p, team, num_sms)), block(kThreads);
    const bool v = p.I % 8 == 0 && whole(p.gate, p.ld_gate, p.elem) && whole(p.up, p.ld_up, p.elem) && whole(p.out, p.ld_out, p.out_elem);
    cudaError_t e;
#define MOE_ACT(T, TO) (v ? launch_kernel(swiglu_kernel<T, TO, 8>, grid, block, 0, s, 1, p, team) : launch_kernel(swiglu_kernel<T, TO, 1>, grid, block, 0, s, 1, p, team))
    if (p.elem == kF32) e = p.out_elem == kF32 ? MOE_ACT(float, float) : MOE_ACT(float, bf16);
    else e = p.out_elem == kF32 ? MOE_ACT(bf16, float) : MOE_ACT(bf16, bf16);
#undef MOE_ACT
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_swiglu_grad(const ActParams& p, int num_sms, cudaStream_t s) {
    const int team = team_of(p, num_sms);
    const dim3 grid(blocks_of(p, team, num_sms)), block(kThreads);
    const bool v = p.I % 8 == 0 && whole(p.gate, p.ld_gate, p.elem) && whole(p.up, p.ld_up, p.elem) && whole(p.dh, p.ld_dh, p.elem) &&
                   whole(p.dgate, p.ld_dgate, p.elem) && whole(p.dup, p.ld_dup, p.elem);
    cudaError_t e;
#define MOE_ACT(T) (v ? launch_kernel(swiglu_grad_kernel<T, 8>, grid, block, 0, s, 1, p, team) : launch_kernel(swiglu_grad_kernel<T, 1>, grid, block, 0, s, 1, p, team))
    e = p.elem == kF32 ? MOE_ACT(float) : MOE_ACT(bf16);
#undef MOE_ACT
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

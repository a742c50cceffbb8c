// Norms before and after a block (moe_norm_pre, moe_norm_post).
//
//   N(v)  = (v - mu) / sqrt(mean((v - mu)^2) + eps) * (w + w_offset) + b,
//           mu = mean(v) (LayerNorm) or 0 (RMSNorm)
//   pre:    n  = N(x)
//   post:   r' = res_scale * r + branch_scale * g * N(y)
//           n' = N_next(r' as stored)
//
// A row is held in registers as fp32, 16 elements a thread, so that every
// tensor passes once: the statistics are sums over the registers (the
// variance is taken about the mean, not from a sum of squares), and the next
// norm reads r' before it leaves them, rounded as it is stored.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kPer = 16;         // elements of a row per thread
constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float load_p(const void* p, int is_bf16, int64_t i) {
    return is_bf16 ? __bfloat162float(__ldg((const bf16*)p + i)) : __ldg((const float*)p + i);
}

// Row access, VEC elements at a time.  VEC = 8: 16-byte accesses (two for
// fp32); thread i of the row takes vectors i and i + nthr.  VEC = 1: any
// alignment, elements i, i + nthr, ...
template <int VEC> struct Row {
    static constexpr int kChunks = kPer / VEC;
    __device__ static int col(int c, int i, int nthr) { return (c * nthr + i) * VEC; }
};

template <int VEC, typename T> __device__ __forceinline__ void load_vec(const T* p, float* v) {
    if constexpr (VEC == 1) {
        v[0] = to_f32(__ldg(p));
    } else if constexpr (sizeof(T) == 2) {
        const uint4 q = __ldg((const uint4*)p);
        const T* e = (const T*)&q;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 q = __ldg((const float4*)p + h);
            v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
        }
    }
}
template <int VEC, typename T> __device__ __forceinline__ void store_vec(T* p, const float* v) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 2) {
        uint4 q;
        T* e = (T*)&q;
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
        *(uint4*)p = q;
    } else {
        ((float4*)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        ((float4*)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
// VEC values of a parameter vector (w, b, a per-channel gate), either type.
template <int VEC> __device__ __forceinline__ void load_par(const void* p, int is_bf16, int64_t i, float* v) {
    if (is_bf16) load_vec<VEC>((const bf16*)p + i, v);
    else load_vec<VEC>((const float*)p + i, v);
}

// Sum over the nthr threads of a row (nthr = 32, or the whole block).
__device__ __forceinline__ float row_sum(float s, int nthr, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (nthr == 32) return s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // the previous sum has been read
    if (lane == 0) red[warp] = s;
    __syncthreads();
    s = lane < (nthr >> 5) ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// v <- N(v) for this thread's elements of the row.
template <int VEC>
__device__ __forceinline__ void normalise(float* v, const NormParams& n, int i, int nthr, int D, float* red) {
    constexpr int C = Row<VEC>::kChunks;
    if (n.kind == MOE_NORM_NONE) return;
    float mu = 0.0f;
    if (n.kind == MOE_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) s += v[e];  // elements past D are zero
        mu = row_sum(s, nthr, red) / (float)D;
    }
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (Row<VEC>::col(c, i, nthr) < D) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[c * VEC + e] - mu;
                s = fmaf(d, d, s);
            }
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum(s, nthr, red) / (float)D + n.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC>::col(c, i, nthr);
        if (col < D) {
            float w[VEC], b[VEC];
            if (n.w) load_par<VEC>(n.w, n.p_bf16, col, w);
            if (n.b) load_par<VEC>(n.b, n.p_bf16, col, b);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float x = (v[c * VEC + e] - mu) * rstd;
                if (n.w) x *= w[e] + n.w_offset;
                if (n.b) x += b[e];
                v[c * VEC + e] = x;
            }
        }
    }
}

// One row per nthr threads; nthr = 32 (several rows a block) or the block.
template <int VEC, typename XT, typename OT>
__global__ void __launch_bounds__(kMaxThreads) norm_pre_kernel(const NormParams n, const XT* __restrict__ x, int64_t ld_x, int T,
                                                    int D, OT* __restrict__ out, int64_t ld_out, int nthr) {
    __shared__ float red[32];
    constexpr int C = Row<VEC>::kChunks;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / nthr) + threadIdx.x / nthr;
    const int i = threadIdx.x % nthr;
    if (t >= T) return;  // whole warps: nthr = 32 here
    float v[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC>::col(c, i, nthr);
        if (col < D) load_vec<VEC>(x + t * ld_x + col, v + c * VEC);
    }
    normalise<VEC>(v, n, i, nthr, D, red);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC>::col(c, i, nthr);
        if (col < D) store_vec<VEC>(out + t * ld_out + col, v + c * VEC);
    }
}

__device__ __forceinline__ float gate_value(float g, int sigmoid) { return sigmoid ? 1.0f / (1.0f + expf(-g)) : g; }

template <int VEC, typename YT, typename RT, typename NT>
__global__ void __launch_bounds__(kMaxThreads) norm_post_kernel(const PostParams p, const YT* __restrict__ y, const RT* res, RT* out,
                                                     NT* __restrict__ next, int nthr) {
    __shared__ float red[32];
    constexpr int C = Row<VEC>::kChunks;
    const int D = p.D;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / nthr) + threadIdx.x / nthr;
    const int i = threadIdx.x % nthr;
    if (t >= p.T) return;
    float v[kPer], r[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = r[e] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC>::col(c, i, nthr);
        if (col < D) {
            load_vec<VEC>(y + t * p.ld_y + col, v + c * VEC);
            load_vec<VEC>(res + t * p.ld_res + col, r + c * VEC);
        }
    }
    normalise<VEC>(v, p.norm, i, nthr, D, red);
    const float gt = p.gate_by == MOE_GATE_TOKEN ? gate_value(load_p(p.gate, p.gate_bf16, t), p.gate_sigmoid) : 1.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC>::col(c, i, nthr);
        if (col < D) {
            float g[VEC];
            if (p.gate_by == MOE_GATE_CHANNEL) load_par<VEC>(p.gate, p.gate_bf16, col, g);
            if (p.gate_by == MOE_GATE_FULL) load_par<VEC>(p.gate, p.gate_bf16, t * p.ld_gate + col, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float a = v[c * VEC + e] * gt;
                if (p.gate_by >= MOE_GATE_CHANNEL && p.gate_by != MOE_GATE_TOKEN) a *= gate_value(g[e], p.gate_sigmoid);
                r[c * VEC + e] = to_f32(from_f32<RT>(p.res_scale * r[c * VEC + e] + p.branch_scale * a));
            }
            store_vec<VEC>(out + t * p.ld_out + col, r + c * VEC);
        }
    }
    if (p.next.kind == MOE_NORM_NONE) return;
    normalise<VEC>(r, p.next, i, nthr, D, red);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC>::col(c, i, nthr);
        if (col < D) store_vec<VEC>(next + t * p.ld_next + col, r + c * VEC);
    }
}

// Threads of a row: 16 elements each, a whole number of warps.
int row_threads(int D) { return std::min<int64_t>(kMaxThreads, 32 * cdiv(cdiv(D, kPer), 32)); }

bool vec_ok(const void* p, int64_t ld, int bytes) {
    return p == nullptr || (((uintptr_t)p & 15) == 0 && (ld * bytes) % 16 == 0);
}
bool par_ok(const NormParams& n) { return vec_ok(n.w, 0, 1) && vec_ok(n.b, 0, 1); }

}  // namespace

bool norm_supported(int D) { return D <= kPer * kMaxThreads; }

cudaError_t launch_norm_pre(const NormParams& n, const void* x, int x_elem, int64_t ld_x, int T, int D, void* out,
                            int out_elem, int64_t ld_out, cudaStream_t stream) {
    const int nthr = row_threads(D), rows = nthr == 32 ? 4 : 1;
    const dim3 grid((unsigned)cdiv(T, rows)), block(nthr * rows);
    const bool vec = D % 8 == 0 && vec_ok(x, ld_x, x_elem == kF32 ? 4 : 2) &&
                     vec_ok(out, ld_out, out_elem == kF32 ? 4 : 2) && par_ok(n);
#define MOE_PRE(XT, OT)                                                                                          \
    do {                                                                                                         \
        if (vec) norm_pre_kernel<8, XT, OT><<<grid, block, 0, stream>>>(n, (const XT*)x, ld_x, T, D, (OT*)out, ld_out, nthr); \
        else norm_pre_kernel<1, XT, OT><<<grid, block, 0, stream>>>(n, (const XT*)x, ld_x, T, D, (OT*)out, ld_out, nthr);     \
    } while (0)
    if (x_elem == kF32) {
        if (out_elem == kF32) MOE_PRE(float, float);
        else MOE_PRE(float, bf16);
    } else {
        if (out_elem == kF32) MOE_PRE(bf16, float);
        else MOE_PRE(bf16, bf16);
    }
#undef MOE_PRE
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_norm_post(const PostParams& p, cudaStream_t stream) {
    const int nthr = row_threads(p.D), rows = nthr == 32 ? 4 : 1;
    const dim3 grid((unsigned)cdiv(p.T, rows)), block(nthr * rows);
    auto bytes = [](int elem) { return elem == kF32 ? 4 : 2; };
    const bool has_next = p.next.kind != MOE_NORM_NONE;
    const bool vec = p.D % 8 == 0 && vec_ok(p.y, p.ld_y, bytes(p.y_elem)) && vec_ok(p.res, p.ld_res, bytes(p.r_elem)) &&
                     vec_ok(p.out, p.ld_out, bytes(p.r_elem)) && par_ok(p.norm) && par_ok(p.next) &&
                     (!has_next || vec_ok(p.next_out, p.ld_next, bytes(p.n_elem))) &&
                     (p.gate_by == MOE_GATE_NONE || p.gate_by == MOE_GATE_TOKEN ||
                      vec_ok(p.gate, p.gate_by == MOE_GATE_FULL ? p.ld_gate : 0, p.gate_bf16 ? 2 : 4));
#define MOE_POST(YT, RT, NT)                                                                                     \
    do {                                                                                                         \
        if (vec)                                                                                                 \
            norm_post_kernel<8, YT, RT, NT><<<grid, block, 0, stream>>>(p, (const YT*)p.y, (const RT*)p.res, (RT*)p.out, \
                                                                        (NT*)p.next_out, nthr);                  \
        else                                                                                                     \
            norm_post_kernel<1, YT, RT, NT><<<grid, block, 0, stream>>>(p, (const YT*)p.y, (const RT*)p.res, (RT*)p.out, \
                                                                        (NT*)p.next_out, nthr);                  \
    } while (0)
#define MOE_POST_N(YT, RT)                                       \
    do {                                                         \
        if (p.n_elem == kF32) MOE_POST(YT, RT, float);           \
        else MOE_POST(YT, RT, bf16);                             \
    } while (0)
    if (p.y_elem == kF32) {
        if (p.r_elem == kF32) MOE_POST_N(float, float);
        else MOE_POST_N(float, bf16);
    } else {
        if (p.r_elem == kF32) MOE_POST_N(bf16, float);
        else MOE_POST_N(bf16, bf16);
    }
#undef MOE_POST_N
#undef MOE_POST
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe

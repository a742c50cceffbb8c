// Products of rows grouped by expert on the CUDA cores, fp32 arithmetic:
// out[m][n] = sum_k A(m, k) B(n, k) with the operands of ProductOp.
//
// Tiles of BM x BM, K in steps of 16 through shared memory, the next step's
// elements in registers while this one's are multiplied.  Any strides and
// alignment: elements are loaded one by one, along whichever dimension is
// contiguous.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "groups.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int BK = 16, kThreads = 256;

// Element (row, col) of the B operand.
template <typename T> struct Dense {
    const T* p;
    int64_t ld;
    __device__ __forceinline__ float at(int64_t row, int col) const { return to_f32(p[row * ld + col]); }
};
struct Coded {
    Int4 q;
    int half, nb, shift;  // bytes and scales of a row, log2 of the group
    __device__ __forceinline__ float at(int64_t row, int col) const {
        const int c = (q.codes[row * half + (col >> 1)] >> (4 * (col & 1))) & 15;
        const int64_t s = row * nb + (col >> shift);
        const int z = q.zeros ? q.zeros[s] : 8;
        return (float)(c - z) * (q.scale_elem == kF32 ? ((const float*)q.scales)[s] : to_f32(((const bf16*)q.scales)[s]));
    }
};

struct Shape {
    int op, rows, G, N, K;
    const int32_t* offsets;
    void* out;
    int out_elem, accumulate;
    int64_t ldo;
};

// One step's elements of an operand, a register each.  Index (i, k): i along
// the tile, k along the sum.  kK: k is the contiguous one.
template <int BM, bool kK> struct Index {
    __device__ __forceinline__ static int i(int e) { return kK ? e / BK : e % BM; }
    __device__ __forceinline__ static int k(int e) { return kK ? e % BK : e / BM; }
};

template <int OP, typename T, typename B, int BM>
__global__ void __launch_bounds__(kThreads) product_simt_kernel(const T* a, int64_t lda, const B b, const Shape p) {
    constexpr int TM = BM / 16, kEach = BM * BK / kThreads, LD = BM + 4;
    constexpr bool kAK = OP != kProductDw, kBK = OP == kProductFwd;  // contiguous along the sum
    __shared__ float sa[BK][LD], sb[BK][LD];
    __shared__ GroupTable tab;
    pdl_wait();
    if (threadIdx.x < 32) group_table(tab, p.offsets, p.G, p.rows, BM);
    __syncthreads();
    pdl_release();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int cols = OP == kProductFwd ? p.N : p.K;       // of the output
    const int cb = (cols + BM - 1) / BM, nb = (p.N + BM - 1) / BM;
    const int64_t units = OP == kProductDw ? (int64_t)p.G * nb * cb : (int64_t)tab.tiles[p.G] * cb;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int t = (int)(u / cb), c0 = (int)(u - (int64_t)t * cb) * BM;
        int g, i0, i1, k0, k1;  // rows of the tile [i0, i1), the sum's range
        if (OP == kProductDw) {
            g = t / nb;
            i0 = (t - g * nb) * BM;
            i1 = p.N;
            k0 = tab.first[g];
            k1 = tab.last[g];
        } else {
            g = find_group_smem(tab.tiles, p.G, t);
            i0 = tab.first[g] + (t - tab.tiles[g]) * BM;
            i1 = tab.last[g];
            k0 = 0;
            k1 = OP == kProductFwd ? p.K : p.N;
        }
        float acc[TM][TM] = {};
        float ra[kEach], rb[kEach];
        auto fetch = [&](int k) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int e = tid + j * kThreads;
                const int ai = i0 + Index<BM, kAK>::i(e), ak = k + Index<BM, kAK>::k(e);
                const int bi = c0 + Index<BM, kBK>::i(e), bk = k + Index<BM, kBK>::k(e);
                ra[j] = ai < i1 && ak < k1 ? to_f32(kAK ? a[(int64_t)ai * lda + ak] : a[(int64_t)ak * lda + ai]) : 0.0f;
                float v = 0.0f;
                if (bi < cols && bk < k1) {
                    if (OP == kProductFwd) v = b.at((int64_t)g * p.N + bi, bk);
                    else if (OP == kProductDx) v = b.at((int64_t)g * p.N + bk, bi);
                    else v = b.at(bk, bi);
                }
                rb[j] = v;
            }
        };
        if (k0 < k1) fetch(k0);
        for (int k = k0; k < k1; k += BK) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int e = tid + j * kThreads;
                sa[Index<BM, kAK>::k(e)][Index<BM, kAK>::i(e)] = ra[j];
                sb[Index<BM, kBK>::k(e)][Index<BM, kBK>::i(e)] = rb[j];
            }
            __syncthreads();
            if (k + BK < k1) fetch(k + BK);
#pragma unroll
            for (int kk = 0; kk < BK; ++kk) {
                float x[TM], y[TM];
#pragma unroll
                for (int h = 0; h < TM / 4; ++h) {
                    *(float4*)(x + 4 * h) = *(const float4*)&sa[kk][h * 64 + ty * 4];
                    *(float4*)(y + 4 * h) = *(const float4*)&sb[kk][h * 64 + tx * 4];
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = i0 + (i >> 2) * 64 + ty * 4 + (i & 3);
            if (r >= i1) continue;
            const int64_t at = (OP == kProductDw ? (int64_t)g * p.N + r : (int64_t)r) * p.ldo;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int c = c0 + (j >> 2) * 64 + tx * 4 + (j & 3);
                if (c >= cols) continue;
                float v = acc[i][j];
                if (p.out_elem == kF32) {
                    float* o = (float*)p.out + at + c;
                    *o = OP == kProductDw && p.accumulate ? *o + v : v;
                } else {
                    bf16* o = (bf16*)p.out + at + c;
                    *o = __float2bfloat16_rn(OP == kProductDw && p.accumulate ? to_f32(*o) + v : v);
                }
            }
        }
    }
}

template <int OP, typename T, typename B>
cudaError_t launch_any(const T* a, int64_t lda, const B& b, const Shape& p, int num_sms, cudaStream_t s) {
    const int cols = OP == kProductFwd ? p.N : p.K;
    auto units = [&](int bm) {
        const int64_t cb = cdiv(cols, bm);
        if (OP == kProductDw) return (int64_t)p.G * cdiv(p.N, bm) * cb;
        return (cdiv(p.rows, bm) + std::min(p.G - 1, p.rows)) * cb;
    };
    cudaError_t e;
    if (units(128) >= 2 * num_sms) {
        e = launch_kernel(product_simt_kernel<OP, T, B, 128>, dim3((unsigned)std::min<int64_t>(units(128), 2 * num_sms)), dim3(kThreads), 0,
                          s, 1, a, lda, b, p);
    } else {
        e = launch_kernel(product_simt_kernel<OP, T, B, 64>, dim3((unsigned)std::min<int64_t>(units(64), 4 * num_sms)), dim3(kThreads), 0,
                          s, 1, a, lda, b, p);
    }
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int OP> cudaError_t launch_typed(const GroupProduct& g, const Shape& p, int num_sms, cudaStream_t s) {
    const int64_t ldb = OP == kProductDw ? g.ldb : g.K;
    if (g.elem == kF32) return launch_any<OP>((const float*)g.a, g.lda, Dense<float>{(const float*)g.b, ldb}, p, num_sms, s);
    return launch_any<OP>((const bf16*)g.a, g.lda, Dense<bf16>{(const bf16*)g.b, ldb}, p, num_sms, s);
}

}  // namespace

cudaError_t launch_product_simt(const GroupProduct& g, int num_sms, cudaStream_t stream) {
    const Shape p = {g.op, g.rows, g.G, g.N, g.K, g.offsets, g.out, g.out_elem, g.accumulate, g.ldo};
    if (g.op == kProductFwd) return launch_typed<kProductFwd>(g, p, num_sms, stream);
    if (g.op == kProductDx) return launch_typed<kProductDx>(g, p, num_sms, stream);
    return launch_typed<kProductDw>(g, p, num_sms, stream);
}

cudaError_t launch_int4_simt(const Int4Product& g, int num_sms, cudaStream_t stream) {
    const Shape p = {kProductFwd, g.rows, g.G, g.N, g.K, g.offsets, g.out, g.out_elem, 0, g.ldo};
    const Coded b = {g.w, g.K / 2, (int)cdiv(g.K, g.w.group), g.w.group == 32 ? 5 : g.w.group == 64 ? 6 : 7};
    if (g.elem == kF32) return launch_any<kProductFwd>((const float*)g.x, g.ldx, b, p, num_sms, stream);
    return launch_any<kProductFwd>((const bf16*)g.x, g.ldx, b, p, num_sms, stream);
}

}  // namespace moe

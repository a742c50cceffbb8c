// Product of two microscaled 4-bit matrices (moe_mx_gemm), dense or grouped:
//   out[r][n] = sum_k a[r][k] * b_g[n][k]   for the rows r of group g.
//
// 64 x 64 output tiles on the CUDA cores: 32-column blocks of both operands
// are read back to fp32 in shared memory and multiplied in fp32.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kT = 64;

template <typename OT>
__global__ void __launch_bounds__(256) gemm_mx_simt_kernel(const MxGemm g) {
    __shared__ float sa[kMxBlock][kT + 1], sb[kMxBlock][kT + 1];
    // the row tile's group: tiles of 64 rows, group after group
    int tile = blockIdx.y, grp = 0, r0 = 0, r1 = g.rows;
    if (g.offsets) {
        for (grp = 0; grp < g.G; ++grp) {
            r0 = min(max(__ldg(g.offsets + grp), 0), g.rows);
            r1 = min(max(__ldg(g.offsets + grp + 1), r0), g.rows);
            const int nt = (r1 - r0 + kT - 1) / kT;
            if (tile < nt) break;
            tile -= nt;
        }
        if (grp == g.G) return;
    }
    const int m0 = r0 + tile * kT, n0 = blockIdx.x * kT;
    const int nb = g.K / kMxBlock;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int kb = 0; kb < nb; ++kb) {
        // thread: one 32-bit word (eight codes) of one row of each operand
        const int lr = threadIdx.x >> 2, lw = threadIdx.x & 3;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int64_t row = side ? (int64_t)grp * g.N + n0 + lr : m0 + lr;
            const bool in = side ? n0 + lr < g.N : m0 + lr < r1;
            float (*dst)[kT + 1] = side ? sb : sa;
            uint32_t h[4] = {0, 0, 0, 0};
            float f = 0.0f;
            if (in) {
                const int64_t blk = row * nb + kb;
                mx_f16x2(__ldg((const uint32_t*)((side ? g.b : g.a) + blk * 16 + lw * 4)), h);
                f = mx_scale(__ldg((side ? g.b_scale : g.a_scale) + blk));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = __half22float2(*(const __half2*)&h[i]);
                dst[lw * 8 + 2 * i][lr] = v.x * f;
                dst[lw * 8 + 2 * i + 1][lr] = v.y * f;
            }
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < kMxBlock; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = sa[k][ty + 16 * i];
                b[i] = sb[k][tx + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (r < r1 && n < g.N) ((OT*)g.out)[(int64_t)r * g.ldo + n] = from_f32<OT>(acc[i][j]);
        }
}

}  // namespace

cudaError_t launch_gemm_mx(const MxGemm& g, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const dim3 grid((unsigned)cdiv(g.N, kT), (unsigned)(cdiv(g.rows, kT) + (g.offsets ? g.G : 0)));
    if (g.out_elem == kF32) gemm_mx_simt_kernel<float><<<grid, 256, 0, stream>>>(g);
    else gemm_mx_simt_kernel<bf16><<<grid, 256, 0, stream>>>(g);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace moe

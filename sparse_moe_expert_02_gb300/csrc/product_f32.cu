// Products of rows grouped by expert in fp32 arithmetic, on the CUDA cores:
// out[m][n] = sum_k A(m, k) B(n, k) with the operands of ProductOp.
//
// Tiles of BM x BM, K in steps through a ring of kStages steps in shared
// memory.  Elements come by cp.async one by one, along whichever dimension is
// contiguous, to where the products read them: any strides and alignment, and
// zeros beyond the edges, without registers between.  Tiles of 128 where there
// is one for each SM (a thread's 8 x 8 sums need the fewest reads of shared
// memory), of 64 or 32 where there are fewer: a short call is bound by one
// block's way through K.  Tiles are counted as the most that the rows can give,
// one more than they fill for each group; so with many groups of few rows most
// of a tile is empty: 64 groups of one row, 1024 x 4096, take 1375 us, the
// weights' bytes 160.
#include <algorithm>

#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace f32 {

constexpr int kThreads = 256, kMaxSplit = 8;

template <int BM> struct Tile {
    static constexpr int BK = BM == 128 ? 16 : 32, kStages = BM == 32 ? 4 : 3, LD = BM + 4;
    static constexpr int TM = BM == 32 ? 4 : 8;                             // a thread's sums: TM x TM
    static constexpr int kSide = BM / TM, kGroups = kThreads / (kSide * kSide);  // threads along a side; groups that share a step's places
    static constexpr int kBytes = kStages * 2 * BK * LD * 4;
    static constexpr int kBlocks = BM == 32 ? 4 : 2;  // an SM
    // the thread's i-th row or column
    __device__ __forceinline__ static int at(int i, int t) { return (i / 4) * 4 * kSide + t * 4 + i % 4; }
};

// Two multiply-adds in one instruction: d0 += x y0, d1 += x y1 (4096 x 1024 x
// 1024: 175 us, 196 one by one).
__device__ __forceinline__ void fma2(float& d0, float& d1, float x, float y0, float y1) {
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %2};\n mov.b64 b, {%3, %4};\n mov.b64 c, {%0, %1};\n fma.rn.f32x2 c, a, b, c;\n"
        " mov.b64 {%0, %1}, c;\n}\n"
        : "+f"(d0), "+f"(d1)
        : "f"(x), "f"(y0), "f"(y1));
}
// Four bytes to shared memory, or zeros.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_all_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// SPLIT: a cluster of `split` blocks shares each tile's sum.
template <int OP, int BM, bool SPLIT>
__global__ void __launch_bounds__(kThreads, Tile<BM>::kBlocks) product_f32_kernel(const GroupProduct p, const int split) {
    using T = Tile<BM>;
    constexpr int TM = T::TM, BK = T::BK, LD = T::LD, kEach = BM * BK / kThreads;
    constexpr bool kAK = OP != kProductDw, kBK = OP == kProductFwd;  // contiguous along the sum
    extern __shared__ __align__(16) float ring[];                    // [stage][A, B][BK][LD]
    __shared__ GroupTable tab;
    const float *a = (const float*)p.a, *b = (const float*)p.b;
    const int64_t ldb = OP == kProductDw ? p.ldb : p.K;
    pdl_wait();
    if (threadIdx.x < 32) group_table(tab, p.offsets, p.G, p.rows, BM);
    __syncthreads();
    pdl_release();
    const int tid = threadIdx.x, group = tid / (T::kSide * T::kSide), tx = tid % T::kSide, ty = tid / T::kSide % T::kSide;
    const int cols = OP == kProductFwd ? p.N : p.K;  // of the output
    const int cb = (cols + BM - 1) / BM, nb = (p.N + BM - 1) / BM;
    const int64_t units = OP == kProductDw ? (int64_t)p.G * nb * cb : (int64_t)tab.tiles[p.G] * cb;
    const int rank = SPLIT ? (int)tc::cluster_rank() : 0, team = SPLIT ? split : 1;
    for (int64_t u = blockIdx.x / team; u < units; u += gridDim.x / team) {
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
        // An operand's elements of a step, kEach a thread: along the sum one place for all of them and every
        // kThreads / BK-th row, or one row and every kThreads / BM-th place.
        const int ak = kAK ? tid % BK : tid / BM, ai = kAK ? tid / BK : tid % BM;
        const int bk = kBK ? tid % BK : tid / BM, bi = kBK ? tid / BK : tid % BM;
        constexpr int kNextI = kThreads / BK, kNextK = kThreads / BM;
        if (SPLIT) {  // this block's part of the sum
            const int n = (k1 - k0 + BK - 1) / BK, from = k0;
            k0 = from + (int)((int64_t)n * rank / split) * BK;
            k1 = min(k1, from + (int)((int64_t)n * (rank + 1) / split) * BK);
        }
        const float* pa = kAK ? a + (int64_t)(i0 + ai) * p.lda + k0 + ak : a + (int64_t)(k0 + ak) * p.lda + i0 + ai;
        const int64_t brow = OP == kProductDw ? 0 : (int64_t)g * p.N;  // row of B that its index 0 is
        const float* pb = kBK ? b + (brow + c0 + bi) * ldb + k0 + bk : b + (brow + k0 + bk) * ldb + c0 + bi;
        const uint32_t da = tc::smem_u32(ring) + (ak * LD + ai) * 4, db = tc::smem_u32(ring) + (BK * LD + bk * LD + bi) * 4;
        auto fetch = [&](int step) {
            const int left = k1 - k0 - step * BK;
            if (left > 0) {
                const uint32_t at = (step % T::kStages) * (2 * BK * LD * 4);
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    const bool ain = kAK ? ak < left && i0 + ai + j * kNextI < i1 : ak + j * kNextK < left && i0 + ai < i1;
                    const bool bin = kBK ? bk < left && c0 + bi + j * kNextI < cols : bk + j * kNextK < left && c0 + bi < cols;
                    copy4(da + at + j * (kAK ? kNextI : kNextK * LD) * 4, ain ? pa + j * (kAK ? kNextI : kNextK) * p.lda : a, ain);
                    copy4(db + at + j * (kBK ? kNextI : kNextK * LD) * 4, bin ? pb + j * (kBK ? kNextI : kNextK) * ldb : b, bin);
                }
                pa += kAK ? BK : BK * p.lda;
                pb += kBK ? BK : BK * ldb;
            }
            commit();  // (a group a step, empty past the end)
        };
        float acc[TM][TM] = {};
        const int steps = (k1 - k0 + BK - 1) / BK;
        for (int s = 0; s < T::kStages - 1; ++s) fetch(s);
        for (int s = 0; s < steps; ++s) {
            wait_all_but<T::kStages - 2>();
            __syncthreads();  // the step is here for everyone, and everyone is done with the one before
            fetch(s + T::kStages - 1);
            const float* sa = ring + (s % T::kStages) * (2 * BK * LD);
            const float* sb = sa + BK * LD;
#pragma unroll
            for (int k = 0; k < BK / T::kGroups; ++k) {
                const int kk = k * T::kGroups + group;
                float x[TM], y[TM];
#pragma unroll
                for (int h = 0; h < TM; h += 4) {
                    *(float4*)(x + h) = *(const float4*)(sa + kk * LD + T::at(h, ty));
                    *(float4*)(y + h) = *(const float4*)(sb + kk * LD + T::at(h, tx));
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TM; j += 2) {
                        if (TM == 8) {  // (4 x 4 sums: no gain)
                            fma2(acc[i][j], acc[i][j + 1], x[i], y[j], y[j + 1]);
                        } else {
                            acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
                            acc[i][j + 1] = fmaf(x[i], y[j + 1], acc[i][j + 1]);
                        }
                    }
            }
        }
        wait_all_but<0>();
        __syncthreads();  // the ring is free
        if constexpr (T::kGroups == 4) {  // groups 2 and 3 to 0 and 1, then 1 to 0
            static_assert(T::kBytes >= 2 * BM * BM * 4, "the ring holds two tiles");
            const int lane = tid % (T::kSide * T::kSide);
#pragma unroll
            for (int from = 2; from; from /= 2) {
                float* half = ring + (group & (from - 1)) * BM * BM + lane;
                if (group >= from && group < 2 * from) {
#pragma unroll
                    for (int i = 0; i < TM * TM; ++i) half[i * T::kSide * T::kSide] = acc[i / TM][i % TM];
                }
                __syncthreads();
                if (group < from) {
#pragma unroll
                    for (int i = 0; i < TM * TM; ++i) acc[i / TM][i % TM] += half[i * T::kSide * T::kSide];
                }
                __syncthreads();
            }
        }
        if constexpr (SPLIT) {
            // Every rank's tile to the first one's ring, [rank][sum][thread], which adds them up in their order.
            constexpr int kTeam = T::kSide * T::kSide;
            static_assert(T::kBytes >= kMaxSplit * BM * BM * 4, "the ring holds every rank's tile");
            tc::cluster_sync();  // the first one's ring is free
            if (group == 0) {
                const uint32_t to = tc::mapa_shared(tc::smem_u32(ring) + (rank * BM * BM + tid) * 4, 0);
#pragma unroll
                for (int i = 0; i < TM * TM; ++i)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * kTeam * 4), "f"(acc[i / TM][i % TM]) : "memory");
            }
            tc::cluster_sync();
            if (rank == 0 && group == 0) {
#pragma unroll
                for (int i = 0; i < TM * TM; ++i) {
                    float v = 0.0f;
                    for (int r = 0; r < split; ++r) v += ring[r * BM * BM + i * kTeam + tid];
                    acc[i / TM][i % TM] = v;
                }
            }
            __syncthreads();  // the ring is free
        }
        if (group || (SPLIT && rank)) continue;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = i0 + T::at(i, ty);
            if (r >= i1) continue;
            const int64_t at = (OP == kProductDw ? (int64_t)g * p.N + r : (int64_t)r) * p.ldo;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int c = c0 + T::at(j, tx);
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

template <int OP, int BM, bool SPLIT> cudaError_t launch(const GroupProduct& g, int64_t units, int split, int num_sms, cudaStream_t s) {
    cudaError_t e = ensure_smem_attr((const void*)product_f32_kernel<OP, BM, SPLIT>, Tile<BM>::kBytes);
    if (e != cudaSuccess) return e;
    e = launch_kernel(product_f32_kernel<OP, BM, SPLIT>, dim3((unsigned)(std::min<int64_t>(units, Tile<BM>::kBlocks * num_sms) * split)),
                      dim3(kThreads), Tile<BM>::kBytes, s, split, g, split);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int OP> cudaError_t launch_op(const GroupProduct& g, int num_sms, cudaStream_t s) {
    const int64_t cols = OP == kProductFwd ? g.N : g.K;
    auto units = [&](int64_t bm) {  // at most
        if (OP == kProductDw) return g.G * cdiv(g.N, bm) * cdiv(cols, bm);
        return (cdiv(g.rows, bm) + std::min(g.G - 1, g.rows)) * cdiv(cols, bm);
    };
    if (units(128) >= num_sms) return launch<OP, 128, false>(g, units(128), 1, num_sms, s);
    if (units(64) >= num_sms) return launch<OP, 64, false>(g, units(64), 1, num_sms, s);
    // Few tiles: a cluster for each, whose blocks split the sum (of dw at most all rows).  dx of 45 x 2536 x 41:
    // 10.8 us, 38 without.
    int split = 1;
    const int64_t steps = cdiv(OP == kProductFwd ? g.K : OP == kProductDx ? g.N : g.rows, Tile<32>::BK);
    while (split < kMaxSplit && units(32) * split * 2 <= num_sms && steps >= 8 * split) split *= 2;
    if (split > 1) return launch<OP, 32, true>(g, units(32), split, num_sms, s);
    return launch<OP, 32, false>(g, units(32), 1, num_sms, s);
}

}  // namespace f32

cudaError_t launch_product_f32(const GroupProduct& g, int num_sms, cudaStream_t stream) {
    if (g.op == kProductFwd) return f32::launch_op<kProductFwd>(g, num_sms, stream);
    if (g.op == kProductDx) return f32::launch_op<kProductDx>(g, num_sms, stream);
    return f32::launch_op<kProductDw>(g, num_sms, stream);
}

}  // namespace moe

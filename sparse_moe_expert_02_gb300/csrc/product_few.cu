// Products of a few rows with their groups' weights, bf16 or 4-bit
// (moe_grouped_gemm, moe_int4_gemm): out[r][n] = sum_k x[r][k] w_g[n][k].
//
// Bound by the bytes of the weights, and with 4 bits by the instructions that
// decode them, so they go straight into mma.sync (m16n8k16: 16 features by 8
// rows): a tensor-memory kernel would write what it decodes to shared memory
// first, for tiles of 128 features by 16 rows that a few rows do not fill.  A
// block takes 16 features of a group at a time, its eight warps a piece of the
// columns each; eight partial sums meet in shared memory.  How the columns are
// divided depends on K alone, so a row's result does not depend on the other
// rows and groups.  The order of the columns within a sum is free as long as x
// follows it, so a lane loads 16 bytes of a row and hands them to successive
// MMAs.
//
// 4 bits: the MMAs sum code - zero, exact in bf16, over one group of columns;
// the fp32 sum is then multiplied by the scale.  fp32 rows go in as three bf16
// parts, which hold all 24 bits.  A group's sum may overflow where its product
// with the scale does not, so what comes out as no finite number is summed
// again with the weights' values.
//
// This kernel: any alignment of x and scales, and columns that 128 does not
// divide; weights to registers, two chunks of 128 columns ahead.  Groups of 32
// and 64 columns need the four lanes that share an MMA's columns to hold codes
// of the same group: they exchange words.  The other, for the rest, is in
// product_few_bulk.cu.
#include <algorithm>

#include "few_rows.cuh"

namespace moe {
namespace few_rows {

// product_few_bulk.cu; cudaErrorNotSupported where its conditions do not hold.
cudaError_t launch_few_bulk(const Args& a, int LG, int elem, int num_sms, cudaStream_t s);

// Words of four lanes exchanged so that word i of every lane is of column
// group i (groups of 32) or i / 2 (of 64).
template <int LG> __device__ __forceinline__ void exchange(uint32_t (&w)[4], int t) {
    if (LG == 5) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, t & 1 ? w[i] : w[i + 1], 1);
            if (t & 1) w[i] = got;
            else w[i + 1] = got;
        }
    }
    if (LG == 5 || LG == 6) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, t & 2 ? w[i] : w[i + 2], 2);
            if (t & 2) w[i] = got;
            else w[i + 2] = got;
        }
    }
}
// First column, within a chunk, of the eight in word i of lane t.
template <int LG> __device__ __forceinline__ int column(int i, int t) {
    if (LG == 7) return 32 * t + 8 * i;
    if (LG == 6) return 64 * (i >> 1) + 32 * (t & 1) + 16 * (t >> 1) + 8 * (i & 1);
    return 32 * i + 8 * t;
}

template <int LG, typename T, typename TS> __global__ void __launch_bounds__(kThreads, 2) product_few_kernel(const Args p) {
    constexpr int kDepth = 2;  // (4: the same within 5 %)
    __shared__ Tables<> tab;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    const int FB = (p.N + kF - 1) / kF, units = build_tables(tab, p), step = gridDim.x;
    if ((int)blockIdx.x >= units) return;
    const int chunks = (p.K + kChunk - 1) / kChunk;
    const int k0 = chunks * warp / kWarps, nk = chunks * (warp + 1) / kWarps - k0, batches = (nk + kDepth - 1) / kDepth;
    const int nb = LG ? (p.K + (1 << LG) - 1) >> LG : 0;

    // Loads of the weights, a batch ahead of their use.
    Chunk<LG, TS> q[kDepth];
    int fu = blockIdx.x, fb = 0;                    // next batch to load
    int left[2];                            // chunks that this lane still has to load of rows g and g + 8
    const uint8_t* wp[2];                   // its part of the batch's first chunk
    int64_t sp[2];                          // first scale of that chunk
    const int lane_k = LG ? (p.K - 32 * t + kChunk - 1) / kChunk - k0 : nk;  // chunks with a code of this lane
    Unit fc = unit_at(fu, FB, p.G, tab), cur = fc;
    auto locate = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = (int64_t)fc.g * p.N + fc.f0 + g + 8 * h;
            left[h] = fu < units && fc.f0 + g + 8 * h < p.N ? nk : 0;
            if (LG == 0) wp[h] = (const uint8_t*)(p.w + row * p.K + k0 * kChunk + 8 * t);
            else wp[h] = p.q.codes + row * (p.K / 2) + k0 * (kChunk / 2) + 16 * t;
            sp[h] = row * nb + (int64_t)k0 * (kChunk >> LG);
        }
    };
    auto fetch = [&](int i, Chunk<LG, TS>& v) {  // slot i of the batch (fu, fb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool on = i < left[h];
            if constexpr (LG == 0) {
                const int c = (k0 + fb * kDepth + i) * kChunk + 8 * t;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v.w[h][j] = on && c + 32 * j < p.K ? load_once(wp[h] + i * 2 * kChunk + 64 * j) : make_uint4(0, 0, 0, 0);
            } else {
                using C = Chunk<LG, TS>;
                v.w[h] = on && fb * kDepth + i < lane_k ? load_once(wp[h] + i * (kChunk / 2)) : make_uint4(0, 0, 0, 0);
                v.z[h] = 0x08080808u;
#pragma unroll
                for (int j = 0; j < (C::kScale ? C::kScale : 1); ++j) v.s[h][j] = 0;
                if (!on) continue;
                const int64_t at = sp[h] + i * C::kGroups;
                const int g0 = (k0 + fb * kDepth + i) * C::kGroups;
#pragma unroll
                for (int j = 0; j < C::kGroups; ++j) {
                    if (g0 + j >= nb) continue;
                    if (sizeof(TS) == 4) v.s[h][j] = ((const uint32_t*)p.q.scales)[at + j];
                    else v.s[h][j >> 1] |= (uint32_t)((const uint16_t*)p.q.scales)[at + j] << (16 * (j & 1));
                    if (p.q.zeros) v.z[h] = (v.z[h] & ~(255u << (8 * j))) | (uint32_t)p.q.zeros[at + j] << (8 * j);
                }
            }
        }
    };
    locate();
#pragma unroll
    for (int i = 0; i < kDepth; ++i) fetch(i, q[i]);

    const int xc = k0 * kChunk + column<LG>(0, t);  // this lane's first column
    const T* x0;
    auto rows_at = [&]() {  // rows past the tile: the last one's, their sums are not stored
        x0 = (const T*)p.x + (int64_t)(cur.row0 + min(g, cur.n - 1)) * p.ldx + xc;
    };
    rows_at();
    int buf = 0;
    for (int u = blockIdx.x; u < units; u += step, buf ^= 1) {
        float acc[4] = {};
        for (int b = 0; b < batches; ++b) {
            if (++fb == batches) {
                fb = 0;
                if ((fu += step) < units) fc = unit_at(fu, FB, p.G, tab);
                locate();
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    left[h] -= kDepth;
                    wp[h] += kDepth * (LG ? kChunk / 2 : 2 * kChunk);
                    sp[h] += kDepth * (LG ? kChunk >> LG : 0);
                }
            }
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                const int k = b * kDepth + i;
                if (k < nk) {
                    const T* xk = x0 + k * kChunk;
                    const int room = p.K - xc - k * kChunk;  // columns from the lane's first on
                    if constexpr (LG == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 a = q[i].w[0][j], e = q[i].w[1][j];
                            Parts<T> x = {};
                            if (32 * j < room) load_x<false>(xk + 32 * j, x);
                            mma(acc, a.x, e.x, a.y, e.y, x.v[0][0], x.v[0][1]);
                            mma(acc, a.z, e.z, a.w, e.w, x.v[0][2], x.v[0][3]);
                        }
                    } else {
                        constexpr int kGroups = 1 << (7 - LG), kWords = 4 / kGroups;  // column groups of a chunk, words of each
                        uint32_t w0[4] = {q[i].w[0].x, q[i].w[0].y, q[i].w[0].z, q[i].w[0].w};
                        uint32_t w1[4] = {q[i].w[1].x, q[i].w[1].y, q[i].w[1].z, q[i].w[1].w};
                        exchange<LG>(w0, t);
                        exchange<LG>(w1, t);
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) {
                            float sum[Parts<T>::n][4] = {};
#pragma unroll
                            for (int j = 0; j < kWords; ++j) {
                                const int wi = gr * kWords + j, col = column<LG>(wi, 0);
                                uint32_t a[4], e[4];
                                int4_pairs(w0[wi], zero_pair(q[i].z[0], gr), a);
                                int4_pairs(w1[wi], zero_pair(q[i].z[1], gr), e);
                                Parts<T> x = {};
                                if (col < room) load_x<false>(xk + col, x);
                                mma8(sum, a, e, x.v);
                            }
                            const float sc[2] = {scale_of(q[i], 0, gr), scale_of(q[i], 1, gr)};
                            add_scaled(acc, sum, sc);
                        }
                    }
                }
                fetch(i, q[i]);
            }
        }
        put_part(tab.part[buf][warp], acc, g, t);
        __syncthreads();
        finish<LG, T>(p, tab.part[buf], cur, nb);
        if (u + step < units) {
            cur = batches ? fc : unit_at(u + step, FB, p.G, tab);
            rows_at();
        }
    }
}

template <int LG, typename T, typename TS> cudaError_t launch(const Args& a, int num_sms, cudaStream_t s) {
    const int64_t tiles = cdiv(a.rows, kRows) + (a.offsets ? std::min(a.G - 1, a.rows) : 0), units = tiles * cdiv(a.N, kF);  // at most
    const dim3 grid((unsigned)std::min<int64_t>(units, 2 * num_sms)), block(kThreads);
    const cudaError_t e = launch_kernel(product_few_kernel<LG, T, TS>, grid, block, 0, s, 1, a);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}
template <int LG> cudaError_t launch_coded(const Args& a, int elem, int num_sms, cudaStream_t s) {
    if (elem == kF32) return a.q.scale_elem == kF32 ? launch<LG, float, float>(a, num_sms, s) : launch<LG, float, bf16>(a, num_sms, s);
    return a.q.scale_elem == kF32 ? launch<LG, bf16, float>(a, num_sms, s) : launch<LG, bf16, bf16>(a, num_sms, s);
}

}  // namespace few_rows

cudaError_t launch_product_few(const GroupProduct& g, int num_sms, cudaStream_t stream) {
    using namespace few_rows;
    if (g.op != kProductFwd || g.elem != kBF16 || g.K % 8 || ((uintptr_t)g.b & 15)) return cudaErrorNotSupported;
    Args a = {};
    a.offsets = g.offsets;
    a.rows = g.rows;
    a.G = g.G;
    a.N = g.N;
    a.K = g.K;
    a.x = g.a;
    a.ldx = g.lda;
    a.w = (const bf16*)g.b;
    a.out = g.out;
    a.out_elem = g.out_elem;
    a.ldo = g.ldo;
    a.err = g.err;
    a.spin_ns = g.spin_ns;
    const cudaError_t e = launch_few_bulk(a, 0, kBF16, num_sms, stream);
    return e != cudaErrorNotSupported ? e : launch<0, bf16, bf16>(a, num_sms, stream);
}

cudaError_t launch_int4_few(const Int4Product& g, int num_sms, cudaStream_t stream) {
    using namespace few_rows;
    Args a = {};
    a.offsets = g.offsets;
    a.rows = g.rows;
    a.G = g.G;
    a.N = g.N;
    a.K = g.K;
    a.x = g.x;
    a.ldx = g.ldx;
    a.q = g.w;
    a.out = g.out;
    a.out_elem = g.out_elem;
    a.ldo = g.ldo;
    a.err = g.err;
    a.spin_ns = g.spin_ns;
    const cudaError_t e = launch_few_bulk(a, g.w.group == 32 ? 5 : g.w.group == 64 ? 6 : 7, g.elem, num_sms, stream);
    if (e != cudaErrorNotSupported) return e;
    if (g.w.group == 32) return launch_coded<5>(a, g.elem, num_sms, stream);
    if (g.w.group == 64) return launch_coded<6>(a, g.elem, num_sms, stream);
    return launch_coded<7>(a, g.elem, num_sms, stream);
}

}  // namespace moe

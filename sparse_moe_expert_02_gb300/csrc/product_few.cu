// Products of a few rows with their groups' weights, bf16 or 4-bit
// (moe_grouped_gemm, moe_int4_gemm): out[r][n] = sum_k x[r][k] w_g[n][k].
//
// Bound by the bytes of the weights, so they go from memory to registers and
// straight into mma.sync (m16n8k16: 16 features by 8 rows), with nothing
// between: a tensor-memory kernel would write what it decodes to shared memory
// first, for tiles of 128 features that a few rows do not fill.  A block takes
// 16 features of a group at a time, its eight warps a piece of the columns
// each; a warp has the loads of its next 512 columns in flight while it
// multiplies.  The order of the columns within a sum is free as long as x
// follows it, so a lane loads 16 bytes of a row and hands them to successive
// MMAs.  Eight partial sums meet in shared memory.  How the columns are
// divided depends on K alone, so a row's result does not depend on the other
// rows and groups.
//
// 4 bits: the MMAs sum code - zero, exact in bf16, over one group of columns;
// the fp32 sum is then multiplied by the scale.  Groups of 32 and 64 columns
// need the four lanes that share an MMA's columns to hold codes of the same
// group: they exchange words first.  fp32 rows go in as three bf16 parts,
// which hold all 24 bits.  A group's sum may overflow where its product with
// the scale does not, so what comes out as no finite number is summed again
// with the weights' values.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "groups.cuh"
#include "int4.cuh"
#include "internal.h"

namespace moe {
namespace few_rows {

#ifndef MOE_FEW_DEPTH
#define MOE_FEW_DEPTH 2
#define MOE_FEW_BLOCKS 2
#endif
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kF = 16, kRows = 16;  // features and rows of a tile
constexpr int kChunk = 128;         // columns a warp takes at a time
constexpr int kPitch = 20;          // floats between the rows of a partial tile: lanes hit different banks

struct Args {
    const int32_t* offsets;
    int rows, G, N, K;
    const void* x;
    int64_t ldx;
    bool fast;
    const bf16* w;
    Int4 q;
    void* out;
    int out_elem;
    int64_t ldo;
};

// A lane's share of a chunk.  Codes in groups of 2^LG columns: 32 codes of
// feature rows g and g + 8, and the scales and zero points of the chunk's
// groups of both, as they lie in memory.  LG = 0: 32 bf16 of each row.
template <int LG, typename TS> struct Chunk {
    static constexpr int kGroups = 1 << (7 - LG), kScale = kGroups * (int)sizeof(TS) / 4;
    uint4 w[2];
    uint32_t s[2][kScale ? kScale : 1];
    uint32_t z[2];
};
template <typename TS> struct Chunk<0, TS> {
    uint4 w[2][4];
};
template <int LG, typename TS> __device__ __forceinline__ float scale_of(const Chunk<LG, TS>& q, int h, int gr) {
    if (sizeof(TS) == 4) return __uint_as_float(q.s[h][gr]);
    return __uint_as_float(gr & 1 ? q.s[h][gr >> 1] & 0xFFFF0000u : q.s[h][gr >> 1] << 16);
}

// Units are (row tile, feature tile).  list: group and tile within it of each
// row tile, so that a block finds its next unit without a search.
constexpr int kMaxTiles = 2 * kProductMaxG;  // (16 rows a group; fp32 rows may be more)
struct Tables {
    GroupTable groups;
    uint32_t list[kMaxTiles];
    float part[2][kWarps][kRows * kPitch];
};
struct Unit {
    int g, f0, row0, n;  // group, first feature, first row of the tile and how many
};
__device__ __forceinline__ Unit unit_at(int u, int FB, int G, const Tables& t) {
    Unit r;
    const int rt = u / FB;
    r.f0 = (u - rt * FB) * kF;
    if (t.groups.tiles[G] <= kMaxTiles) {
        const uint32_t e = t.list[rt];
        r.g = (int)(e & 2047u);
        r.row0 = t.groups.first[r.g] + (int)(e >> 11) * kRows;
    } else {
        r.g = find_group_smem(t.groups.tiles, G, rt);
        r.row0 = t.groups.first[r.g] + (rt - t.groups.tiles[r.g]) * kRows;
    }
    r.n = min(kRows, t.groups.last[r.g] - r.row0);
    return r;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: no place in L1, which x keeps.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Eight columns of x as the parts of MMA operands: one for bf16; for fp32
// three, each the leading eight bits of what the ones before leave, the second
// times 2^8 and the third times 2^16: within range for the largest numbers,
// and no bits lost below bf16's smallest for the smallest.
template <typename T> struct Parts { static constexpr int n = sizeof(T) == 4 ? 3 : 1; uint32_t v[n][4]; };

template <bool VEC> __device__ __forceinline__ void load_x(const bf16* x, Parts<bf16>& o) {
    if constexpr (VEC) {
        const uint4 v = __ldg((const uint4*)x);
        o.v[0][0] = v.x; o.v[0][1] = v.y; o.v[0][2] = v.z; o.v[0][3] = v.w;
    } else {
        const uint16_t* h = (const uint16_t*)x;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[0][j] = (uint32_t)__ldg(h + 2 * j) | (uint32_t)__ldg(h + 2 * j + 1) << 16;
    }
}
template <bool VEC> __device__ __forceinline__ void load_x(const float* x, Parts<float>& o) {
    float f[8];
    if constexpr (VEC) {
        *(float4*)f = __ldg((const float4*)x);
        *(float4*)(f + 4) = __ldg((const float4*)x + 1);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __ldg(x + j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t part[3][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float v = f[2 * j + h];
            const uint32_t u = __float_as_uint(v);
            const bool odd = (u & 0x7F800000u) == 0x7F800000u;  // an infinity or a NaN goes whole into the first part
            part[0][h] = odd && (u & 0x007FFFFFu) ? 0x7FC00000u : u & 0xFFFF0000u;
            const float r1 = odd ? 0.0f : v - __uint_as_float(part[0][h]);
            const float r2 = r1 * 256.0f;
            part[1][h] = __float_as_uint(r2) & 0xFFFF0000u;
            part[2][h] = __float_as_uint((r2 - __uint_as_float(part[1][h])) * 256.0f);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) o.v[i][j] = __byte_perm(part[i][0], part[i][1], 0x7632);
    }
}

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

// FAST: K a multiple of 128, 16-byte loads of x, a chunk's scales and zero
// points in one load each.
template <int LG, typename T, typename TS, bool FAST>
__global__ void __launch_bounds__(kThreads, MOE_FEW_BLOCKS) product_few_kernel(const Args p) {
    constexpr int kDepth = LG ? MOE_FEW_DEPTH : 2;
    __shared__ Tables tab;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    if (warp == 0) group_table(tab.groups, p.offsets, p.G, p.rows, kRows);
    __syncthreads();
    pdl_release();
    for (int i = threadIdx.x; i < p.G && tab.groups.tiles[p.G] <= kMaxTiles; i += kThreads)
        for (int j = tab.groups.tiles[i], n = 0; j < tab.groups.tiles[i + 1]; ++j, ++n) tab.list[j] = (uint32_t)i | (uint32_t)n << 11;
    __syncthreads();
    const int FB = (p.N + kF - 1) / kF, units = tab.groups.tiles[p.G] * FB, step = gridDim.x;
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
                    v.w[h][j] = on && (FAST || c + 32 * j < p.K) ? load_once(wp[h] + i * 2 * kChunk + 64 * j) : make_uint4(0, 0, 0, 0);
            } else {
                using C = Chunk<LG, TS>;
                v.w[h] = on && (FAST || fb * kDepth + i < lane_k) ? load_once(wp[h] + i * (kChunk / 2)) : make_uint4(0, 0, 0, 0);
                v.z[h] = 0x08080808u;
#pragma unroll
                for (int j = 0; j < (C::kScale ? C::kScale : 1); ++j) v.s[h][j] = 0;
                if (!on) continue;
                const int64_t at = sp[h] + i * C::kGroups;
                if constexpr (FAST) {
                    const TS* s = (const TS*)p.q.scales + at;
                    constexpr int kBytes = C::kGroups * (int)sizeof(TS);
                    if constexpr (kBytes == 2) v.s[h][0] = __ldg((const uint16_t*)s);
                    else if constexpr (kBytes == 4) v.s[h][0] = __ldg((const uint32_t*)s);
                    else if constexpr (kBytes == 8) *(uint2*)v.s[h] = __ldg((const uint2*)s);
                    else *(uint4*)v.s[h] = __ldg((const uint4*)s);
                    if (p.q.zeros) {
                        const uint8_t* z = p.q.zeros + at;
                        if constexpr (C::kGroups == 1) v.z[h] = __ldg(z);
                        else if constexpr (C::kGroups == 2) v.z[h] = __ldg((const uint16_t*)z);
                        else v.z[h] = __ldg((const uint32_t*)z);
                    }
                } else {
                    const int g0 = (k0 + fb * kDepth + i) * C::kGroups;
#pragma unroll
                    for (int j = 0; j < C::kGroups; ++j) {
                        if (g0 + j >= nb) continue;
                        if (sizeof(TS) == 4) v.s[h][j] = __ldg((const uint32_t*)p.q.scales + at + j);
                        else v.s[h][j >> 1] |= (uint32_t)__ldg((const uint16_t*)p.q.scales + at + j) << (16 * (j & 1));
                        if (p.q.zeros) v.z[h] = (v.z[h] & ~(255u << (8 * j))) | (uint32_t)__ldg(p.q.zeros + at + j) << (8 * j);
                    }
                }
            }
        }
    };
    locate();
#pragma unroll
    for (int i = 0; i < kDepth; ++i) fetch(i, q[i]);

    const int xc = k0 * kChunk + column<LG>(0, t);  // this lane's first column
    const T *x0, *x1;
    auto rows_at = [&]() {  // rows past the tile: the last one's, their sums are not stored
        x0 = (const T*)p.x + (int64_t)(cur.row0 + min(g, cur.n - 1)) * p.ldx + xc;
        x1 = (const T*)p.x + (int64_t)(cur.row0 + min(g + 8, cur.n - 1)) * p.ldx + xc;
    };
    rows_at();
    int buf = 0;
    for (int u = blockIdx.x; u < units; u += step, buf ^= 1) {
        const bool two = cur.n > 8;
        float acc[2][4] = {};
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
                    const T *xk = x0 + k * kChunk, *yk = x1 + k * kChunk;
                    const int room = p.K - xc - k * kChunk;  // columns from the lane's first on
                    if constexpr (LG == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 a = q[i].w[0][j], e = q[i].w[1][j];
                            Parts<T> x = {};
                            if (FAST || 32 * j < room) load_x<FAST>(xk + 32 * j, x);
                            mma(acc[0], a.x, e.x, a.y, e.y, x.v[0][0], x.v[0][1]);
                            mma(acc[0], a.z, e.z, a.w, e.w, x.v[0][2], x.v[0][3]);
                            if (two) {
                                Parts<T> y = {};
                                if (FAST || 32 * j < room) load_x<FAST>(yk + 32 * j, y);
                                mma(acc[1], a.x, e.x, a.y, e.y, y.v[0][0], y.v[0][1]);
                                mma(acc[1], a.z, e.z, a.w, e.w, y.v[0][2], y.v[0][3]);
                            }
                        }
                    } else {
                        constexpr int kGroups = 1 << (7 - LG), kWords = 4 / kGroups;  // column groups of a chunk, words of each
                        constexpr int kFirst = sizeof(T) == 4 ? 1 : 4;                // words whose x is loaded ahead
                        Parts<T> x[kFirst] = {};
                        if constexpr (kFirst == 4) {
#pragma unroll
                            for (int wi = 0; wi < 4; ++wi)
                                if (FAST || column<LG>(wi, 0) < room) load_x<FAST>(xk + column<LG>(wi, 0), x[wi]);
                        }
                        uint32_t w0[4] = {q[i].w[0].x, q[i].w[0].y, q[i].w[0].z, q[i].w[0].w};
                        uint32_t w1[4] = {q[i].w[1].x, q[i].w[1].y, q[i].w[1].z, q[i].w[1].w};
                        exchange<LG>(w0, t);
                        exchange<LG>(w1, t);
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) {
                            uint32_t z[2];  // 128 + zero in both halves
#pragma unroll
                            for (int h = 0; h < 2; ++h) z[h] = __byte_perm(q[i].z[h], 0x43434343u, 0x4040 + 0x0101 * gr);
                            float sum[Parts<T>::n][2][4] = {};
#pragma unroll
                            for (int j = 0; j < kWords; ++j) {
                                const int wi = gr * kWords + j, col = column<LG>(wi, 0);
                                uint32_t a[4], e[4];
                                int4_pairs(w0[wi], *(const __nv_bfloat162*)&z[0], a);
                                int4_pairs(w1[wi], *(const __nv_bfloat162*)&z[1], e);
                                Parts<T> xj = {};
                                if constexpr (kFirst == 4) xj = x[wi];
                                else if (FAST || col < room) load_x<FAST>(xk + col, xj);
#pragma unroll
                                for (int m = 0; m < Parts<T>::n; ++m) {
                                    mma(sum[m][0], a[0], e[0], a[1], e[1], xj.v[m][0], xj.v[m][1]);
                                    mma(sum[m][0], a[2], e[2], a[3], e[3], xj.v[m][2], xj.v[m][3]);
                                }
                                if (two) {
                                    Parts<T> y = {};
                                    if (FAST || col < room) load_x<FAST>(yk + col, y);
#pragma unroll
                                    for (int m = 0; m < Parts<T>::n; ++m) {
                                        mma(sum[m][1], a[0], e[0], a[1], e[1], y.v[m][0], y.v[m][1]);
                                        mma(sum[m][1], a[2], e[2], a[3], e[3], y.v[m][2], y.v[m][3]);
                                    }
                                }
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (h && !two) break;
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    float v = sum[0][h][m];
                                    if constexpr (Parts<T>::n == 3)
                                        v += fmaf(sum[2][h][m], 0x1p-16f, sum[1][h][m] * 0x1p-8f);
                                    acc[h][m] = fmaf(scale_of(q[i], m >> 1, gr), v, acc[h][m]);
                                }
                            }
                        }
                    }
                }
                fetch(i, q[i]);
            }
        }
        // D(g, 2t), D(g, 2t + 1), D(g + 8, 2t), D(g + 8, 2t + 1): feature, row
        float* mine = tab.part[buf][warp];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h && !two) break;
#pragma unroll
            for (int m = 0; m < 4; ++m) mine[(8 * h + 2 * t + (m & 1)) * kPitch + g + 8 * (m >> 1)] = acc[h][m];
        }
        __syncthreads();
        const int f = threadIdx.x & (kF - 1), r = threadIdx.x / kF;
        if (r < cur.n && cur.f0 + f < p.N) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += tab.part[buf][w][r * kPitch + f];
            if constexpr (LG != 0) {
                if (!isfinite(v)) {  // a group's sum may have overflown before its scale
                    const T* x = (const T*)p.x + (int64_t)(cur.row0 + r) * p.ldx;
                    const int64_t row = (int64_t)cur.g * p.N + cur.f0 + f;
                    v = 0.0f;
                    for (int k = 0; k < p.K; ++k) {
                        const int64_t at = row * nb + (k >> LG);
                        const int cd = (p.q.codes[row * (p.K / 2) + (k >> 1)] >> (4 * (k & 1))) & 15;
                        const float s = p.q.scale_elem == kF32 ? ((const float*)p.q.scales)[at] : to_f32(((const bf16*)p.q.scales)[at]);
                        v = fmaf(to_f32(x[k]), (float)(cd - (p.q.zeros ? p.q.zeros[at] : 8)) * s, v);
                    }
                }
            }
            const int64_t at = (int64_t)(cur.row0 + r) * p.ldo + cur.f0 + f;
            if (p.out_elem == kF32) ((float*)p.out)[at] = v;
            else ((bf16*)p.out)[at] = __float2bfloat16_rn(v);
        }
        if (u + step < units) {
            cur = batches ? fc : unit_at(u + step, FB, p.G, tab);
            rows_at();
        }
    }
}

template <int LG, typename T, typename TS> cudaError_t launch(const Args& a, int num_sms, cudaStream_t s) {
    const int64_t tiles = cdiv(a.rows, kRows) + (a.offsets ? std::min(a.G - 1, a.rows) : 0), units = tiles * cdiv(a.N, kF);  // at most
    const dim3 grid((unsigned)std::min<int64_t>(units, MOE_FEW_BLOCKS * num_sms)), block(kThreads);
    const cudaError_t e = a.fast ? launch_kernel(product_few_kernel<LG, T, TS, true>, grid, block, 0, s, 1, a)
                                 : launch_kernel(product_few_kernel<LG, T, TS, false>, grid, block, 0, s, 1, a);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}
template <int LG> cudaError_t launch_coded(const Args& a, int elem, int num_sms, cudaStream_t s) {
    if (elem == kF32) return a.q.scale_elem == kF32 ? launch<LG, float, float>(a, num_sms, s) : launch<LG, float, bf16>(a, num_sms, s);
    return a.q.scale_elem == kF32 ? launch<LG, bf16, float>(a, num_sms, s) : launch<LG, bf16, bf16>(a, num_sms, s);
}

bool aligned16(const void* p, int64_t ld, int elem) { return ((uintptr_t)p & 15) == 0 && ld * (elem == kF32 ? 4 : 2) % 16 == 0; }

}  // namespace few_rows

cudaError_t launch_product_few(const GroupProduct& g, int num_sms, cudaStream_t stream) {
    using namespace few_rows;
    if (g.rows > kRows * (int64_t)g.G || g.op != kProductFwd || g.elem != kBF16 || g.K % 8 || ((uintptr_t)g.b & 15)) return cudaErrorNotSupported;
    Args a = {};
    a.offsets = g.offsets;
    a.rows = g.rows;
    a.G = g.G;
    a.N = g.N;
    a.K = g.K;
    a.x = g.a;
    a.ldx = g.lda;
    a.fast = g.K % kChunk == 0 && aligned16(g.a, g.rows > 1 ? g.lda : 0, kBF16);
    a.w = (const bf16*)g.b;
    a.out = g.out;
    a.out_elem = g.out_elem;
    a.ldo = g.ldo;
    return launch<0, bf16, bf16>(a, num_sms, stream);
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
    const int bytes = kChunk / g.w.group * (g.w.scale_elem == kF32 ? 4 : 2);  // scales of a chunk
    a.fast = g.K % kChunk == 0 && aligned16(g.x, g.rows > 1 ? g.ldx : 0, g.elem) && (uintptr_t)g.w.scales % bytes == 0 && (uintptr_t)g.w.zeros % (kChunk / g.w.group) == 0;
    if (g.w.group == 32) return launch_coded<5>(a, g.elem, num_sms, stream);
    if (g.w.group == 64) return launch_coded<6>(a, g.elem, num_sms, stream);
    return launch_coded<7>(a, g.elem, num_sms, stream);
}

}  // namespace moe

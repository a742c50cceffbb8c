// What the two kernels for a few rows a group share (product_few.cu,
// product_few_bulk.cu): tiles, x as MMA operands, sums of the warps' parts.
#pragma once

#include "common.cuh"
#include "groups.cuh"
#include "int4.cuh"
#include "internal.h"

namespace moe {
namespace few_rows {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kF = 16, kRows = 8;   // features and rows of a tile
constexpr int kChunk = 128;         // columns a warp takes at a time

struct Args {
    const int32_t* offsets;
    int rows, G, N, K;
    const void* x;
    int64_t ldx;
    const bf16* w;
    Int4 q;
    void* out;
    int out_elem;
    int64_t ldo;
    uint32_t* err;
    int64_t spin_ns;
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
constexpr int kMaxTiles = 2 * kProductMaxG;  // (8 rows a group; fp32 rows may be more)
struct TileList {
    GroupTable groups;
    uint32_t list[kMaxTiles];
};
// F features a tile; their partial sums, for two units in turn or one.
template <int F = kF, int BUFS = 2> struct Tables : TileList {
    static constexpr int kPitch = F + 4;  // floats between the rows of a partial tile: lanes hit different banks
    float part[BUFS][kWarps][kRows * kPitch];
};
struct Unit {
    int g, f0, row0, n;  // group, first feature, first row of the tile and how many
};
template <int F = kF> __device__ __forceinline__ Unit unit_at(int u, int FB, int G, const TileList& t) {
    Unit r;
    const int rt = u / FB;
    r.f0 = (u - rt * FB) * F;
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

// The tables, and the number of units with tiles of F features: a block at or
// past it has none, and must not ask for one (its entry of the list is not
// written).  The grid is made for the most tiles that the rows of x may give,
// which are more than these where rows belong to no group or groups are empty.
template <int F = kF> __device__ __forceinline__ int build_tables(TileList& t, const Args& p) {
    if (threadIdx.x < 32) group_table(t.groups, p.offsets, p.G, p.rows, kRows);
    __syncthreads();
    pdl_release();
    if (t.groups.tiles[p.G] <= kMaxTiles)
        for (int i = threadIdx.x; i < p.G; i += blockDim.x)
            for (int j = t.groups.tiles[i], n = 0; j < t.groups.tiles[i + 1]; ++j, ++n) t.list[j] = (uint32_t)i | (uint32_t)n << 11;
    __syncthreads();
    return t.groups.tiles[p.G] * ((p.N + F - 1) / F);
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: no place in L1, which x keeps.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Eight columns of x as the parts of MMA operands: one for bf16; for fp32
// three, each the leading eight bits of what the ones before leave, the second
// times 2^8 and the third times 2^16: within range for the largest numbers,
// and no bits lost below bf16's smallest for the smallest.
template <typename T> struct Parts { static constexpr int n = sizeof(T) == 4 ? 3 : 1; uint32_t v[n][4]; };

template <bool VEC> __device__ __forceinline__ void load_x(const bf16* x, Parts<bf16>& o) {
    if constexpr (VEC) {
        const uint4 v = *(const uint4*)x;
        o.v[0][0] = v.x; o.v[0][1] = v.y; o.v[0][2] = v.z; o.v[0][3] = v.w;
    } else {
        const uint16_t* h = (const uint16_t*)x;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[0][j] = (uint32_t)h[2 * j] | (uint32_t)h[2 * j + 1] << 16;
    }
}
template <bool VEC> __device__ __forceinline__ void load_x(const float* x, Parts<float>& o) {
    float f[8];
    if constexpr (VEC) {
        *(float4*)f = *(const float4*)x;
        *(float4*)(f + 4) = *((const float4*)x + 1);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = x[j];
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

// Multiplies eight columns: features' pairs a (row g) and e (g + 8) of two
// bf16 each by x's parts, a sum for each part.
template <int N>
__device__ __forceinline__ void mma8(float (&sum)[N][4], const uint32_t (&a)[4], const uint32_t (&e)[4], const uint32_t (&x)[N][4]) {
#pragma unroll
    for (int m = 0; m < N; ++m) {
        mma(sum[m], a[0], e[0], a[1], e[1], x[m][0], x[m][1]);
        mma(sum[m], a[2], e[2], a[3], e[3], x[m][2], x[m][3]);
    }
}
// acc += scales (of features g and g + 8) times the parts' sum.
template <int N> __device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&sum)[N][4], const float (&s)[2]) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        float v = sum[0][m];
        if constexpr (N == 3) v += fmaf(sum[2][m], 0x1p-16f, sum[1][m] * 0x1p-8f);
        acc[m] = fmaf(s[m >> 1], v, acc[m]);
    }
}
// 128 + zero, of column group gr, in both halves.
__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z, int gr) {
    const uint32_t v = __byte_perm(z, 0x43434343u, 0x4040 + 0x0101 * gr);
    return *(const __nv_bfloat162*)&v;
}

// A warp's sums to its partial tile: D(g, 2t), D(g, 2t + 1), D(g + 8, 2t) and
// D(g + 8, 2t + 1), feature and row.
template <int F = kF> __device__ __forceinline__ void put_part(float* mine, const float (&acc)[4], int g, int t) {
#pragma unroll
    for (int m = 0; m < 4; ++m) mine[(2 * t + (m & 1)) * (F + 4) + g + 8 * (m >> 1)] = acc[m];
}
// A feature's result for a row, where the tiles' sum is no finite number: a
// group's sum may have overflown before its scale.  By whole warps, W lanes of
// which have the same row (x; nullptr: none); again: whether this lane's is to be
// summed.  A NaN of the row, or of the feature's scales, is one of the result and
// needs no second sum: the lanes look for it together (80 rows of 128 experts,
// 1024 x 4096, a call on a cold cache: 83 us, of NaN 145, 2400 when each was summed
// again, of infinities, which are, 1650).
template <int LG, typename T, int W>
__device__ __forceinline__ float sum_again(const Args& p, const T* x, int64_t row, int nb, bool again, float v) {
    const int lane = threadIdx.x & 31;
    bool nan = false;
    if (x)
        for (int k = lane % W; k < p.K; k += W) nan |= isnan(to_f32(x[k]));
    nan = (__ballot_sync(0xffffffffu, nan) >> (lane & ~(W - 1)) & (uint32_t)((1ull << W) - 1)) != 0;
    if (!again) return v;
    auto scale = [&](int g) {
        const int64_t at = row * nb + g;
        return p.q.scale_elem == kF32 ? ((const float*)p.q.scales)[at] : to_f32(((const bf16*)p.q.scales)[at]);
    };
    for (int g = 0; g < nb && !nan; ++g) nan = isnan(scale(g));
    if (nan) return __int_as_float(0x7FC00000);
    v = 0.0f;
    for (int g = 0; g < nb; ++g) {
        const float s = scale(g);
        const int z = p.q.zeros ? p.q.zeros[row * nb + g] : 8;
        const uint8_t* c = p.q.codes + row * (p.K / 2);
        for (int k = g << LG; k < min(p.K, (g + 1) << LG); k += 2) {
            const int cd = c[k >> 1];
            v = fmaf(to_f32(x[k]), (float)((cd & 15) - z) * s, v);
            v = fmaf(to_f32(x[k + 1]), (float)((cd >> 4) - z) * s, v);
        }
    }
    return v;
}

// The partial tiles' sum, stored; by kThreads threads.
template <int LG, typename T, int F = kF>
__device__ __forceinline__ void finish(const Args& p, const float (*part)[kRows * (F + 4)], const Unit& cur, int nb) {
    const int f = threadIdx.x & (F - 1);
    for (int r0 = 0; r0 < kRows; r0 += kThreads / F) {
        const int r = r0 + (int)threadIdx.x / F;
        const bool in = r < cur.n && cur.f0 + f < p.N;
        float v = 0.0f;
        if (in) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += part[w][r * (F + 4) + f];
        }
        if constexpr (LG != 0) {
            const bool again = !isfinite(v);
            if (__any_sync(0xffffffffu, again))
                v = sum_again<LG, T, (F < 32 ? F : 32)>(p, r < cur.n ? (const T*)p.x + (int64_t)(cur.row0 + r) * p.ldx : nullptr,
                                                       (int64_t)cur.g * p.N + cur.f0 + f, nb, again, v);
        }
        if (!in) continue;
        const int64_t at = (int64_t)(cur.row0 + r) * p.ldo + cur.f0 + f;
        if (p.out_elem == kF32) ((float*)p.out)[at] = v;
        else ((bf16*)p.out)[at] = __float2bfloat16_rn(v);
    }
}

}  // namespace few_rows
}  // namespace moe

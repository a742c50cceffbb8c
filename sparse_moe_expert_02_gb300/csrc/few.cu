// The whole layer for a few tokens (moe_forward_few): one persistent
// cooperative kernel, a CTA per SM.
//
// At these sizes the layer is its weights: each touched expert's three
// matrices pass through the SMs once (T = 1, D = 4096, I = 1024, top_k = 10:
// 277 MB in bf16, 73 MB in 4 bits) and everything else is latency.  So the
// kernel is a weight stream.  A producer warp fills two rings of 16 KB
// stages by TMA, as far ahead as shared memory allows and across the phases
// below; each ring feeds a group of eight consumer warps, which
// split a tile's columns and multiply it with mma.sync, the weight rows as
// the M side and the tokens as the N side (16 x 8): a tile costs the same for
// one token as for eight, and one group multiplies while the other reduces.
// tcgen05 would want 128 rows and its operands in its own layout; at HBM
// speed mma.sync is far from its limit.
//
//   P0  router logits: the CTA's share of the E rows; arrive at barrier 1
//   P1  shared expert's gate/up (needs no routing): its share of I features
//   --  wait for barrier 1; every CTA takes the top-k of all T tokens and
//       builds the same list of distinct experts
//   P2  routed gate/up: its share of the (expert, feature) pairs, in tiles of
//       8 gate rows and the 8 up rows of the same features, so that a
//       thread's accumulators hold both and SwiGLU is local; h to global
//   --  barrier 2 (the ring is already filling with P3's weights)
//   P3  down: the CTA's share of the D output rows, over all experts, h
//       brought into shared memory (and quantised) a batch of experts at a
//       time: the sum over experts stays in registers, in list order, so
//       there are no atomics and no partial outputs, and the result does not
//       vary
//
// Work is split to the row (flattened ranges, tiles cut where a range or an
// expert ends), so the SMs' byte counts differ by a row at most.  Eight rows
// come as one box of 8 x 1 KB (a copy costs the SM some 80 cycles to issue
// whatever its size: with one bulk copy a row the bf16 layer took 100 us at
// T = 1 instead of 70); the rows left over come as row copies, longer where
// there are few.  A dot product does not mind the order of its terms, so each
// lane takes 16 contiguous bytes (4-bit: 4) of its row and the same columns
// of its token as fragments; no shuffles, no ldmatrix.
//
// Arithmetic, as moe_forward's: products of weights and activations as the
// type holds them (x and h quantised for FP8 and MXFP4; h as fp16 against
// W_down's fp16 copy, or as a bf16 pair, for bf16), fp32 accumulation, block
// scales applied in fp32 to each block's partial sum.  E4M3 codes are MMA
// operands as they are; E2M1 codes become E4M3 by two shifts and masks
// (their bits placed in E4M3's exponent and mantissa read as 2^-6 of the
// value), against activations held as 2^6 of theirs (at most 384), so the
// products are exact.
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu
}
namespace few {

constexpr int NC = 8;                        // warps of a consumer group
constexpr int NG = 2;                        // consumer groups
constexpr int kCons = 32 * NC * NG;          // consumer threads
constexpr int kThreads = kCons + 32;         // the last warp is the producer
constexpr int kBoxRow = 1024;                // bytes of a box's rows: 8 KB boxes, two a stage
constexpr int kMaxPairs = kFewMax * 32;      // (token, slot) pairs
constexpr int kMaxStages = 12;
constexpr int W_HILO = 4;                    // MOE_BF16 with h as a bf16 pair against a bf16 W_down

// Per weight type: bytes of 64 columns; columns a warp takes at a time (its
// slice, `in` bytes: one swizzled line of a box); bytes of an activation x
// and h; activation scales per 128 columns.
template <int W> struct Tr;
template <> struct Tr<MOE_F32> { static constexpr int b64 = 256, slice = 32, in = 128, xpad = 16, xb = 4, hb = 4, nsc = 0; };
template <> struct Tr<MOE_BF16> { static constexpr int b64 = 128, slice = 64, in = 128, xpad = 64, xb = 2, hb = 2, nsc = 0; };
template <> struct Tr<W_HILO> { static constexpr int b64 = 128, slice = 64, in = 128, xpad = 64, xb = 2, hb = 4, nsc = 0; };
template <> struct Tr<MOE_FP8_E4M3_B128> { static constexpr int b64 = 64, slice = 128, in = 128, xpad = 64, xb = 1, hb = 1, nsc = 1; };
template <> struct Tr<MOE_MXFP4> { static constexpr int b64 = 32, slice = 128, in = 64, xpad = 64, xb = 1, hb = 1, nsc = 4; };

__host__ __device__ constexpr int up(int v, int a) { return (v + a - 1) / a * a; }
__host__ __device__ constexpr int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ constexpr int imax(int a, int b) { return a > b ? a : b; }

// Bytes of n columns (n a multiple of 64).
template <int W> __host__ __device__ constexpr int bytes_of(int n) { return n / 64 * Tr<W>::b64; }

template <int W> struct Plan {
    static constexpr int kc = kBoxRow / Tr<W>::b64 * 64;         // columns of a box: one or two slices a warp
    static constexpr int data = 16 * (kBoxRow + 16);             // row copies: 16 bytes between rows
    static constexpr int scales = W == MOE_MXFP4 ? 1024 : 0;     // scale bytes of a stage
    static constexpr int stage = up(data + scales, 1024);        // boxes are swizzled by address
    static constexpr int rslice = W == MOE_F32 ? 32 : 64;        // columns of router rows a warp takes
    static constexpr int eb = W == MOE_F32 ? 4 : 2;              // bytes of a router weight
    // columns of a stage of n row copies (at most 16) of rows of K columns
    __host__ __device__ static constexpr int row_cols(int n, int K) { return imin(K, (16 * kBoxRow / n & -256) / Tr<W>::b64 * 64); }
};
// Shared-memory row strides of x and of h (one chunk of columns), and the
// bytes of a row's scales.
template <int W> __host__ __device__ constexpr int x_stride(int D) { return up(D * Tr<W>::xb, 128) + Tr<W>::xpad; }
template <int W> __host__ __device__ constexpr int h_stride(int I) { return up(imin(I, Plan<W>::kc) * Tr<W>::hb, 128) + Tr<W>::xpad; }
template <int W> __host__ __device__ constexpr int x_scales(int D) { return D / 128 * Tr<W>::nsc * 4; }
template <int W> __host__ __device__ constexpr int h_scales(int I) { return imin(I, Plan<W>::kc) / 128 * Tr<W>::nsc * 4; }

// Fixed shared memory: barriers and flags, the expert list, reductions.
struct Misc {
    uint64_t full[kMaxStages], empty[kMaxStages], list_ready;
    int abort, n;               // n: distinct experts
    uint32_t scan[NC * NG];
    uint32_t mask[512];         // token bits of each expert (two a word), then its place in the list
    uint16_t expert[kMaxPairs]; // the list: expert, token bits, first row of h
    uint16_t tokens[kMaxPairs];
    uint16_t hrow[kMaxPairs + 1];
    uint16_t sel[kMaxPairs];    // [T, k] chosen experts
    float selw[kMaxPairs];
    float wt[kMaxPairs];        // routing weight of each row of h
    float4 red[NG][2 * NC * 32];  // each group: [2 buffers][warp][lane], or [warp][2][lane] with two token tiles
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return tc::smem_u32(p); }
// One lane of the converged producer warp, which runs its loops with all
// lanes: what the copies take is then in uniform registers (issued from one
// lane's own branch, a copy costs some 80 cycles more).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.b32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void group_sync(int grp) { asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * NC) : "memory"); }
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 7, %0;" ::"n"(kCons) : "memory"); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row, int line) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(line), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&h;
}
// Two E8M0 scale bytes as floats (exact; 255: NaN).
__device__ __forceinline__ void e8m0_floats(uint16_t two, float& a, float& b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(two));
    a = __uint_as_float(r << 16);
    b = __uint_as_float(r & 0xFFFF0000u);
}

// A lane's weight rows, g and g + 8 of a tile, at a slice: 16-byte piece c
// lies at `p + (16 c ^ x)`.
struct RowPair {
    const uint8_t *a, *b;
    int xa, xb;
};

// Products of 16 weight rows with NT tiles of 8 tokens over one slice of
// columns; lane (g, q) = (lane / 4, lane % 4) accumulates rows g and g + 8 of
// tokens 2q and 2q + 1.  xa[n]: this lane's token row (token 8 n + g) at the
// slice.

// 16-bit rows, 64 columns: a lane's words are columns 32 i + 8 q + 2 j.
template <int NT, bool F16>
__device__ __forceinline__ void dot16(const RowPair& r, const uint8_t* const (&xa)[NT], float (&c)[NT][4]) {
    const int q = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int o = 64 * i + q * 16;
        const uint4 a = *(const uint4*)(r.a + (o ^ r.xa)), d = *(const uint4*)(r.b + (o ^ r.xb));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 b = *(const uint4*)(xa[n] + o);
            if (F16) {
                mma_f16(c[n], a.x, d.x, a.y, d.y, b.x, b.y);
                mma_f16(c[n], a.z, d.z, a.w, d.w, b.z, b.w);
            } else {
                mma_bf16(c[n], a.x, d.x, a.y, d.y, b.x, b.y);
                mma_bf16(c[n], a.z, d.z, a.w, d.w, b.z, b.w);
            }
        }
    }
}
// E4M3 rows, 128 columns: a lane's bytes are columns 64 i + 16 q + 0..15;
// sa, sb: the block scales of rows g and g + 8, sx: of the two tokens.
template <int NT>
__device__ __forceinline__ void dot_fp8(const RowPair& r, const uint8_t* const (&xa)[NT], float sa, float sb, const float (&sx)[NT][2],
                                        float (&acc)[NT][4]) {
    const int q = threadIdx.x & 3;
    float c[NT][4] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int o = 64 * i + q * 16;
        const uint4 a = *(const uint4*)(r.a + (o ^ r.xa)), d = *(const uint4*)(r.b + (o ^ r.xb));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 b = *(const uint4*)(xa[n] + o);
            mma_e4m3(c[n], a.x, d.x, a.y, d.y, b.x, b.y);
            mma_e4m3(c[n], a.z, d.z, a.w, d.w, b.z, b.w);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        acc[n][0] = fmaf(c[n][0], sa * sx[n][0], acc[n][0]);
        acc[n][1] = fmaf(c[n][1], sa * sx[n][1], acc[n][1]);
        acc[n][2] = fmaf(c[n][2], sb * sx[n][0], acc[n][2]);
        acc[n][3] = fmaf(c[n][3], sb * sx[n][1], acc[n][3]);
    }
}
// E2M1 rows, 128 columns: a lane's word i is columns 32 i + 8 q + 0..7; ka,
// kb: the four scale bytes of rows g and g + 8, sx: the scales of the two
// tokens.  The activations lie so that a lane's 16 bytes at 64 j + 16 q hold
// the even and odd columns of its words 2 j and 2 j + 1.
template <int NT>
__device__ __forceinline__ void dot_mx(const RowPair& r, const uint8_t* const (&xa)[NT], uint32_t ka, uint32_t kb,
                                       const float4 (&sx)[NT][2], float (&acc)[NT][4]) {
    const int q = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float sa[2], sb[2];
        e8m0_floats((uint16_t)(ka >> (16 * j)), sa[0], sa[1]);
        e8m0_floats((uint16_t)(kb >> (16 * j)), sb[0], sb[1]);
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = *(const uint4*)(xa[n] + 64 * j + q * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = 32 * j + 16 * h;
            const uint32_t a = *(const uint32_t*)(r.a + (o ^ r.xa) + q * 4), d = *(const uint32_t*)(r.b + (o ^ r.xb) + q * 4);
            const uint32_t ae = ((a << 4) & 0x80808080u) | ((a << 2) & 0x1C1C1C1Cu), ao = (a & 0x80808080u) | ((a >> 2) & 0x1C1C1C1Cu);
            const uint32_t de = ((d << 4) & 0x80808080u) | ((d << 2) & 0x1C1C1C1Cu), od = (d & 0x80808080u) | ((d >> 2) & 0x1C1C1C1Cu);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float c[4] = {};
                mma_e4m3(c, ae, de, ao, od, h ? b[n].z : b[n].x, h ? b[n].w : b[n].y);
                const float s0 = j ? (h ? sx[n][0].w : sx[n][0].z) : (h ? sx[n][0].y : sx[n][0].x);
                const float s1 = j ? (h ? sx[n][1].w : sx[n][1].z) : (h ? sx[n][1].y : sx[n][1].x);
                acc[n][0] = fmaf(c[0], sa[h] * s0, acc[n][0]);
                acc[n][1] = fmaf(c[1], sa[h] * s1, acc[n][1]);
                acc[n][2] = fmaf(c[2], sb[h] * s0, acc[n][2]);
                acc[n][3] = fmaf(c[3], sb[h] * s1, acc[n][3]);
            }
        }
    }
}
// fp32 rows, 32 columns, on the CUDA cores: the same accumulators; t0 and t1
// point at the 32 columns of the lane's two tokens.
__device__ __forceinline__ void dot_f32(const RowPair& r, const uint8_t* t0, const uint8_t* t1, float (&acc)[4]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float4 a = *(const float4*)(r.a + (16 * k ^ r.xa)), d = *(const float4*)(r.b + (16 * k ^ r.xb)),
                     x = ((const float4*)t0)[k], y = ((const float4*)t1)[k];
        acc[0] = fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, acc[0]))));
        acc[1] = fmaf(a.x, y.x, fmaf(a.y, y.y, fmaf(a.z, y.z, fmaf(a.w, y.w, acc[1]))));
        acc[2] = fmaf(d.x, x.x, fmaf(d.y, x.y, fmaf(d.z, x.z, fmaf(d.w, x.w, acc[2]))));
        acc[3] = fmaf(d.x, y.x, fmaf(d.y, y.y, fmaf(d.z, y.z, fmaf(d.w, y.w, acc[3]))));
    }
}

// 16 values (of a group that `lanes` neighbouring lanes share) to operand
// bytes at dst (if `on`); returns the scale.
__device__ __forceinline__ float quant16_fp8(const float (&v)[16], uint8_t* dst, bool on) {  // 8 lanes: 128 columns
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
    const float f = a > 0.0f ? 448.0f / a : 1.0f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = f32x2_to_e4m3x2(v[4 * i] * f, v[4 * i + 1] * f) | ((uint32_t)f32x2_to_e4m3x2(v[4 * i + 2] * f, v[4 * i + 3] * f) << 16);
    if (on) *(uint4*)dst = make_uint4(w[0], w[1], w[2], w[3]);
    return a > 0.0f ? a / 448.0f : 1.0f;
}
// 2 lanes: 32 columns (lane parity `half`); dst: the operand bytes of the
// 64-column group that holds the block, `odd` the block's place in it.
__device__ __forceinline__ float quant16_mx(const float (&v)[16], uint8_t* dst, int half, int odd, bool on) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t s = mx_scale_byte(m);
    const float f = s == 255u ? 0.0f : mx_inv_scale(s);
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // eight columns: quad lane 2 half + u of the fragment
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // E2M1 of the pair, then 2^6 of it as E4M3 (exact)
            uint32_t h;
            uint16_t e;
            asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n"
                : "=r"(h)
                : "f"(v[8 * u + 2 * i] * f), "f"(v[8 * u + 2 * i + 1] * f));
            const __half2 h64 = __hmul2(*(const __half2*)&h, __floats2half2_rn(64.0f, 64.0f));
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(e) : "r"(*(const uint32_t*)&h64));
            p[i] = e;
        }
        const uint32_t lo = p[0] | p[1] << 16, hi = p[2] | p[3] << 16;
        uint2 o = make_uint2(__byte_perm(lo, hi, 0x6420), __byte_perm(lo, hi, 0x7531));
        if (s == 255u) o = make_uint2(0, 0);
        if (on) *(uint2*)(dst + (2 * half + u) * 16 + odd * 8) = o;
    }
    return mx_scale(s);
}

// Top-k of one token's logits by one warp: largest first, the lower index on
// a tie; non-finite logits count as -inf (and are reported).  Each lane keeps
// its four best in order and refills when they are used up.
template <int J>
__device__ __forceinline__ void topk_token(const FewParams& p, int t, Misc& m, uint32_t& bad) {
    const int lane = threadIdx.x & 31;
    uint32_t key[J];  // order-preserving image of the logit; 0: no expert
    bool finite = true;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane + 32 * j;
        key[j] = e < p.E ? __float_as_uint(__ldcg(p.logits + (int64_t)t * p.E + e)) : 0u;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (lane + 32 * j < p.E) {
            uint32_t u = key[j];
            if ((u & 0x7F800000u) == 0x7F800000u) {
                finite = false;
                u = 0xFF800000u;
            }
            if (u == 0x80000000u) u = 0u;  // -0 and +0 tie
            key[j] = (u >> 31) ? ~u : (u | 0x80000000u);
        }
    }
    if (!__all_sync(0xffffffffu, finite)) bad |= 1u << t;
    constexpr int H = 4;
    uint32_t hk[H];
    int hj[H];
    // the H best that come after (ak, aj) in the order
    auto build = [&](uint32_t ak, int aj) {
#pragma unroll
        for (int h = 0; h < H; ++h) hk[h] = 0u, hj[h] = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint32_t kj = key[j];
            int ij = j;
            if (kj < ak || (kj == ak && j > aj)) {
#pragma unroll
                for (int h = 0; h < H; ++h) {  // insert: equal keys keep their order
                    const bool above = kj > hk[h];
                    const uint32_t tk = above ? hk[h] : kj;
                    const int tj = above ? hj[h] : ij;
                    hk[h] = above ? kj : hk[h];
                    hj[h] = above ? ij : hj[h];
                    kj = tk;
                    ij = tj;
                }
            }
        }
    };
    build(0xFFFFFFFFu, -1);
    uint32_t z = 0;
    int used = 0;
    for (int r = 0; r < p.k; ++r) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, hk[0]);
        const uint32_t e = __reduce_min_sync(0xffffffffu, hk[0] == top ? (uint32_t)(lane + 32 * hj[0]) : 0xFFFFFFFFu);
        if (lane == r) {
            z = top;
            m.sel[t * p.k + r] = (uint16_t)e;
        }
        if ((e & 31u) == (uint32_t)lane) {
            const uint32_t lk = hk[0];
            const int lj = hj[0];
#pragma unroll
            for (int h = 0; h + 1 < H; ++h) hk[h] = hk[h + 1], hj[h] = hj[h + 1];
            hk[H - 1] = 0u;
            if (++used == H) {
                build(lk, lj);
                used = 0;
            }
        }
    }
    const float zv = __uint_as_float((z >> 31) ? (z & 0x7FFFFFFFu) : ~z);
    const float zmax = __shfl_sync(0xffffffffu, zv, 0);
    const float ex = lane < p.k ? expf(zv - zmax) : 0.0f;
    float sum = ex;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < p.k) m.selw[t * p.k + lane] = ex / sum;
}

// Grid barrier on a counter that only grows (every launch adds whole
// multiples of the grid): arrive returns the count to wait for.
__device__ __forceinline__ unsigned long long grid_arrive(unsigned long long* bar) {
    __threadfence();
    return (atomicAdd(bar, 1ull) / gridDim.x + 1) * gridDim.x;
}
__device__ __forceinline__ bool grid_wait(const unsigned long long* bar, unsigned long long target, int64_t limit_ns, volatile int* abort) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        unsigned long long v;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(bar) : "memory");
        if (v >= target) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if ((int64_t)(t - t0) > limit_ns) return false;
        }
    }
}

// The next tile of each group from rows (or features) [from, to): full tiles
// while there are two, then one and what is left, then halves.
struct Pair {
    int at0, n0, n1;
    __device__ __forceinline__ Pair(int from, int to, int most) {
        const int rem = to - from;
        at0 = from;
        n0 = rem >= most ? most : (rem + 1) / 2;
        n1 = min(rem - n0, most);
    }
    __device__ __forceinline__ int at(int grp) const { return grp ? at0 + n0 : at0; }
    __device__ __forceinline__ int n(int grp) const { return grp ? n1 : n0; }
    __device__ __forceinline__ int end() const { return at0 + n0 + n1; }
};

// P3 goes through the shared expert (x = -1) and the n listed ones in
// batches: as many whole experts as fit h's buffer.  Rows of h: listed
// experts' first, then the shared one's (Tk ..).
struct Batch {
    int x0, x1;    // experts [x0, x1)
    int shared;    // rows of the shared expert in it (T or 0), first in the buffer
    int row0;      // h row of its first listed expert
    int rows;      // rows in the buffer
};
__device__ __forceinline__ Batch next_batch(const Misc& m, int x0, int n, int T, int cap) {
    Batch b;
    b.x0 = x0;
    b.shared = x0 < 0 ? T : 0;
    const int first = max(x0, 0);
    b.row0 = m.hrow[first];
    int x = first;
    while (x < n && b.shared + m.hrow[x + 1] - b.row0 <= cap) ++x;
    b.x1 = x;
    b.rows = b.shared + m.hrow[x] - b.row0;
    return b;
}

// Weight matrices as [line][row][in] boxes of 8 rows (gate, up, down), and
// their scale bytes in 4 bits.
struct Maps {
    CUtensorMap w[3], s[3];
};

// Columns of a stage of a tile of n features (n gate rows and n up rows), and
// of n router rows.
template <int W> __device__ __forceinline__ int tile_cols(int n, int K) { return n == 8 || n == 0 ? Plan<W>::kc : Plan<W>::row_cols(2 * n, K); }
template <int W> __device__ __forceinline__ int router_cols(int n, int K) { return min(K, (16 * kBoxRow / n & -256) / Plan<W>::eb); }

template <int W, int NT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ Maps maps) {
    using P = Plan<W>;
    constexpr bool kScaled = W == MOE_FP8_E4M3_B128 || W == MOE_MXFP4;
    constexpr int kSlice = Tr<W>::slice;
    extern __shared__ __align__(1024) uint8_t smem[];
    Misc& m = *(Misc*)smem;
    uint8_t* act = smem + up(sizeof(Misc), 128);  // x (P1, P2), then batches of h (P3)
    uint8_t* ring = smem + p.ring_at;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int cta = blockIdx.x, grid = gridDim.x;
    const int D = p.D, I = p.I, E = p.E, T = p.T, k = p.k;
    const int64_t lim = p.spin_ns;
    volatile int* abort = &m.abort;
    if (threadIdx.x == kCons) {
        for (int s = 0; s < NG * p.stages; ++s) {
            tc::mbar_init(smem_u32(m.full + s), 1);
            tc::mbar_init(smem_u32(m.empty + s), NC);
        }
        tc::mbar_init(smem_u32(&m.list_ready), 1);
        m.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        // this call's error word; only waits that run out record an error
        // before barrier 1
        if (cta == 0 && p.tok0 == 0) p.err[0] = p.err[1] = p.err[2] = p.err[3] = 0;
    }
    __syncthreads();

    // shares of this CTA: router rows, shared features, output rows
    const int e_lo = (int)((int64_t)E * cta / grid), e_hi = (int)((int64_t)E * (cta + 1) / grid);
    const int f_lo = (int)((int64_t)I * cta / grid), f_hi = (int)((int64_t)I * (cta + 1) / grid);
    const int d_lo = (int)((int64_t)D * cta / grid), d_hi = (int)((int64_t)D * (cta + 1) / grid);

    if (warp == NC * NG) {
        // ------------------------------------------------------- producer
        const uint32_t ring0 = smem_u32(ring);
        int next[NG] = {0, p.stages};  // group g's ring: stages [g * p.stages, (g + 1) * p.stages)
        uint32_t phases[NG] = {0, 0};
        bool ok = true;
        auto wait_stage = [&](int grp) -> bool {
            if (!ok) return false;
            ok = tc::mbar_wait(smem_u32(m.empty + next[grp]), phases[grp] ^ 1, lim, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok && lane == 0 && !*abort) {
                record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 41, cta, 0);
                *abort = 1;
            }
            return ok;
        };
        auto advance = [&](int grp) {
            if (++next[grp] == (grp + 1) * p.stages) {
                next[grp] = grp * p.stages;
                phases[grp] ^= 1;
            }
        };
        // A stage of a group's ring: rows from row0 of matrix wa and from row1 of wb (0 gate, 1 up, 2
        // down), na and nb of them, columns c0 .. of K; whole boxes of eight, or row copies of `cols`.
        auto fill = [&](int grp, int wa, int64_t row0, int na, int wb, int64_t row1, int nb, int K, int c0, int cols) {
            if (!wait_stage(grp)) return;
            if (elect_one()) {
                const uint32_t bar = smem_u32(m.full + next[grp]), base = ring0 + next[grp] * P::stage;
                const int bytes = bytes_of<W>(cols), sbytes = cols / 32;
                const bool boxa = na == 8, boxb = nb == 8;
                const uint32_t sc = base + P::data;
                const bool scaled = W == MOE_MXFP4 && p.tma_scales;
                // where the second region's rows and scales start
                const uint32_t base1 = base + (boxa ? 8 * kBoxRow : na * (bytes + 16)), sc1 = sc + (boxa ? 8 * P::kc / 32 : na * sbytes);
                uint32_t total = (boxa ? 8 * kBoxRow : na * bytes) + (boxb ? 8 * kBoxRow : nb * bytes);
                if (scaled) total += (boxa ? 8 * P::kc / 32 : na * sbytes) + (boxb ? 8 * P::kc / 32 : nb * sbytes);
                tc::mbar_expect_tx(bar, total);
                const int line = bytes_of<W>(c0) / Tr<W>::in;
                auto rows = [&](int w, int64_t row, int n, uint32_t dst, uint32_t sdst) {
                    const uint8_t* src = (const uint8_t*)(w == 0 ? p.w_gate : w == 1 ? p.w_up : p.w_down) + row * bytes_of<W>(K) + bytes_of<W>(c0);
                    const uint8_t* ss = (const uint8_t*)(w == 0 ? p.s_gate : w == 1 ? p.s_up : p.s_down) + row * (K / 32) + c0 / 32;
                    for (int r = 0; r < n; ++r) {
                        bulk_load(dst + r * (bytes + 16), src + (int64_t)r * bytes_of<W>(K), bytes, bar);
                        if (scaled) bulk_load(sdst + r * sbytes, ss + (int64_t)r * (K / 32), sbytes, bar);
                    }
                };
                if (boxa) {
                    box_load(base, &maps.w[wa], bar, (int)row0, line);
                    if (scaled) tc::tma_load_2d(sc, &maps.s[wa], bar, c0 / 32, (int)row0);
                } else {
                    rows(wa, row0, na, base, sc);
                }
                if (boxb) {
                    box_load(base1, &maps.w[wb], bar, (int)row1, line);
                    if (scaled) tc::tma_load_2d(sc1, &maps.s[wb], bar, c0 / 32, (int)row1);
                } else {
                    rows(wb, row1, nb, base1, sc1);
                }
            }
            __syncwarp();
            advance(grp);
        };
        // P0: router rows (fp32 or bf16), row copies
        for (int e = e_lo; e < e_hi;) {
            const Pair t(e, e_hi, 16);
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) {
                const int n = t.n(grp);
                if (!n) continue;
                const int step = router_cols<W>(n, D);
                for (int c0 = 0; c0 < D; c0 += step) {
                    if (!wait_stage(grp)) break;
                    if (elect_one()) {
                        const uint32_t bar = smem_u32(m.full + next[grp]), base = ring0 + next[grp] * P::stage;
                        const int bytes = min(step, D - c0) * P::eb;
                        tc::mbar_expect_tx(bar, (uint32_t)(n * bytes));
                        const uint8_t* src = (const uint8_t*)p.w_router + ((int64_t)t.at(grp) * D + c0) * P::eb;
                        for (int r = 0; r < n; ++r) bulk_load(base + r * (bytes + 16), src + (int64_t)r * D * P::eb, bytes, bar);
                    }
                    __syncwarp();
                    advance(grp);
                }
            }
            e = t.end();
        }
        // features of expert e, a tile for each group: gate rows, then the up rows of the same features
        auto gateup = [&](int e, const Pair& t) {
            const int step0 = tile_cols<W>(t.n(0), D), step1 = tile_cols<W>(t.n(1), D);
            for (int i = 0, c0 = 0, c1 = 0; c0 < D || c1 < D; ++i, c0 += step0, c1 += step1) {
                const int64_t row = (int64_t)e * I;
                if (c0 < D) fill(0, 0, row + t.at(0), t.n(0), 1, row + t.at(0), t.n(0), D, c0, min(step0, D - c0));
                if (c1 < D && t.n(1)) fill(1, 0, row + t.at(1), t.n(1), 1, row + t.at(1), t.n(1), D, c1, min(step1, D - c1));
            }
        };
        // P1: the shared expert
        for (int f = f_lo; f < f_hi;) {
            const Pair t(f, f_hi, 8);
            gateup(E, t);
            f = t.end();
        }
        // P2: the routed experts, once the list is there
        if (ok && !tc::mbar_wait(smem_u32(&m.list_ready), 0, lim, abort)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        const int n = uniform(ok ? m.n : 0);
        const int64_t lo = (int64_t)n * I * cta / grid, hi = (int64_t)n * I * (cta + 1) / grid;
        for (int64_t f = lo; f < hi;) {
            const int pos = (int)(f / I);
            const int64_t first = (int64_t)pos * I;  // the expert's feature 0
            const Pair t((int)(f - first), (int)min((int64_t)I, hi - first), 8);
            gateup(uniform(m.expert[pos]), t);
            f = first + t.end();
        }
        // P3: down rows, pass by pass, batch by batch
        for (int d0 = d_lo; ok && d0 < d_hi; d0 += 16 * NG) {
            const Pair t(d0, min(d_hi, d0 + 16 * NG), 16);
            for (int bx = -1; bx < n;) {
                const Batch bt = next_batch(m, bx, n, T, p.hcap);
                for (int c0 = 0; c0 < I; c0 += P::kc) {
                    const int cols = min(P::kc, I - c0);
                    for (int x = bt.x0; x < bt.x1; ++x) {
                        const int64_t row = (int64_t)uniform(x < 0 ? E : m.expert[x]) * D;
#pragma unroll
                        for (int grp = 0; grp < NG; ++grp) {
                            const int nr = t.n(grp), r0 = t.at(grp);
                            if (nr) fill(grp, 2, row + r0, min(nr, 8), 2, row + r0 + 8, max(nr - 8, 0), I, c0, cols);
                        }
                    }
                }
                bx = bt.x1;
            }
        }
        if (!ok) tc::sleep_ns(200000);  // copies already issued land before the CTA leaves
        return;
    }

    // ---------------------------------------------------------- consumers
    // A wait that runs out raises the abort flag; every warp then runs on
    // through the same barriers (later waits return at once) to the end.
    const int grp = warp / NC, wg = warp - grp * NC;  // group, and warp of the group
    int stage = grp * p.stages;
    uint32_t phase = 0;
    const int tid = threadIdx.x;
    auto stage_wait = [&]() -> const uint8_t* {
        if (!tc::mbar_wait(smem_u32(m.full + stage), phase, lim, abort) && !*abort) {
            record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 42, cta, 0);
            *abort = 1;
        }
        __syncwarp();
        return ring + stage * P::stage;
    };
    auto stage_done = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(smem_u32(m.empty + stage));
        if (++stage == (grp + 1) * p.stages) {
            stage = grp * p.stages;
            phase ^= 1;
        }
    };
    // The tile rows this lane takes: rows 0 and 4 are neighbours in the
    // fragment order, 1 and 5, ...: their 16-byte pieces then lie in different
    // banks, swizzled or 16 bytes apart.
    const int rw = (g >> 1) | ((g & 1) << 2);
    const int swz = Tr<W>::in == 128 ? rw * 16 : ((rw >> 1) & 3) * 16;
    // This lane's two rows at slice c (of the stage's cols columns): na and
    // nb rows in the tile's halves, boxes where they are whole.
    auto rows_at = [&](const uint8_t* tile, int na, int nb, int cols, int c) {
        const int bytes = bytes_of<W>(cols), at = c / kSlice * Tr<W>::in;
        const bool boxa = na == 8, boxb = nb == 8;
        const uint8_t* tile1 = tile + (boxa ? 8 * kBoxRow : na * (bytes + 16));
        RowPair r;
        r.a = boxa ? tile + at * 8 + rw * Tr<W>::in : tile + min(rw, na - 1) * (bytes + 16) + at;
        r.xa = boxa ? swz : 0;
        r.b = boxb ? tile1 + at * 8 + rw * Tr<W>::in : nb ? tile1 + min(rw, nb - 1) * (bytes + 16) + at : r.a;
        r.xb = boxb ? swz : nb ? 0 : r.xa;
        return r;
    };
    // and, in 4 bits, their scale bytes: from the stage, or from memory (the
    // two rows' scale bytes at column 0 of the stage) where a row of scales is
    // no multiple of 16 bytes
    auto scales_at = [&](const uint8_t* tile, int na, int nb, int cols, int c, const uint8_t* ga, const uint8_t* gb, uint32_t& ka, uint32_t& kb) {
        if (p.tma_scales) {
            const uint8_t* sc = tile + P::data;
            const bool boxa = na == 8, boxb = nb == 8;
            const uint8_t* sc1 = sc + (boxa ? 8 * P::kc / 32 : na * (cols / 32));
            ka = *(const uint32_t*)(sc + (boxa ? rw * (P::kc / 32) : min(rw, na - 1) * (cols / 32)) + c / 32);
            kb = nb ? *(const uint32_t*)(sc1 + (boxb ? rw * (P::kc / 32) : min(rw, nb - 1) * (cols / 32)) + c / 32) : ka;
        } else {
            ka = __ldg((const uint32_t*)(ga + c / 32));
            kb = __ldg((const uint32_t*)(gb + c / 32));
        }
    };
    const int xstride = x_stride<W>(D);
    float* xsc = (float*)(act + up(T * xstride, 128));  // its scales, [T][per row]
    const int nxs = x_scales<W>(D) / 4;
    // x into shared memory, as the expert products read it
    if constexpr (!kScaled) {
        const int per = D * Tr<W>::xb / 16;
        for (int u = tid; u < T * per; u += kCons) {
            const int t = u / per, c = u - t * per;
            *(uint4*)(act + t * xstride + c * 16) = __ldg((const uint4*)p.x + (int64_t)t * per + c);
        }
    } else {
        const int per = D / 16, total = T * per;  // a unit: 16 columns; whole warps stay together
        for (int u0 = tid & ~31; u0 < total; u0 += kCons) {
            const int u = min(u0 + lane, total - 1), t = u / per, c = u - t * per;
            const uint4* src = (const uint4*)p.x + (int64_t)u * 2;
            const uint4 a = __ldg(src), b = __ldg(src + 1);
            float v[16];
            const bf16 *pa = (const bf16*)&a, *pb = (const bf16*)&b;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(pa[i]), v[8 + i] = __bfloat162float(pb[i]);
            uint8_t* row = act + t * xstride;
            if constexpr (W == MOE_FP8_E4M3_B128) {
                const float s = quant16_fp8(v, row + c * 16, u0 + lane < total);
                if ((c & 7) == 0 && u0 + lane < total) xsc[t * nxs + c / 8] = s;
            } else {
                const float s = quant16_mx(v, row + c / 4 * 64, c & 1, (c >> 1) & 1, u0 + lane < total);
                if ((c & 1) == 0 && u0 + lane < total) xsc[t * nxs + c / 2] = s;
            }
        }
    }
    for (int i = tid; i < 512; i += kCons) m.mask[i] = 0;

    // Sum of a tile's accumulators over the group's warps; the warp that returns true holds it in acc.
    auto reduce = [&](float (&acc)[NT][4], int turn) -> bool {
        float4* red = m.red[grp] + (NT == 1 ? (turn & 1) * NC * 32 : 0);
        const int owner = turn % NC;
#pragma unroll
        for (int n = 0; n < NT; ++n) red[(wg * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        group_sync(grp);
        if (wg == owner) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float4 s = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int w = 0; w < NC; ++w) {
                    const float4 v = red[(w * NT + n) * 32 + lane];
                    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
                }
                acc[n][0] = s.x; acc[n][1] = s.y; acc[n][2] = s.z; acc[n][3] = s.w;
            }
        }
        if (NT == 2) group_sync(grp);  // one buffer
        return wg == owner;
    };
    int turns = 0;  // reductions this group has made

    // -------------------------------------------------------------- P0
    // (x straight from global memory: its rows are in the caches, and the
    // products below read it quantised)
    for (int e = e_lo; e < e_hi;) {
        const Pair t(e, e_hi, 16);
        e = t.end();
        const int e0 = t.at(grp), ne = t.n(grp);
        if (!ne) continue;
        float acc[NT][4] = {};
        const int step = router_cols<W>(ne, D);
        for (int c0 = 0; c0 < D; c0 += step) {
            const int cols = min(step, D - c0), stride = cols * P::eb + 16;
            const uint8_t* tile = stage_wait();
            RowPair r = {tile + min(rw, ne - 1) * stride, tile + min(rw + 8, ne - 1) * stride, 0, 0};
            r.a += wg * P::rslice * P::eb;
            r.b += wg * P::rslice * P::eb;
            for (int c = wg * P::rslice; c < cols; c += NC * P::rslice) {
                const uint8_t* xg = (const uint8_t*)p.x + (int64_t)(c0 + c) * P::eb;
                if constexpr (W == MOE_F32) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        dot_f32(r, xg + (int64_t)min(8 * n + 2 * q, T - 1) * D * 4, xg + (int64_t)min(8 * n + 2 * q + 1, T - 1) * D * 4, acc[n]);
                } else {
                    const uint8_t* xa[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) xa[n] = xg + (int64_t)min(8 * n + g, T - 1) * D * 2;
                    dot16<NT, false>(r, xa, acc);
                }
                r.a += NC * P::rslice * P::eb;
                r.b += NC * P::rslice * P::eb;
            }
            stage_done();
        }
        if (reduce(acc, turns++)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = rw + 8 * r;
                    const float bias = p.b_router && row < ne ? __ldg(p.b_router + e0 + row) : 0.0f;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int tok = 8 * n + 2 * q + s;
                        if (row < ne && tok < T) p.logits[(int64_t)tok * E + e0 + row] = acc[n][2 * r + s] + bias;
                    }
                }
        }
    }
    consumers_sync();  // logits written, x in shared memory
    unsigned long long target = 0;
    if (tid == 0) target = grid_arrive(p.bar);

    bool overflow = false;
    // nf features from f0 of expert e; tokens: the tokens that want it, hrow: h row of a token
    auto gateup = [&](int e, int f0, int nf, uint32_t tokens, auto hrow) {
        float acc[NT][4] = {};
        const int step = tile_cols<W>(nf, D);
        const int64_t row = (int64_t)e * I + f0 + min(rw, nf - 1);
        for (int c0 = 0; c0 < D; c0 += step) {
            const int cols = min(step, D - c0);
            [[maybe_unused]] float wa[2], wb[2];  // FP8: block scales of this warp's slices
            [[maybe_unused]] const float *ga = nullptr, *gb = nullptr;
            if constexpr (W == MOE_FP8_E4M3_B128) {
                const int64_t at = ((int64_t)e * (I / 128) + (f0 + min(rw, nf - 1)) / 128) * (D / 128) + c0 / 128;
                ga = (const float*)p.s_gate + at;
                gb = (const float*)p.s_up + at;
                if (wg * kSlice < cols) {
                    wa[0] = __ldg(ga + wg);
                    wb[0] = __ldg(gb + wg);
                }
            }
            const uint8_t* tile = stage_wait();
            const uint8_t* xa[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xa[n] = act + min(8 * n + g, T - 1) * xstride;
#pragma unroll 1
            for (int c = wg * kSlice; c < cols; c += NC * kSlice) {
                const RowPair r = rows_at(tile, nf, nf, cols, c);
                if constexpr (W == MOE_F32) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        dot_f32(r, act + min(8 * n + 2 * q, T - 1) * xstride + (c0 + c) * 4,
                                act + min(8 * n + 2 * q + 1, T - 1) * xstride + (c0 + c) * 4, acc[n]);
                } else {
                    const uint8_t* xc[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) xc[n] = xa[n] + (c0 + c) * Tr<W>::xb;
                    if constexpr (W == MOE_BF16 || W == W_HILO) {
                        dot16<NT, false>(r, xc, acc);
                    } else if constexpr (W == MOE_FP8_E4M3_B128) {
                        float sx[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int s = 0; s < 2; ++s) sx[n][s] = xsc[min(8 * n + 2 * q + s, T - 1) * nxs + (c0 + c) / 128];
                        const bool first = c == wg * kSlice;
                        dot_fp8<NT>(r, xc, first ? wa[0] : __ldg(ga + c / 128), first ? wb[0] : __ldg(gb + c / 128), sx, acc);
                    } else {
                        float4 sx[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int s = 0; s < 2; ++s)
                                sx[n][s] = *(const float4*)(xsc + min(8 * n + 2 * q + s, T - 1) * nxs + (c0 + c) / 32);
                        uint32_t ka, kb;
                        const int64_t at = row * (D / 32) + c0 / 32;
                        scales_at(tile, nf, nf, cols, c, (const uint8_t*)p.s_gate + at, (const uint8_t*)p.s_up + at, ka, kb);
                        dot_mx<NT>(r, xc, ka, kb, sx, acc);
                    }
                }
            }
            stage_done();
        }
        if (reduce(acc, turns++)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int t = 8 * n + 2 * q + s;
                    if (rw < nf && t < T && ((tokens >> t) & 1u)) {
                        const float h = swiglu(acc[n][s], acc[n][2 + s]);
                        const int64_t at = (int64_t)hrow(t) * I + f0 + rw;
                        if constexpr (W == MOE_BF16) {
                            if (!(fabsf(h) <= 65504.0f)) overflow = true;
                            ((f16*)p.h)[at] = __float2half_rn(h);
                        } else {
                            p.h[at] = h;
                        }
                    }
                }
        }
    };
    // -------------------------------------------------------------- P1
    for (int f = f_lo; f < f_hi;) {
        const Pair t(f, f_hi, 8);
        if (t.n(grp)) gateup(E, t.at(grp), t.n(grp), 0xFFFFu, [&](int tok) { return T * k + tok; });
        f = t.end();
    }

    // ---------------------------------------------- barrier 1, top-k, list
    if (tid == 0 && !grid_wait(p.bar, target, lim, abort)) {
        if (!*abort) record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 43, cta, 0);
        *abort = 1;
    }
    consumers_sync();
    uint32_t bad = 0;
    for (int t = warp; t < T; t += NC * NG) {
        if (E <= 128) topk_token<4>(p, t, m, bad);
        else if (E <= 512) topk_token<16>(p, t, m, bad);
        else topk_token<32>(p, t, m, bad);
        __syncwarp();
        if (lane < k) {
            const int i = t * k + lane, e = m.sel[i];
            atomicOr(&m.mask[e >> 1], 1u << (t + 16 * (e & 1)));
            if (cta == 0) {
                p.blob[i] = e;
                p.blob[p.plane + i] = __float_as_int(m.selw[i]);
            }
        }
    }
    if (bad && cta == 0 && lane == 0) record_error(p.err, MOE_ERR_NONFINITE, (uint32_t)(p.tok0 + __ffs(bad) - 1), 0, 0);
    consumers_sync();
    {
        // ascending list of the touched experts: two experts (a word) a thread
        const uint32_t both = m.mask[tid];
        const uint32_t mine[2] = {both & 0xFFFFu, both >> 16};
        const uint32_t sum = (mine[0] ? 1u : 0u) + (mine[1] ? 1u : 0u) + ((uint32_t)__popc(both) << 16);  // experts | rows << 16
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) m.scan[warp] = inc;
        consumers_sync();
        uint32_t at = inc - sum;
#pragma unroll
        for (int w = 0; w < NC * NG; ++w) at += w < warp ? m.scan[w] : 0u;
        uint32_t place[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            place[j] = at & 0xFFFFu;
            if (mine[j]) {
                m.expert[place[j]] = (uint16_t)(2 * tid + j);
                m.tokens[place[j]] = (uint16_t)mine[j];
                m.hrow[place[j]] = (uint16_t)(at >> 16);
                at += 1u + ((uint32_t)__popc(mine[j]) << 16);
            }
        }
        m.mask[tid] = place[0] | place[1] << 16;
        if (tid == kCons - 1) {
            m.n = at & 0xFFFFu;
            m.hrow[at & 0xFFFFu] = (uint16_t)(at >> 16);
        }
    }
    consumers_sync();
    if (tid == 0) tc::mbar_arrive(smem_u32(&m.list_ready));
    for (int i = tid; i < T * k; i += kCons) {
        const int pos = ((const uint16_t*)m.mask)[m.sel[i]], t = i / k;
        m.wt[m.hrow[pos] + __popc(m.tokens[pos] & ((1u << t) - 1u))] = m.selw[i];  // read after the next barrier
    }
    const int n = m.n;

    // -------------------------------------------------------------- P2
    {
        const int64_t lo = (int64_t)n * I * cta / grid, hi = (int64_t)n * I * (cta + 1) / grid;
        for (int64_t f = lo; f < hi;) {
            const int pos = (int)(f / I);
            const int64_t first = (int64_t)pos * I;
            const Pair t((int)(f - first), (int)min((int64_t)I, hi - first), 8);
            const uint32_t tokens = m.tokens[pos];
            const int row = m.hrow[pos];
            if (t.n(grp)) gateup(m.expert[pos], t.at(grp), t.n(grp), tokens, [&](int tok) { return row + __popc(tokens & ((1u << tok) - 1u)); });
            f = first + t.end();
        }
    }
    if (overflow) record_error(p.err, MOE_ERR_NONFINITE, 5, cta, 0);
    consumers_sync();
    if (tid == 0) {
        target = grid_arrive(p.bar);
        if (!grid_wait(p.bar, target, lim, abort)) {
            if (!*abort) record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 44, cta, 0);
            *abort = 1;
        }
    }
    consumers_sync();

    // -------------------------------------------------------------- P3
    const int hstride = h_stride<W>(I), nhs = h_scales<W>(I) / 4;
    float* hsc = (float*)(act + up(p.hcap * hstride, 128));
    const int lo_at = min(I, P::kc) * 2;  // W_HILO: a row is its high halves, then its low halves
    for (int d0 = d_lo; d0 < d_hi; d0 += 16 * NG) {
        const Pair rows(d0, min(d_hi, d0 + 16 * NG), 16);
        const int r0 = rows.at(grp), nr = rows.n(grp);
        float out[NT][4] = {};
        for (int bx = -1; bx < n;) {
            const Batch bt = next_batch(m, bx, n, T, p.hcap);
            for (int c0 = 0; c0 < I; c0 += P::kc) {
                const int cols = min(P::kc, I - c0);
                consumers_sync();  // the buffer's last batch has been read
                {
                    // this batch's rows of h, 16 columns (8 in fp32) a unit
                    constexpr int kUnit = W == MOE_F32 ? 8 : 16;
                    const int per = cols / kUnit, total = bt.rows * per;
                    for (int u0 = tid & ~31; u0 < total; u0 += kCons) {
                        const int u = min(u0 + lane, total - 1), r = u / per, c = u - r * per;
                        const int64_t row = r < bt.shared ? T * k + r : bt.row0 + r - bt.shared;
                        uint8_t* dst = act + r * hstride;
                        if constexpr (W == MOE_BF16) {
                            const uint4* src = (const uint4*)((const f16*)p.h + row * I + c0 + c * 16);
                            const uint4 a = __ldcg(src), b = __ldcg(src + 1);
                            ((uint4*)(dst + c * 32))[0] = a;
                            ((uint4*)(dst + c * 32))[1] = b;
                        } else if constexpr (W == MOE_F32) {
                            const float4* src = (const float4*)(p.h + row * I + c0 + c * 8);
                            const float4 a = __ldcg(src), b = __ldcg(src + 1);
                            ((float4*)(dst + c * 32))[0] = a;
                            ((float4*)(dst + c * 32))[1] = b;
                        } else {
                            const float4* src = (const float4*)(p.h + row * I + c0 + c * 16);
                            float v[16];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 a = __ldcg(src + i);
                                v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
                            }
                            if constexpr (W == MOE_FP8_E4M3_B128) {
                                const float s = quant16_fp8(v, dst + c * 16, u0 + lane < total);
                                if ((c & 7) == 0 && u0 + lane < total) hsc[r * nhs + c / 8] = s;
                            } else if constexpr (W == MOE_MXFP4) {
                                const float s = quant16_mx(v, dst + c / 4 * 64, c & 1, (c >> 1) & 1, u0 + lane < total);
                                if ((c & 1) == 0 && u0 + lane < total) hsc[r * nhs + c / 2] = s;
                            } else {
                                uint32_t hi[8], lo[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    hi[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                                    const float2 b = __bfloat1622float2(*(const __nv_bfloat162*)&hi[i]);
                                    lo[i] = pack_bf16(v[2 * i] - b.x, v[2 * i + 1] - b.y);
                                }
                                for (int i = 0; i < 2; ++i) {
                                    ((uint4*)(dst + c * 32))[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                                    ((uint4*)(dst + lo_at + c * 32))[i] = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                                }
                            }
                        }
                    }
                }
                consumers_sync();
                for (int x = bt.x0; x < bt.x1; ++x) {
                    const uint32_t tokens = x < 0 ? 0xFFFFu : m.tokens[x];
                    const int grow = x < 0 ? 0 : m.hrow[x];                       // row of wt
                    const int brow = x < 0 ? 0 : bt.shared + grow - bt.row0;      // row of the buffer
                    if (!nr) continue;
                    const int na = min(nr, 8), nb = max(nr - 8, 0);
                    const int64_t erow = (int64_t)(x < 0 ? E : m.expert[x]) * D + r0;
                    int rank[NT][2];  // of the lane's accumulator tokens among the expert's; -1: not its token
                    const uint8_t* ha[NT];
#pragma unroll
                    for (int u = 0; u < NT; ++u) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int t = 8 * u + 2 * q + s;
                            rank[u][s] = t < T && ((tokens >> t) & 1u) ? __popc(tokens & ((1u << t) - 1u)) : -1;
                        }
                        const int t = 8 * u + g;
                        const int r = t < T && ((tokens >> t) & 1u) ? __popc(tokens & ((1u << t) - 1u)) : 0;
                        ha[u] = act + (brow + r) * hstride;
                    }
                    [[maybe_unused]] float fa = 0.0f, fb = 0.0f;
                    if constexpr (W == MOE_FP8_E4M3_B128) {
                        if (wg * kSlice < cols) {
                            const float* sd = (const float*)p.s_down + c0 / 128 + wg;
                            const int64_t blk = (int64_t)(x < 0 ? E : m.expert[x]) * (D / 128);
                            fa = __ldg(sd + (blk + (r0 + min(rw, na - 1)) / 128) * (I / 128));
                            fb = __ldg(sd + (blk + (r0 + min(rw + 8, nr - 1)) / 128) * (I / 128));
                        }
                    }
                    const uint8_t* tile = stage_wait();
                    float y[NT][4] = {};
#pragma unroll 1
                    for (int c = wg * kSlice; c < cols; c += NC * kSlice) {
                        const RowPair rp = rows_at(tile, na, nb, cols, c);
                        if constexpr (W == MOE_F32) {
#pragma unroll
                            for (int u = 0; u < NT; ++u)
                                dot_f32(rp, act + (brow + max(rank[u][0], 0)) * hstride + c * 4,
                                        act + (brow + max(rank[u][1], 0)) * hstride + c * 4, y[u]);
                        } else {
                            const uint8_t* hc[NT];
#pragma unroll
                            for (int u = 0; u < NT; ++u) hc[u] = ha[u] + c * (W == W_HILO ? 2 : Tr<W>::hb);
                            if constexpr (W == MOE_BF16) {
                                dot16<NT, true>(rp, hc, y);
                            } else if constexpr (W == W_HILO) {
                                dot16<NT, false>(rp, hc, y);
#pragma unroll
                                for (int u = 0; u < NT; ++u) hc[u] += lo_at;
                                dot16<NT, false>(rp, hc, y);
                            } else if constexpr (W == MOE_FP8_E4M3_B128) {
                                float sx[NT][2];
#pragma unroll
                                for (int u = 0; u < NT; ++u)
#pragma unroll
                                    for (int s = 0; s < 2; ++s) sx[u][s] = hsc[(brow + max(rank[u][s], 0)) * nhs + wg];
                                dot_fp8<NT>(rp, hc, fa, fb, sx, y);
                            } else {
                                float4 sx[NT][2];
#pragma unroll
                                for (int u = 0; u < NT; ++u)
#pragma unroll
                                    for (int s = 0; s < 2; ++s)
                                        sx[u][s] = *(const float4*)(hsc + (brow + max(rank[u][s], 0)) * nhs + c / 32);
                                uint32_t ka, kb;
                                const uint8_t* sd = (const uint8_t*)p.s_down + c0 / 32;
                                scales_at(tile, na, nb, cols, c, sd + (erow + min(rw, na - 1)) * (I / 32), sd + (erow + min(rw + 8, nr - 1)) * (I / 32), ka, kb);
                                dot_mx<NT>(rp, hc, ka, kb, sx, y);
                            }
                        }
                    }
                    stage_done();
#pragma unroll
                    for (int u = 0; u < NT; ++u)
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            if (rank[u][s] >= 0) {
                                const float wt = x < 0 ? 1.0f : m.wt[grow + rank[u][s]];
                                out[u][s] = fmaf(wt, y[u][s], out[u][s]);
                                out[u][2 + s] = fmaf(wt, y[u][2 + s], out[u][2 + s]);
                            }
                }
            }
            bx = bt.x1;
        }
        if (nr && reduce(out, turns++)) {
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int t = 8 * u + 2 * q + s, d = rw + 8 * r;
                        if (t < T && d < nr) {
                            const int64_t at = (int64_t)t * D + r0 + d;
                            if (p.out_elem == kF32) ((float*)p.out)[at] = out[u][2 * r + s];
                            else ((bf16*)p.out)[at] = __float2bfloat16_rn(out[u][2 * r + s]);
                        }
                    }
        }
    }
}

constexpr int kSmemLimit = 232448;

// Shared memory for T tokens: rows of h's buffer, where the ring starts, and
// its stages.
template <int W> bool plan_smem(int T, int D, int I, int k, int* hcap, int* ring_at, int* stages) {
    const int64_t misc = up((int)sizeof(Misc), 128);
    const int64_t x = (int64_t)up(T * x_stride<W>(D), 128) + up(T * x_scales<W>(D), 128);
    const int64_t hrow = h_stride<W>(I) + h_scales<W>(I);
    // h's buffer takes x's place; at least the rows of one expert, at most
    // all of them, and beyond x only what leaves two rings of four stages
    const int64_t all = (int64_t)T * (k + 1);
    const int64_t room = std::max(x, std::min(all * hrow + 256, (int64_t)kSmemLimit - misc - 4 * NG * Plan<W>::stage));
    const int64_t cap = std::max<int64_t>(T, std::min(all, (room - 256) / hrow));
    const int64_t at = misc + std::max(x, cap * hrow + 256);
    if (at > kSmemLimit) return false;
    *hcap = (int)cap;
    *ring_at = up((int)at, 1024);
    *stages = std::min(kMaxStages, (kSmemLimit - *ring_at) / Plan<W>::stage) / NG;  // of each ring
    return *stages >= 2;
}

// A matrix of `rows` rows of `bytes` as boxes of 8 rows and kBoxRow bytes,
// laid out [line of `in` bytes][row][in], swizzled over a line.
template <int W> bool weight_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes) {
    constexpr int in = Tr<W>::in;
    const cuuint64_t dims[3] = {in, (cuuint64_t)rows, (cuuint64_t)(bytes / in)};
    const cuuint64_t strides[2] = {(cuuint64_t)bytes, in};
    const cuuint32_t box[3] = {in, 8, kBoxRow / in}, es[3] = {1, 1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           in == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Scale bytes [rows, bytes], boxes of 8 rows and a stage's columns.
bool scale_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes) {
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {Plan<MOE_MXFP4>::kc / 32, 8}, es[2] = {1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int W, int NT> cudaError_t launch(FewParams p, const Maps& maps, int num_sms, cudaStream_t s) {
    if (!plan_smem<W>(p.T, p.D, p.I, p.k, &p.hcap, &p.ring_at, &p.stages)) return cudaErrorInvalidConfiguration;
    const int bytes = p.ring_at + NG * p.stages * Plan<W>::stage;
    cudaError_t e = ensure_smem_attr((const void*)few_kernel<W, NT>, kSmemLimit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait on one another: all resident or no launch
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, few_kernel<W, NT>, p, maps);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int W> cudaError_t launch_chunks(const FewParams& p, int num_sms, cudaStream_t s) {
    // As many tokens at a time as their x leaves room for two rings of
    // two stages (16 at D = 4096; wider rows take a few launches).
    int per = std::min(p.T, kFewMax), hcap, ring_at, stages;
    while (per > 1 && !plan_smem<W>(per, p.D, p.I, p.k, &hcap, &ring_at, &stages)) --per;
    Maps maps = {};
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    const int64_t gr = (int64_t)(p.E + 1) * p.I, dr = (int64_t)(p.E + 1) * p.D;
    bool ok = weight_map<W>(&maps.w[0], p.w_gate, gr, bytes_of<W>(p.D)) && weight_map<W>(&maps.w[1], p.w_up, gr, bytes_of<W>(p.D)) &&
              weight_map<W>(&maps.w[2], p.w_down, dr, bytes_of<W>(p.I));
    // scales by TMA where their rows are whole 16-byte pieces
    const bool tma_scales = W == MOE_MXFP4 && p.D % 512 == 0 && p.I % 512 == 0;
    if (tma_scales)
        ok = ok && scale_map(&maps.s[0], p.s_gate, gr, p.D / 32) && scale_map(&maps.s[1], p.s_up, gr, p.D / 32) &&
             scale_map(&maps.s[2], p.s_down, dr, p.I / 32);
    if (!ok) return cudaErrorInvalidValue;
    for (int t0 = 0; t0 < p.T; t0 += per) {
        FewParams c = p;
        c.T = std::min(per, p.T - t0);
        c.tok0 = t0;
        c.tma_scales = tma_scales;
        c.plane = p.T * p.k;
        c.x = (const char*)p.x + (int64_t)t0 * p.D * (W == MOE_F32 ? 4 : 2);
        c.logits = p.logits + (int64_t)t0 * p.E;
        c.blob = p.blob + t0 * p.k;
        c.out = (char*)p.out + (int64_t)t0 * p.D * (p.out_elem == kF32 ? 4 : 2);
        const cudaError_t e = c.T <= 8 ? launch<W, 1>(c, maps, num_sms, s) : launch<W, 2>(c, maps, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace few

cudaError_t launch_few(const FewParams& p, int num_sms, cudaStream_t s) {
    switch (p.dtype) {
        case MOE_F32: return few::launch_chunks<MOE_F32>(p, num_sms, s);
        case MOE_BF16: return p.down_f16 ? few::launch_chunks<MOE_BF16>(p, num_sms, s) : few::launch_chunks<few::W_HILO>(p, num_sms, s);
        case MOE_FP8_E4M3_B128: return few::launch_chunks<MOE_FP8_E4M3_B128>(p, num_sms, s);
        default: return few::launch_chunks<MOE_MXFP4>(p, num_sms, s);
    }
}

}  // namespace moe

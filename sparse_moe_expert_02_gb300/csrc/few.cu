// The whole layer for a few tokens (moe_forward_few): one persistent
// cooperative kernel, a CTA per SM.
//
// At these sizes the layer is its weights: each touched expert's three
// matrices pass through the SMs once (T = 1, D = 4096, I = 1024, top_k = 10:
// 277 MB in bf16, 73 MB in 4 bits) and everything else is latency.  So the
// kernel is a weight stream.  Four producer warps fill a ring of 8 KB (16-bit
// weights: 16 KB) stages by TMA, as far ahead as shared memory allows and
// across the phases below; twelve consumer warps each take tiles of 16 weight
// rows through all of their columns, a stage at a time, with mma.sync: the
// rows are the M side, the tokens the N side (16 x 8), so a tile costs the
// same for one token as for eight, its sums stay in one warp's registers, and
// the pointers, waits and routing of a tile are paid once.  (Two groups of
// eight warps that split a tile's columns and add up through shared memory
// took 57.2 us where this takes 37.2, 4 bits, T = 1: the 4-bit layer is bound
// by instructions.)  tcgen05 would want 128 rows and its operands in its own
// layout; at HBM speed mma.sync is far from its limit.
//
// Measured (D = 4096, I = 1024, top_k = 10, weights from HBM): T = 1 bf16 58.3
// us, 4.8 TB/s of weights over the whole call, 6 in P2 and 5.2 in P3; 4 bits
// 34.9 us; T = 8 FP8 112 us, 5.1 TB/s.  From some ten tokens on moe_forward is
// the faster (MoELayer.few_pays).  What is left is 9 to 12 us until the
// list of experts stands (launch, router, barrier, top-k: a chain of
// latencies), 3 us from the last gate/up tile to the first down product, and
// code that is read from memory on its first use: the kernel runs each line
// about once, and halving its size (one copy of the fill and of the gate/up
// loop, loops left rolled) took 48.0 us to 38.4 (4 bits) and 29.4 to 24.6
// (fp32, T = 5).  So most loops here are kept rolled on purpose.
//
//   P0  router logits: the CTA's share of the E rows; arrive at barrier 1
//   --  wait for barrier 1; every CTA takes the top-k of all T tokens and
//       builds the same list of distinct experts
//   P1  shared expert's gate/up: its share of I features, whose weights need
//       no list and are in the ring by then
//   P2  routed gate/up: its share of the (expert, feature) pairs.  Tiles of 8
//       gate rows and the 8 up rows of the same features, so that a thread's
//       accumulators hold both and SwiGLU is local; h to global
//   --  barrier 2 (the ring is already filling with P3's weights)
//   P3  down: the CTA's share of the D output rows, over all experts, h
//       brought into shared memory (and quantised) a batch of experts at a
//       time: a warp takes the same rows of every sixth or twelfth expert and
//       keeps their weighted sum in registers; the warps' sums are added once,
//       in warp order, so there are no atomics and the result does not vary
//
// Gate and up are split by tiles (flattened over the experts), down to the
// row.  Eight rows come as one box; rows left over come as row copies.  (Gate
// and up split to the feature even out the bytes, 67 features a CTA instead of
// 64 or 72, but then the one tile of row copies is last to finish: 4 bits 37.5
// us instead of 34.4.)  A dot product does not mind the order of its terms, so
// each lane takes 16 contiguous bytes (4-bit: 4 or 16) of its row and the same
// columns of its token as fragments; no shuffles, no ldmatrix.
//
// Arithmetic, as moe_forward's: products of weights and activations as the
// type holds them (x and h quantised for FP8 and MXFP4; h as fp16 against
// W_down's fp16 copy, or as a bf16 pair, for bf16), fp32 accumulation, block
// scales applied in fp32 to each block's partial sum.  E4M3 and E2M1 codes
// become fp16 MMA operands by one conversion per two of them, exactly, and
// the quantised activations are held as fp16.  (mma.sync with E4M3 operands,
// the 4-bit codes made E4M3 by shifts and masks, took 58.5 us instead of 44.3
// at 4 bits, T = 1, on otherwise the same kernel.)
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

constexpr int NW = 12;                       // consumer warps
constexpr int NP = 4;                        // producer warps, every fourth tile each
constexpr int kCons = 32 * NW;               // consumer threads
constexpr int kThreads = kCons + 32 * NP;
constexpr int kMaxPairs = kFewMax * 32;      // (token, slot) pairs
constexpr int kMaxStages = 20;
constexpr int kHCols = 1024;                 // columns of h in shared memory at a time
constexpr int W_HILO = 4;                    // MOE_BF16 with h as a bf16 pair against a bf16 W_down

// Per weight type: bytes of 64 columns; columns a warp takes at a time (its
// slice, `in` bytes: one swizzled line of a box); bytes of an activation x
// and h; activation scales per 128 columns.
template <int W> struct Tr;
template <> struct Tr<MOE_F32> { static constexpr int b64 = 256, slice = 32, in = 128, xpad = 16, xb = 4, hb = 4, nsc = 0; };
template <> struct Tr<MOE_BF16> { static constexpr int b64 = 128, slice = 64, in = 128, xpad = 64, xb = 2, hb = 2, nsc = 0; };
template <> struct Tr<W_HILO> { static constexpr int b64 = 128, slice = 64, in = 128, xpad = 64, xb = 2, hb = 4, nsc = 0; };
template <> struct Tr<MOE_FP8_E4M3_B128> { static constexpr int b64 = 64, slice = 128, in = 128, xpad = 16, xb = 2, hb = 2, nsc = 1; };
template <> struct Tr<MOE_MXFP4> { static constexpr int b64 = 32, slice = 128, in = 64, xpad = 64, xb = 2, hb = 2, nsc = 4; };

__host__ __device__ constexpr int up(int v, int a) { return (v + a - 1) / a * a; }
__host__ __device__ constexpr int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ constexpr int imax(int a, int b) { return a > b ? a : b; }

// Bytes of n columns (n a multiple of 64).
template <int W> __host__ __device__ constexpr int bytes_of(int n) { return n / 64 * Tr<W>::b64; }

// Bytes of a box's rows, two boxes of eight rows a stage.  16-bit weights like
// longer rows (one token 56.9 us against 59.3, five with D = 7168 239 against
// 264) while the ring keeps eight stages or so (16 tokens: 498 against 443);
// the other types need the stages (4 bits 39.8 against 37.2, FP8 123 against
// 115).
template <int W, int NT> struct Plan {
    static constexpr int box = NT == 1 && (W == MOE_BF16 || W == W_HILO) ? 1024 : 512;
    static constexpr int kc = box / Tr<W>::b64 * 64;         // columns of a box
    static constexpr int data = 16 * (box + 16);             // row copies: 16 bytes between rows
    static constexpr int scales = W == MOE_MXFP4 ? 16 * kc / kMxBlock : 0;  // scale bytes of a stage
    static constexpr int stage = up(data + scales, 1024);        // boxes are swizzled by address
    static constexpr int rslice = W == MOE_F32 ? 32 : 64;        // columns of router rows taken at a time
    static constexpr int eb = W == MOE_F32 ? 4 : 2;              // bytes of a router weight
};
// Shared-memory row strides of x and of h (one chunk of columns), and the
// bytes of a row's scales.
template <int W> __host__ __device__ constexpr int x_stride(int D) { return up(D * Tr<W>::xb, 128) + Tr<W>::xpad; }
template <int W> __host__ __device__ constexpr int h_stride(int I) { return up(imin(I, kHCols) * Tr<W>::hb, 128) + Tr<W>::xpad; }
template <int W> __host__ __device__ constexpr int x_scales(int D) { return D / 128 * Tr<W>::nsc * 4; }
template <int W> __host__ __device__ constexpr int h_scales(int I) { return imin(I, kHCols) / 128 * Tr<W>::nsc * 4; }

// Fixed shared memory: barriers and flags, the expert list, reductions.
struct Misc {
    uint64_t full[kMaxStages], empty[kMaxStages], list_ready, producers;
    int abort, n;               // n: distinct experts
    uint32_t scan[16];
    uint32_t mask[512];         // token bits of each expert (two a word), then its place in the list
    uint16_t expert[kMaxPairs]; // the list: expert, token bits, first row of h
    uint16_t tokens[kMaxPairs];
    uint16_t hrow[kMaxPairs + 1];
    uint16_t sel[kMaxPairs];    // [T, k] chosen experts
    float selw[kMaxPairs];
    float wt[kMaxPairs];        // routing weight of each row of h
    uint4 zeros[4];
    float4 red[NW * 2 * 32];    // [warp][token tile][lane]
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
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kCons) : "memory"); }
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
// Two codes of an operand as fp16 (exact).
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// The eight codes of a word.
__device__ __forceinline__ void e2m1_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
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
    int line_a, line_b;  // bytes from a slice to the next
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
        const uint32_t aw[8] = {e4m3_f16(a.x), e4m3_f16(a.x >> 16), e4m3_f16(a.y), e4m3_f16(a.y >> 16),
                                e4m3_f16(a.z), e4m3_f16(a.z >> 16), e4m3_f16(a.w), e4m3_f16(a.w >> 16)};
        const uint32_t dw[8] = {e4m3_f16(d.x), e4m3_f16(d.x >> 16), e4m3_f16(d.y), e4m3_f16(d.y >> 16),
                                e4m3_f16(d.z), e4m3_f16(d.z >> 16), e4m3_f16(d.w), e4m3_f16(d.w >> 16)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 b = *(const uint4*)(xa[n] + 2 * o), e = *(const uint4*)(xa[n] + 2 * o + 16);
            mma_f16(c[n], aw[0], dw[0], aw[1], dw[1], b.x, b.y);
            mma_f16(c[n], aw[2], dw[2], aw[3], dw[3], b.z, b.w);
            mma_f16(c[n], aw[4], dw[4], aw[5], dw[5], e.x, e.y);
            mma_f16(c[n], aw[6], dw[6], aw[7], dw[7], e.z, e.w);
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
// tokens.
template <int NT>
__device__ __forceinline__ void dot_mx(const RowPair& r, const uint8_t* const (&xa)[NT], uint32_t ka, uint32_t kb,
                                       const float4 (&sx)[NT][2], float (&acc)[NT][4]) {
    const int q = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sa[2], sb[2];
        e8m0_floats((uint16_t)(ka >> (i & 2) * 8), sa[0], sa[1]);
        e8m0_floats((uint16_t)(kb >> (i & 2) * 8), sb[0], sb[1]);
        uint32_t a[4], d[4];
        e2m1_f16(*(const uint32_t*)(r.a + (16 * i ^ r.xa) + q * 4), a);
        e2m1_f16(*(const uint32_t*)(r.b + (16 * i ^ r.xb) + q * 4), d);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 b = *(const uint4*)(xa[n] + 64 * i + q * 16);
            float c[4] = {};
            mma_f16(c, a[0], d[0], a[1], d[1], b.x, b.y);
            mma_f16(c, a[2], d[2], a[3], d[3], b.z, b.w);
            const float s0 = ((const float*)&sx[n][0])[i], s1 = ((const float*)&sx[n][1])[i];
            acc[n][0] = fmaf(c[0], sa[i & 1] * s0, acc[n][0]);
            acc[n][1] = fmaf(c[1], sa[i & 1] * s1, acc[n][1]);
            acc[n][2] = fmaf(c[2], sb[i & 1] * s0, acc[n][2]);
            acc[n][3] = fmaf(c[3], sb[i & 1] * s1, acc[n][3]);
        }
    }
}
// One token against E2M1 rows, `slices` times 128 columns.  The eight token
// columns of an MMA are eight 32-column blocks of the one token: lane q takes
// the 16 bytes of a row that are block q (q + 4 in the second half of 256
// columns) and only column q (q + 4) of the activations is not zero at its
// places, so sixteen MMAs add up to the eight blocks' sums apart, and scales
// are multiplied once per 256 columns instead of once per block.  x: the
// lane's token; ka, kb: scale bytes of rows g and g + 8, sx: of the token;
// acc[0], acc[2]: this lane's share of rows g and g + 8.
__device__ __forceinline__ void dot_one(RowPair r, const uint8_t* x, int slices, const uint8_t* ka, const uint8_t* kb, const float* sx,
                                        const uint8_t* zeros, float (&acc)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint8_t *x0 = g == q ? x + q * 64 : zeros, *x1 = g == q + 4 ? x + 256 + q * 64 : zeros;
    const int step0 = g == q ? 512 : 0, step1 = g == q + 4 ? 512 : 0;
    const int oa = 16 * q ^ r.xa, ob = 16 * q ^ r.xb;
    auto half = [&](const uint4& a, const uint4& d, const uint8_t* xb, float (&c)[4]) {
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint4 b = ((const uint4*)xb)[w];
            uint32_t af[4], df[4];
            e2m1_f16(aw[w], af);
            e2m1_f16(dw[w], df);
            mma_f16(c, af[0], df[0], af[1], df[1], b.x, b.y);
            mma_f16(c, af[2], df[2], af[3], df[3], b.z, b.w);
        }
    };
#pragma unroll 2
    for (int s = 0; s < slices; s += 2) {
        float c[4] = {};
        const bool both = s + 1 < slices;
        // this lane's blocks: 2 q and 2 q + 1 of the eight
        const bool on = both || q < 2;
        const uint16_t wa = on ? *(const uint16_t*)(ka + 4 * s + 2 * q) : (uint16_t)0, wb = on ? *(const uint16_t*)(kb + 4 * s + 2 * q) : (uint16_t)0;
        const float2 t = on ? *(const float2*)(sx + 4 * s + 2 * q) : make_float2(0, 0);
        half(*(const uint4*)(r.a + oa), *(const uint4*)(r.b + ob), x0, c);
        if (both) half(*(const uint4*)(r.a + r.line_a + oa), *(const uint4*)(r.b + r.line_b + ob), x1, c);
        float a0, a1, b0, b1;
        e8m0_floats(wa, a0, a1);
        e8m0_floats(wb, b0, b1);
        acc[0] = fmaf(c[0], a0 * t.x, fmaf(c[1], a1 * t.y, acc[0]));
        acc[2] = fmaf(c[2], b0 * t.x, fmaf(c[3], b1 * t.y, acc[2]));
        r.a += 2 * r.line_a;
        r.b += 2 * r.line_b;
        x0 += step0;
        x1 += step1;
    }
}
// fp32 rows, 32 columns, on the CUDA cores: the same accumulators; t0 and t1
// point at the 32 columns of the lane's two tokens.  The 32 are summed by
// themselves first: one chain over a whole row had two to three times the
// rounding error (D = 512: 5e-7 of the output's rms).
__device__ __forceinline__ void dot_f32(const RowPair& r, const uint8_t* t0, const uint8_t* t1, float (&acc)[4]) {
    float c[4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float4 a = *(const float4*)(r.a + (16 * k ^ r.xa)), d = *(const float4*)(r.b + (16 * k ^ r.xb)),
                     x = ((const float4*)t0)[k], y = ((const float4*)t1)[k];
        c[0] = fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, c[0]))));
        c[1] = fmaf(a.x, y.x, fmaf(a.y, y.y, fmaf(a.z, y.z, fmaf(a.w, y.w, c[1]))));
        c[2] = fmaf(d.x, x.x, fmaf(d.y, x.y, fmaf(d.z, x.z, fmaf(d.w, x.w, c[2]))));
        c[3] = fmaf(d.x, y.x, fmaf(d.y, y.y, fmaf(d.z, y.z, fmaf(d.w, y.w, c[3]))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += c[i];
}

// 16 values (of a block that some neighbouring lanes share) to fp16 operands
// at dst (if `on`); returns the block's scale.
__device__ __forceinline__ float quant16_fp8(const float (&v)[16], uint8_t* dst, bool on) {  // 8 lanes: 128 columns
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
    const float f = a > 0.0f ? 448.0f / a : 1.0f;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = e4m3_f16(f32x2_to_e4m3x2(v[2 * i] * f, v[2 * i + 1] * f));
    if (on) {
        ((uint4*)dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        ((uint4*)dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return a > 0.0f ? a / 448.0f : 1.0f;
}
__device__ __forceinline__ float quant16_mx(const float (&v)[16], uint8_t* dst, bool on) {  // 2 lanes: 32 columns
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t s = mx_scale_byte(m);
    const float f = s == 255u ? 0.0f : mx_inv_scale(s);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n"
            : "=r"(w[i])
            : "f"(v[2 * i] * f), "f"(v[2 * i + 1] * f));
        if (s == 255u) w[i] = 0;
    }
    if (on) {
        ((uint4*)dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        ((uint4*)dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return mx_scale(s);
}

// Top-k of one token's logits by one warp, with room for its E keys in shared
// memory: largest first, the lower index on a tie; non-finite logits count as
// -inf (and are reported).  Each lane keeps the two best of its own (every
// 32nd) in order and looks for the next two when they are used up.
__device__ __forceinline__ void topk_token(const FewParams& p, int t, Misc& m, uint32_t* key, uint32_t& bad) {
    const int lane = threadIdx.x & 31;
    bool finite = true;
#pragma unroll 8
    for (int e = lane; e < p.E; e += 32) {
        uint32_t u = __float_as_uint(__ldcg(p.logits + (int64_t)t * p.E + e));
        if ((u & 0x7F800000u) == 0x7F800000u) {
            finite = false;
            u = 0xFF800000u;
        }
        if (u == 0x80000000u) u = 0u;  // -0 and +0 tie
        key[e] = (u >> 31) ? ~u : (u | 0x80000000u);  // order-preserving, never 0
    }
    if (!__all_sync(0xffffffffu, finite)) bad |= 1u << t;
    uint32_t k0 = 0, k1 = 0, z = 0, lk = 0xFFFFFFFFu;  // lk, le: the last one used
    int e0 = 0, e1 = 0, used = 2, le = -1;
    for (int r = 0; r < p.k; ++r) {
        if (used == 2) {
            used = 0;
            k0 = k1 = 0;
#pragma unroll 4
            for (int e = lane; e < p.E; e += 32) {
                const uint32_t v = key[e];
                if (v < lk || (v == lk && e > le)) {  // equal keys keep their order
                    if (v > k0) {
                        k1 = k0, e1 = e0;
                        k0 = v, e0 = e;
                    } else if (v > k1) {
                        k1 = v, e1 = e;
                    }
                }
            }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, k0);
        const uint32_t e = __reduce_min_sync(0xffffffffu, k0 == top ? (uint32_t)e0 : 0xFFFFFFFFu);
        if (lane == r) {
            z = top;
            m.sel[t * p.k + r] = (uint16_t)e;
        }
        if (k0 == top && (uint32_t)e0 == e) {
            lk = k0, le = e0;
            k0 = k1, e0 = e1;
            k1 = 0;
            ++used;
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

// `total` units over the consumers, UNITS of a thread's at a time: all of
// their loads (of WORDS 16-byte words), then what is done with each.  Whole
// warps stay together; `on`: the unit is the lane's own.
template <int WORDS, int UNITS, class Load, class Store>
__device__ __forceinline__ void each_unit(int total, Load load, Store store) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int u0 = threadIdx.x & ~31; u0 < total; u0 += UNITS * kCons) {
        uint4 v[UNITS][WORDS];
#pragma unroll
        for (int j = 0; j < UNITS; ++j) load(min(u0 + j * kCons + lane, total - 1), v[j]);
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int u = u0 + j * kCons + lane;
            if (u0 + j * kCons < total) store(min(u, total - 1), u < total, v[j]);
        }
    }
}

// Grid barrier on a counter that only grows: every launch adds whole multiples
// of the grid, so what a CTA reads before it arrives tells the count to wait
// for, and nobody waits for an atomic's answer.
__device__ __forceinline__ void grid_arrive(unsigned long long* bar) {
    asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(bar), "l"(1ull) : "memory");
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

// A phase (P3: a batch of experts) is a round: `units` units of `steps` stages
// each, unit u on warp u % n.  A round has a window of the ring to itself, n
// times as many stages as fit from `base` on, and each warp its own of them
// (every nth), which it goes round; a stage is filled for one warp, by one
// producer, for the length of the round.  Consumers end a round together and
// producers start one together, so who waits for a stage's nth filling or
// emptying knows the one before to have happened, and a barrier's phase bit
// says no more than that.
struct Walk {
    int stages, base;
    uint32_t phases;  // bit s: parity of the next filling of stage s
    __device__ __forceinline__ void finish(int n, int units, int steps) {
        const int rows = stages / n, q = units / n, extra = units - q * n;  // warps < extra: q + 1 units
        const int sa = (q + 1) * steps, sb = q * steps;
        uint64_t flips = 0;
#pragma unroll 1
        for (int j = 0; j < rows; ++j) {  // stages j n .. of the window
            uint32_t m = 0;
            if ((sa / rows + (j < sa % rows)) & 1) m |= (1u << extra) - 1u;
            if ((sb / rows + (j < sb % rows)) & 1) m |= (1u << n) - (1u << extra);
            flips |= (uint64_t)m << (base + j * n);
        }
        phases ^= (uint32_t)(flips | flips >> stages) & ((1u << stages) - 1u);
        base += min(extra ? sa : sb, rows) * n;
        if (base >= stages) base -= stages;
    }
};
// A warp's place in a round (i: its number; a producer: 0, and it adds i).
struct Turn {
    int at, len, n, base, stages;
    uint32_t phases, parity;
    __device__ __forceinline__ Turn(const Walk& w, int warps, int i)
        : at(i), len(w.stages / warps * warps), n(warps), base(w.base), stages(w.stages), phases(w.phases), parity(0) {}
    __device__ __forceinline__ void next() {
        at += n;
        if (at >= len) {
            at -= len;
            parity ^= 1;
        }
    }
    __device__ __forceinline__ int stage(int i = 0) const { const int s = base + at + i; return s < stages ? s : s - stages; }
    __device__ __forceinline__ uint32_t phase(int s) const { return (phases >> s & 1u) ^ parity; }
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

// Columns of a stage of n router rows: a twelfth of them, if it holds that.
template <int W, int NT> __device__ __forceinline__ int router_cols(int n, int D) {
    return min(up((D + NW - 1) / NW, 64), (16 * Plan<W, NT>::box / n & -256) / Plan<W, NT>::eb);
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// This CTA's share of n things: [lo, hi).
__device__ __forceinline__ void share(int n, int cta, int grid, int& lo, int& hi) {
    const int per = n / grid, more = n - per * grid;
    lo = per * cta + min(cta, more);
    hi = lo + per + (cta < more);
}
// dot_one's shares, summed over the four lanes of a row pair.
__device__ __forceinline__ void sum_quad(float (&acc)[4]) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        acc[2] += __shfl_xor_sync(0xffffffffu, acc[2], o);
    }
}
// FP8: the weights' scales of a stage's blocks, fetched before the wait for it.
struct BlockScales {
    float s[4];
    __device__ __forceinline__ void fetch(const void* p, int cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = 128 * i < cols ? __ldg((const float*)p + i) : 0.0f;
    }
};
struct No { static constexpr bool value = false; };
struct Yes { static constexpr bool value = true; };

// ONE: a single token, against 4-bit weights.
template <int W, int NT, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ Maps maps) {
    using P = Plan<W, NT>;
    constexpr bool kScaled = W == MOE_FP8_E4M3_B128 || W == MOE_MXFP4;
    constexpr int kSlice = Tr<W>::slice, kIn = Tr<W>::in;
    extern __shared__ __align__(1024) uint8_t smem[];
    Misc& m = *(Misc*)smem;
    uint8_t* act = smem + up(sizeof(Misc), 128);  // x (P1, P2), then batches of h (P3)
    uint8_t* ring = smem + p.ring_at;
    const uint8_t* smem_zeros = (const uint8_t*)m.zeros;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int cta = blockIdx.x, grid = gridDim.x;
    const int D = p.D, I = p.I, E = p.E, T = p.T, k = p.k;
    const int most = min(NW, p.stages);  // tiles side by side: at most one stage of each in the ring
    const int64_t lim = p.spin_ns;
    volatile int* abort = &m.abort;
    if (threadIdx.x == kCons) {
#pragma unroll 1
        for (int s = 0; s < p.stages; ++s) {
            tc::mbar_init(smem_u32(m.full + s), 1);
            tc::mbar_init(smem_u32(m.empty + s), 1);
        }
        tc::mbar_init(smem_u32(&m.list_ready), 1);
        tc::mbar_init(smem_u32(&m.producers), NP);
        m.abort = 0;
        for (int i = 0; i < 4; ++i) m.zeros[i] = make_uint4(0, 0, 0, 0);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        // this call's error word; only waits that run out record an error
        // before barrier 1
        if (cta == 0 && p.tok0 == 0) p.err[0] = p.err[1] = p.err[2] = p.err[3] = 0;
    }
    __syncthreads();

    // shares of this CTA: router rows, tiles of the shared expert's features, output rows
    int e_lo, e_hi, f_lo, f_hi, d_lo, d_hi;
    share(E, cta, grid, e_lo, e_hi);
    share(I / 8, cta, grid, f_lo, f_hi);
    share(D, cta, grid, d_lo, d_hi);
    Walk at = {p.stages, 0, 0};

    if (warp >= NW) {
        // ------------------------------------------------------ producers
        const uint32_t ring0 = smem_u32(ring);
        const int me = warp - NW;
        bool ok = true;
        uint32_t rounds = 0;
        auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
            if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, lim, abort));
            if (!ok && elect_one() && !*abort) {
                record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 41, cta, 0);
                *abort = 1;
            }
            __syncwarp();
            return ok;
        };
        // Tile i's next stage (this producer's to fill), once it is free.
        auto stage_free = [&](const Turn& t, int i, int& st) -> bool {
            st = t.stage(i);
            return wait(smem_u32(m.empty + st), t.phase(st) ^ 1);
        };
        auto finish = [&](int n, int units, int steps) {
            at.finish(n, units, steps);
            if (ok && elect_one()) tc::mbar_arrive(smem_u32(&m.producers));
            __syncwarp();
            wait(smem_u32(&m.producers), rounds++ & 1);
        };
        // Warp i's next stage: rows from row0 of matrix wa and from row1 of wb (0 gate, 1 up, 2 down), na and
        // nb of them, columns c0 .. of K; whole boxes of eight, or row copies of `cols`.
        auto fill = [&](const Turn& t, int i, int wa, int64_t row0, int na, int wb, int64_t row1, int nb, int K, int c0, int cols) {
            int st;
            if (stage_free(t, i, st) && elect_one()) {
                const uint32_t bar = smem_u32(m.full + st), bytes = bytes_of<W>(cols), sbytes = cols / 32;
                const bool scaled = W == MOE_MXFP4 && p.tma_scales;
                const uint32_t per = bytes + (scaled ? sbytes : 0), box = 8 * P::box + (scaled ? 8 * P::kc / 32 : 0);
                tc::mbar_expect_tx(bar, (na == 8 ? box : na * per) + (nb == 8 ? box : nb * per));
                uint32_t dst = ring0 + st * P::stage, sdst = dst + P::data;
                const int line = bytes_of<W>(c0) / kIn;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int w = half ? wb : wa, n = half ? nb : na;
                    const int64_t row = half ? row1 : row0;
                    if (n == 8) {
                        box_load(dst, &maps.w[w], bar, (int)row, line);
                        if (scaled) tc::tma_load_2d(sdst, &maps.s[w], bar, c0 / 32, (int)row);
                        dst += 8 * P::box;
                        sdst += 8 * P::kc / 32;
                    } else {
                        const uint8_t* src = (const uint8_t*)(w == 0 ? p.w_gate : w == 1 ? p.w_up : p.w_down) + row * bytes_of<W>(K) + bytes_of<W>(c0);
                        const uint8_t* ss = (const uint8_t*)(w == 0 ? p.s_gate : w == 1 ? p.s_up : p.s_down) + row * (K / 32) + c0 / 32;
#pragma unroll 1
                        for (int r = 0; r < n; ++r) {
                            bulk_load(dst, src, bytes, bar);
                            if (scaled) bulk_load(sdst, ss, sbytes, bar);
                            dst += bytes + 16;
                            sdst += sbytes;
                            src += bytes_of<W>(K);
                            ss += K / 32;
                        }
                    }
                }
            }
            __syncwarp();
        };
        // P0: router rows (fp32 or bf16), row copies
        for (int e = e_lo; e < e_hi; e += 16) {
            const int n = min(16, e_hi - e), step = router_cols<W, NT>(n, D), chunks = ceil_div(D, step);
            Turn t(at, most, 0);
            for (int c = 0, i = 0; c < chunks; ++c) {
                int st;
                if (i % NP == me && stage_free(t, i, st) && elect_one()) {
                    const uint32_t bar = smem_u32(m.full + st), base = ring0 + st * P::stage;
                    const int c0 = c * step, bytes = min(step, D - c0) * P::eb;
                    tc::mbar_expect_tx(bar, (uint32_t)(n * bytes));
                    const uint8_t* src = (const uint8_t*)p.w_router + ((int64_t)e * D + c0) * P::eb;
#pragma unroll 1
                    for (int r = 0; r < n; ++r) bulk_load(base + r * (bytes + 16), src + (int64_t)r * D * P::eb, bytes, bar);
                }
                __syncwarp();
                if (++i == most) {
                    i = 0;
                    t.next();
                }
            }
            finish(most, chunks, 1);
        }
        // P1 (tiles of the shared expert, their stages spread over the warps), P2, then P3's batches
        int phase = 1, n = 0, f1 = f_lo, bx = -1, h0 = 0, d0 = d_lo, t_lo = 0, t_hi = 0;
        Batch bt = {};
#pragma unroll 1
        while (true) {
            int units, warps, steps, K = D, col0 = 0, width = D;  // columns [col0, col0 + width) of rows of K
            int tp = 1, nr = 0;
            if (phase == 1 && f1 >= f_hi) {
                // the routed experts, once the list is there
                n = wait(smem_u32(&m.list_ready), 0) ? uniform(m.n) : 0;
                share(n * (I / 8), cta, grid, t_lo, t_hi);
                phase = t_hi > t_lo ? 2 : 3;
            }
            if (phase == 1) {
                units = ceil_div(D, P::kc);
                warps = most;
                steps = 1;
            } else if (phase == 2) {
                units = t_hi - t_lo;
                warps = min(units, most);
                steps = ceil_div(D, P::kc);
            } else {
                if (!ok || d0 >= d_hi) break;
                if (h0 == 0) bt = next_batch(m, bx, n, T, p.hcap);
                nr = min(32, d_hi - d0);
                tp = (nr + 15) / 16;
                units = (bt.x1 - bt.x0) * tp;
                warps = min(units, most / tp * tp);
                K = I;
                col0 = h0;
                width = min(kHCols, I - h0);
                steps = ceil_div(width, P::kc);
            }
            Turn t(at, warps, 0);
#pragma unroll 1
            for (int u0 = 0; u0 < units; u0 += warps) {
                // lane v: the unit of this producer's vth warp
                const int u = u0 + me + lane * NP;
                const bool have = me + lane * NP < min(warps, units - u0);
                int64_t row = 0;
                int count = 0, c0 = 0;  // count: rows of its first matrix, and of the second << 8
                if (have && phase == 1) {
                    row = (int64_t)E * I + 8 * f1;
                    count = 8 * 0x101;
                    c0 = u * P::kc;
                } else if (have && phase == 2) {
                    const int pos = (t_lo + u) / (I / 8);
                    row = (int64_t)m.expert[pos] * I + 8 * (t_lo + u - pos * (I / 8));
                    count = 8 * 0x101;
                } else if (have) {
                    const int x = bt.x0 + (tp == 2 ? u >> 1 : u), j = tp == 2 ? u & 1 : 0, rows = min(16, nr - 16 * j);
                    row = (int64_t)(x < 0 ? E : m.expert[x]) * D + d0 + 16 * j;
                    count = min(rows, 8) | max(rows - 8, 0) << 8;
                }
                const int mine = __popc(__ballot_sync(0xffffffffu, have));
#pragma unroll 1
                for (int s = 0; s < steps; ++s, t.next())
#pragma unroll 1
                    for (int v = 0; v < mine; ++v) {
                        const int64_t r = __shfl_sync(0xffffffffu, row, v);
                        const int c = __shfl_sync(0xffffffffu, count, v), at0 = __shfl_sync(0xffffffffu, c0, v) + s * P::kc;
                        const bool down = phase == 3;
                        fill(t, me + v * NP, down ? 2 : 0, r, c & 255, down ? 2 : 1, down ? r + 8 : r, c >> 8, K, col0 + at0, min(P::kc, width - at0));
                    }
            }
            finish(warps, units, steps);
            if (phase == 1) {
                ++f1;
            } else if (phase == 2) {
                phase = 3;
            } else if ((h0 += kHCols) >= I) {  // the next batch; after the last, the next rows
                h0 = 0;
                bx = bt.x1;
                if (bx >= n) {
                    bx = -1;
                    d0 += 32;
                }
            }
        }
        if (!ok) tc::sleep_ns(200000);  // copies already issued land before the CTA leaves
        return;
    }

    // ---------------------------------------------------------- consumers
    // A wait that runs out raises the abort flag; every warp then runs on
    // through the same barriers (later waits return at once) to the end.
    const int tid = threadIdx.x;
    auto stage_wait = [&](const Turn& t) -> const uint8_t* {
        const int s = t.stage();
        if (!tc::mbar_wait(smem_u32(m.full + s), t.phase(s), lim, abort) && !*abort) {
            record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 42, cta, 0);
            *abort = 1;
        }
        __syncwarp();
        return ring + s * P::stage;
    };
    auto stage_done = [&](Turn& t) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(smem_u32(m.empty + t.stage()));
        t.next();
    };
    // The tile rows this lane takes, such that the 16-byte pieces of lanes 0
    // to 7, of two rows, lie in different banks: rows 0 and 4 (1 and 5, ..) of
    // lines of 128 bytes, neighbours where lines are 64 bytes.
    const int rw = kIn == 128 ? (g >> 1) | ((g & 1) << 2) : g;
    const int swz = kIn == 128 ? rw * 16 : ((rw >> 1) & 3) * 16;
    const int xstride = x_stride<W>(D);
    float* xsc = (float*)(act + up(T * xstride, 128));  // its scales, [T][per row]
    const int nxs = x_scales<W>(D) / 4;

    // One stage of a tile of na and nb rows (halves that are boxes where they
    // are whole): `cols` columns against the activation rows ta (this lane's
    // token row of each token tile at the stage's first column; fp32: the
    // lane's two accumulator tokens in t0, t1), with their scales sc0, sc1 (of
    // the two accumulator tokens) and the weights' block scales (FP8: wa,
    // wb; 4 bits: in the stage, or ga, gb in memory).
    auto stage_dot = [&](const uint8_t* tile, int na, int nb, int cols, const uint8_t* const (&ta)[NT], const uint8_t* const (&tb)[NT],
                         const float* const (&sc0)[NT], const float* const (&sc1)[NT], const void* ga, const void* gb, const BlockScales& wa,
                         const BlockScales& wb, auto f16,
                         int lo_at, float (&acc)[NT][4]) {
        const int bytes = bytes_of<W>(cols);
        const bool boxa = na == 8, boxb = nb == 8;
        const uint8_t* tile1 = tile + (boxa ? 8 * P::box : na * (bytes + 16));
        RowPair r;
        r.a = tile + (boxa ? rw * kIn : min(rw, na - 1) * (bytes + 16));
        r.xa = boxa ? swz : 0;
        r.b = nb == 0 ? r.a : tile1 + (boxb ? rw * kIn : min(rw, nb - 1) * (bytes + 16));
        r.xb = nb == 0 ? r.xa : boxb ? swz : 0;
        const int da = boxa ? 8 * kIn : kIn, db = nb == 0 ? da : boxb ? 8 * kIn : kIn;
        r.line_a = da;
        r.line_b = db;
        [[maybe_unused]] const uint8_t *ka = nullptr, *kb = nullptr;
        if constexpr (W == MOE_MXFP4) {
            if (p.tma_scales) {
                const uint8_t* sc = tile + P::data;
                ka = sc + (boxa ? rw * (P::kc / 32) : min(rw, na - 1) * (cols / 32));
                kb = nb == 0 ? ka : sc + (boxa ? 8 * P::kc / 32 : na * (cols / 32)) + (boxb ? rw * (P::kc / 32) : min(rw, nb - 1) * (cols / 32));
            } else {
                ka = (const uint8_t*)ga;
                kb = (const uint8_t*)gb;
            }
        }
        const int slices = cols / kSlice;
        if constexpr (ONE) {
            dot_one(r, ta[0], slices, ka, kb, sc0[0], smem_zeros, acc[0]);
        } else if constexpr (W == MOE_FP8_E4M3_B128) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s < slices) {
                    const uint8_t* xc[NT];
                    float sx[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) xc[n] = ta[n] + s * kSlice * Tr<W>::xb, sx[n][0] = sc0[n][s], sx[n][1] = sc1[n][s];
                    dot_fp8<NT>(r, xc, wa.s[s], wb.s[s], sx, acc);
                    r.a += da;
                    r.b += db;
                }
            }
        } else {
#pragma unroll 2
        for (int s = 0; s < slices; ++s) {
            if constexpr (W == MOE_F32) {
#pragma unroll
                for (int n = 0; n < NT; ++n) dot_f32(r, ta[n] + s * kSlice * 4, tb[n] + s * kSlice * 4, acc[n]);
            } else {
                const uint8_t* xc[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) xc[n] = ta[n] + s * kSlice * Tr<W>::xb;
                if constexpr (W == MOE_BF16) {
                    dot16<NT, decltype(f16)::value>(r, xc, acc);
                } else if constexpr (W == W_HILO) {
                    dot16<NT, false>(r, xc, acc);
                    if (lo_at) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) xc[n] += lo_at;
                        dot16<NT, false>(r, xc, acc);
                    }
                } else {
                    float4 sx[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) sx[n][0] = *(const float4*)(sc0[n] + 4 * s), sx[n][1] = *(const float4*)(sc1[n] + 4 * s);
                    dot_mx<NT>(r, xc, *(const uint32_t*)(ka + 4 * s), *(const uint32_t*)(kb + 4 * s), sx, acc);
                }
            }
            r.a += da;
            r.b += db;
        }
        }
    };

    unsigned long long target = 0;
    if (tid == 0) {
        unsigned long long v;
        asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p.bar) : "memory");
        target = (v / grid + 1) * grid;
    }
    // x into shared memory, as the expert products read it
    if constexpr (!kScaled) {
        const int per = D * Tr<W>::xb / 32;
        each_unit<2, 2>(
            T * per, [&](int u, uint4* v) { v[0] = __ldg((const uint4*)p.x + 2 * u), v[1] = __ldg((const uint4*)p.x + 2 * u + 1); },
            [&](int u, bool on, const uint4* v) {
                const int t = u / per, c = u - t * per;
                uint4* dst = (uint4*)(act + t * xstride + c * 32);
                if (on) dst[0] = v[0], dst[1] = v[1];
            });
    } else {
        const int per = D / 16;  // a unit: 16 columns
        each_unit<2, 2>(
            T * per, [&](int u, uint4* v) { v[0] = __ldg((const uint4*)p.x + 2 * u), v[1] = __ldg((const uint4*)p.x + 2 * u + 1); },
            [&](int u, bool on, const uint4* x) {
                const int t = u / per, c = u - t * per;
                float v[16];
                const bf16* b = (const bf16*)x;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __bfloat162float(b[i]);
                uint8_t* row = act + t * xstride;
                if constexpr (W == MOE_FP8_E4M3_B128) {
                    const float s = quant16_fp8(v, row + c * 32, on);
                    if ((c & 7) == 0 && on) xsc[t * nxs + c / 8] = s;
                } else {
                    const float s = quant16_mx(v, row + c * 32, on);
                    if ((c & 1) == 0 && on) xsc[t * nxs + c / 2] = s;
                }
            });
    }
#pragma unroll 1
    for (int i = tid; i < 512; i += kCons) m.mask[i] = 0;
    // x rows of this lane: tokens 8 n + g, and its accumulators' tokens (8 n + 2 q, + 1)
    const uint8_t *xrow[NT], *xrow0[NT], *xrow1[NT];
    const float *xs0[NT], *xs1[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t0 = min(8 * n + 2 * q, T - 1), t1 = min(8 * n + 2 * q + 1, T - 1);
        xrow[n] = act + min(8 * n + g, T - 1) * xstride;
        xrow0[n] = act + t0 * xstride;
        xrow1[n] = act + t1 * xstride;
        xs0[n] = xsc + t0 * nxs;
        xs1[n] = xsc + t1 * nxs;
    }

    // -------------------------------------------------------------- P0
    // One tile of rows, its stages spread over the warps.  (x straight from
    // global memory: its rows are in the caches, and the products below read
    // it quantised)
    for (int e0 = e_lo; e0 < e_hi; e0 += 16) {
        const int ne = min(16, e_hi - e0), step = router_cols<W, NT>(ne, D), chunks = ceil_div(D, step);
        float acc[NT][4] = {};
        if (warp < most) {
            Turn turn(at, most, warp);
            for (int c = warp; c < chunks; c += most) {
                const int c0 = c * step, cols = min(step, D - c0), stride = cols * P::eb + 16;
                const uint8_t* tile = stage_wait(turn);
                RowPair r = {tile + min(rw, ne - 1) * stride, tile + min(rw + 8, ne - 1) * stride, 0, 0, 0, 0};
#pragma unroll 4
                for (int i = 0; i < cols; i += P::rslice) {
                    const uint8_t* xg = (const uint8_t*)p.x + (int64_t)(c0 + i) * P::eb;
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
                    r.a += P::rslice * P::eb;
                    r.b += P::rslice * P::eb;
                }
                stage_done(turn);
            }
        }
        at.finish(most, chunks, 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) m.red[(warp * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        consumers_sync();
        if (warp < NT) {  // warp n: token tile n
            float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 4
            for (int v = 0; v < NW; ++v) {
                const float4 a = m.red[(v * NT + warp) * 32 + lane];
                s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
            }
            const float z[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = rw + 8 * r;
                const float bias = p.b_router && row < ne ? __ldg(p.b_router + e0 + row) : 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int tok = 8 * warp + 2 * q + t;
                    if (row < ne && tok < T) p.logits[(int64_t)tok * E + e0 + row] = z[2 * r + t] + bias;
                }
            }
        }
        consumers_sync();  // logits written, red read
    }
    consumers_sync();  // x in shared memory (also where there are no router rows)
    if (tid == 0) grid_arrive(p.bar);

    bool overflow = false;
    auto put_h = [&](int64_t o, float h) {
        if constexpr (W == MOE_BF16) {
            if (!(fabsf(h) <= 65504.0f)) overflow = true;
            ((f16*)p.h)[o] = __float2half_rn(h);
        } else {
            p.h[o] = h;
        }
    };
    // h of the tile of eight features f0 .. of the expert at place pos (-1: shared)
    auto put_tile = [&](float (&acc)[NT][4], int pos, int f0) {
        if constexpr (ONE) sum_quad(acc[0]);
        const int row = pos < 0 ? T * k : m.hrow[pos];
        const uint32_t tokens = pos < 0 ? 0xFFFFu : m.tokens[pos];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int t = 8 * u + 2 * q + s;
                if (t < T && ((tokens >> t) & 1u))
                    put_h((int64_t)(row + __popc(tokens & ((1u << t) - 1u))) * I + f0 + rw,
                          W == MOE_F32 ? swiglu_f32(acc[u][s], acc[u][2 + s]) : swiglu(acc[u][s], acc[u][2 + s]));
            }
    };
    // the warps' sums of token tile u, in warp order
    auto sum_red = [&](int u, float (&z)[4]) {
        z[0] = z[1] = z[2] = z[3] = 0.0f;
#pragma unroll 4
        for (int v = 0; v < NW; ++v) {
            const float4 a = m.red[(v * NT + u) * 32 + lane];
            z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
        }
    };
    // A stage, columns c0 .., of the tile of eight features f0 .. of expert e.
    auto gateup_stage = [&](Turn& turn, int e, int f0, int c0, float (&acc)[NT][4]) {
        const int cols = min(P::kc, D - c0), fr = f0 + rw;
        const uint8_t *ta[NT], *tb[NT];
        const float *sa[NT], *sb[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            ta[u] = (W == MOE_F32 ? xrow0[u] : xrow[u]) + c0 * Tr<W>::xb;
            tb[u] = xrow1[u] + c0 * Tr<W>::xb;
            sa[u] = xs0[u] + c0 / 128 * Tr<W>::nsc;
            sb[u] = xs1[u] + c0 / 128 * Tr<W>::nsc;
        }
        const void *ga = nullptr, *gb = nullptr;
        BlockScales wa = {}, wb = {};
        if constexpr (W == MOE_FP8_E4M3_B128) {
            const int64_t blk = ((int64_t)e * (I / 128) + fr / 128) * (D / 128) + c0 / 128;
            wa.fetch((const float*)p.s_gate + blk, cols);
            wb.fetch((const float*)p.s_up + blk, cols);
        } else if constexpr (W == MOE_MXFP4) {
            const int64_t blk = ((int64_t)e * I + fr) * (D / 32) + c0 / 32;
            ga = (const uint8_t*)p.s_gate + blk;
            gb = (const uint8_t*)p.s_up + blk;
        }
        const uint8_t* tile = stage_wait(turn);
        stage_dot(tile, 8, 8, cols, ta, tb, sa, sb, ga, gb, wa, wb, No{}, 0, acc);
        stage_done(turn);
    };
    // ---------------------------------------------- barrier 1, top-k, list
    if (tid == 0 && !grid_wait(p.bar, target, lim, abort)) {
        if (!*abort) record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 43, cta, 0);
        *abort = 1;
    }
    consumers_sync();
    uint32_t bad = 0;
    const int keyed = min(NW, (int)sizeof(m.red) / (4 * E));  // warps that have room for their keys
    for (int t = warp < keyed ? warp : T; t < T; t += keyed) {
        topk_token(p, t, m, (uint32_t*)m.red + warp * E, bad);
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
        // ascending list of the touched experts: four experts (two words) a thread of the first eight warps
        uint32_t both[2] = {0, 0}, sum = 0, inc = 0;
        if (warp < 8) {
            both[0] = m.mask[2 * tid];
            both[1] = m.mask[2 * tid + 1];
#pragma unroll
            for (int j = 0; j < 2; ++j)  // experts | rows << 16
                sum += ((both[j] & 0xFFFFu) ? 1u : 0u) + ((both[j] >> 16) ? 1u : 0u) + ((uint32_t)__popc(both[j]) << 16);
            inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) m.scan[warp] = inc;
        }
        consumers_sync();
        if (warp < 8) {
            uint32_t pl = inc - sum;
#pragma unroll
            for (int v = 0; v < 8; ++v) pl += v < warp ? m.scan[v] : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t bits = (both[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, place = pl & 0xFFFFu;
                if (bits) {
                    m.expert[place] = (uint16_t)(4 * tid + j);
                    m.tokens[place] = (uint16_t)bits;
                    m.hrow[place] = (uint16_t)(pl >> 16);
                    pl += 1u + ((uint32_t)__popc(bits) << 16);
                }
                both[j >> 1] = (both[j >> 1] & ~(0xFFFFu << (16 * (j & 1)))) | place << (16 * (j & 1));
            }
            m.mask[2 * tid] = both[0];
            m.mask[2 * tid + 1] = both[1];
            if (tid == 255) {
                m.n = pl & 0xFFFFu;
                m.hrow[pl & 0xFFFFu] = (uint16_t)(pl >> 16);
            }
        }
    }
    consumers_sync();
    if (tid == 0) tc::mbar_arrive(smem_u32(&m.list_ready));
#pragma unroll 1
    for (int i = tid; i < T * k; i += kCons) {
        const int pos = ((const uint16_t*)m.mask)[m.sel[i]], t = i / k;
        m.wt[m.hrow[pos] + __popc(m.tokens[pos] & ((1u << t) - 1u))] = m.selw[i];  // read after the next barrier
    }
    const int n = m.n;

    // ------------------------------------------------------------ P1, P2
    // P1's tiles (the shared expert's), as P0's: stages spread over the
    // warps; then P2's, a tile a warp.
    int t_lo, t_hi;
    share(n * (I / 8), cta, grid, t_lo, t_hi);
#pragma unroll 1
    for (int f1 = f_lo;; ++f1) {
        const bool p1 = f1 < f_hi;
        const int chunks = ceil_div(D, P::kc), units = p1 ? chunks : t_hi - t_lo, warps = p1 ? most : min(units, most);
        if (units == 0) break;
        float acc[NT][4] = {};
        int pos = -1, f0 = 8 * f1;
        Turn turn(at, warps, warp);
#pragma unroll 1
        for (int j = warp; j < (warp < warps ? units : 0); j += warps) {
            if (!p1) {
                pos = (t_lo + j) / (I / 8);
                f0 = 8 * (t_lo + j - pos * (I / 8));
            }
            const int e = p1 ? E : m.expert[pos];
#pragma unroll 1
            for (int c0 = p1 ? j * P::kc : 0, c1 = p1 ? c0 + 1 : D; c0 < c1; c0 += P::kc) gateup_stage(turn, e, f0, c0, acc);
            if (!p1) {
                put_tile(acc, pos, f0);
#pragma unroll
                for (int u = 0; u < NT; ++u) acc[u][0] = acc[u][1] = acc[u][2] = acc[u][3] = 0.0f;
            }
        }
        at.finish(warps, units, p1 ? 1 : chunks);
        if (!p1) break;
#pragma unroll
        for (int u = 0; u < NT; ++u) m.red[(warp * NT + u) * 32 + lane] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
        consumers_sync();
        if (warp == 0) {
#pragma unroll
            for (int u = 0; u < NT; ++u) sum_red(u, acc[u]);
            put_tile(acc, -1, f0);
        }
        consumers_sync();
    }
    if (overflow) record_error(p.err, MOE_ERR_NONFINITE, 5, cta, 0);
    consumers_sync();
    if (tid == 0) {
        grid_arrive(p.bar);
        target += grid;
        if (!grid_wait(p.bar, target, lim, abort)) {
            if (!*abort) record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 44, cta, 0);
            *abort = 1;
        }
    }
    consumers_sync();

    // -------------------------------------------------------------- P3
    const int hstride = h_stride<W>(I), nhs = h_scales<W>(I) / 4;
    float* hsc = (float*)(act + up(p.hcap * hstride, 128));
    const int lo_at = W == W_HILO ? min(I, kHCols) * 2 : 0;  // a row is its high halves, then its low halves
    for (int d0 = d_lo; d0 < d_hi; d0 += 32) {
        // tile t of the pass: rows 16 t ..; warp: tile warp % tp, of every (units)th expert
        const int nrows = min(32, d_hi - d0), tp = (nrows + 15) / 16, tile_no = warp % tp;
        const int nr = min(16, nrows - 16 * tile_no), na = min(nr, 8), nb = max(nr - 8, 0), r0 = d0 + 16 * tile_no;
        float out[NT][4] = {};
        for (int bx = -1; bx < n;) {
            const Batch bt = next_batch(m, bx, n, T, p.hcap);
            for (int h0 = 0; h0 < I; h0 += kHCols) {
                const int hc = min(kHCols, I - h0);
                {
                    // this batch's rows of h, 16 columns (8 in fp32) a unit
                    constexpr int kUnit = W == MOE_F32 ? 8 : 16, kWords = W == MOE_F32 || W == MOE_BF16 ? 2 : 4;
                    const int per = hc / kUnit;
                    each_unit<kWords, 2>(
                        bt.rows * per,
                        [&](int u, uint4* v) {
                            const int r = u / per, c = u - r * per;
                            const int64_t row = r < bt.shared ? T * k + r : bt.row0 + r - bt.shared;
                            const uint4* src = (const uint4*)((const uint8_t*)p.h + (row * I + h0 + c * kUnit) * (W == MOE_BF16 ? 2 : 4));
#pragma unroll
                            for (int i = 0; i < kWords; ++i) v[i] = __ldcg(src + i);
                        },
                        [&](int u, bool on, const uint4* h) {
                            const int r = u / per, c = u - r * per;
                            uint8_t* dst = act + r * hstride + c * 32;
                            if constexpr (kWords == 2) {
                                if (on) ((uint4*)dst)[0] = h[0], ((uint4*)dst)[1] = h[1];
                            } else {
                                float v[16];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    v[4 * i] = __uint_as_float(h[i].x), v[4 * i + 1] = __uint_as_float(h[i].y);
                                    v[4 * i + 2] = __uint_as_float(h[i].z), v[4 * i + 3] = __uint_as_float(h[i].w);
                                }
                                if constexpr (W == MOE_FP8_E4M3_B128) {
                                    const float s = quant16_fp8(v, dst, on);
                                    if ((c & 7) == 0 && on) hsc[r * nhs + c / 8] = s;
                                } else if constexpr (W == MOE_MXFP4) {
                                    const float s = quant16_mx(v, dst, on);
                                    if ((c & 1) == 0 && on) hsc[r * nhs + c / 2] = s;
                                } else if (on) {
                                    uint32_t hi[8], lo[8];
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        hi[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                                        const float2 b = __bfloat1622float2(*(const __nv_bfloat162*)&hi[i]);
                                        lo[i] = pack_bf16(v[2 * i] - b.x, v[2 * i + 1] - b.y);
                                    }
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        ((uint4*)dst)[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                                        ((uint4*)(dst + lo_at))[i] = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                                    }
                                }
                            }
                        });
                }
                consumers_sync();
                const int units = (bt.x1 - bt.x0) * tp, warps = min(units, most / tp * tp);
                Turn turn(at, warps, warp);
                for (int un = warp; un < (warp < warps ? units : 0); un += warps) {
                    const int x = bt.x0 + (tp == 2 ? un >> 1 : un);
                    {
                        const uint32_t tokens = x < 0 ? 0xFFFFu : m.tokens[x];
                        const int grow = x < 0 ? 0 : m.hrow[x];                    // row of wt
                        const int brow = x < 0 ? 0 : bt.shared + grow - bt.row0;   // row of the buffer
                        const int e = x < 0 ? E : m.expert[x];
                        int rank[NT][2];  // of the lane's accumulator tokens among the expert's; -1: not its token
                        const uint8_t *ha[NT], *hb[NT];
                        const float *sa[NT], *sb[NT];
#pragma unroll
                        for (int u = 0; u < NT; ++u) {
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                const int t = 8 * u + 2 * q + s;
                                rank[u][s] = t < T && ((tokens >> t) & 1u) ? __popc(tokens & ((1u << t) - 1u)) : -1;
                            }
                            const int t = 8 * u + g;
                            const int r = t < T && ((tokens >> t) & 1u) ? __popc(tokens & ((1u << t) - 1u)) : 0;
                            ha[u] = act + (brow + (W == MOE_F32 ? max(rank[u][0], 0) : r)) * hstride;
                            hb[u] = act + (brow + max(rank[u][1], 0)) * hstride;
                            sa[u] = hsc + (brow + max(rank[u][0], 0)) * nhs;
                            sb[u] = hsc + (brow + max(rank[u][1], 0)) * nhs;
                        }
                        const void *ga = nullptr, *gb = nullptr;
                        if constexpr (W == MOE_FP8_E4M3_B128) {
                            const float* sd = (const float*)p.s_down + h0 / 128;
                            ga = sd + ((int64_t)e * (D / 128) + (r0 + min(rw, na - 1)) / 128) * (I / 128);
                            gb = sd + ((int64_t)e * (D / 128) + (r0 + min(rw + 8, nr - 1)) / 128) * (I / 128);
                        } else if constexpr (W == MOE_MXFP4) {
                            const uint8_t* sd = (const uint8_t*)p.s_down + h0 / 32;
                            ga = sd + ((int64_t)e * D + r0 + min(rw, na - 1)) * (I / 32);
                            gb = sd + ((int64_t)e * D + r0 + min(rw + 8, nr - 1)) * (I / 32);
                        }
                        float y[NT][4] = {};
#pragma unroll 1
                        for (int c0 = 0; c0 < hc; c0 += P::kc) {
                            const int cols = min(P::kc, hc - c0);
                            BlockScales wa = {}, wb = {};
                            if constexpr (W == MOE_FP8_E4M3_B128) {
                                wa.fetch(ga, cols);
                                wb.fetch(gb, cols);
                            }
                            const uint8_t* tile = stage_wait(turn);
                            stage_dot(tile, na, nb, cols, ha, hb, sa, sb, ga, gb, wa, wb, Yes{}, lo_at, y);
                            stage_done(turn);
#pragma unroll
                            for (int u = 0; u < NT; ++u) {
                                ha[u] += P::kc * (W == W_HILO ? 2 : Tr<W>::hb);
                                hb[u] += P::kc * Tr<W>::hb;
                                sa[u] += P::kc / 128 * Tr<W>::nsc;
                                sb[u] += P::kc / 128 * Tr<W>::nsc;
                            }
                            if constexpr (W == MOE_FP8_E4M3_B128) {
                                ga = (const float*)ga + P::kc / 128;
                                gb = (const float*)gb + P::kc / 128;
                            } else if constexpr (W == MOE_MXFP4) {
                                ga = (const uint8_t*)ga + P::kc / 32;
                                gb = (const uint8_t*)gb + P::kc / 32;
                            }
                        }
                        if constexpr (ONE) sum_quad(y[0]);
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
                at.finish(warps, units, ceil_div(hc, P::kc));
                consumers_sync();  // the batch, and with it the buffer, is done
            }
            bx = bt.x1;
        }
        // the warps' sums, by tile, in warp order
#pragma unroll
        for (int u = 0; u < NT; ++u) m.red[(warp * NT + u) * 32 + lane] = make_float4(out[u][0], out[u][1], out[u][2], out[u][3]);
        consumers_sync();
        if (warp < tp * NT) {
            const int tl = warp % tp, u = warp / tp, rows = min(16, nrows - 16 * tl);
            float s[4] = {0, 0, 0, 0};
#pragma unroll 2
            for (int v = tl; v < NW; v += tp) {
                const float4 a = m.red[(v * NT + u) * 32 + lane];
                s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int tok = 8 * u + 2 * q + t, d = rw + 8 * r;
                    if (tok < T && d < rows) {
                        const int64_t o = (int64_t)tok * D + d0 + 16 * tl + d;
                        if (p.out_elem == kF32) ((float*)p.out)[o] = s[2 * r + t];
                        else ((bf16*)p.out)[o] = __float2bfloat16_rn(s[2 * r + t]);
                    }
                }
        }
        consumers_sync();
    }
}

constexpr int kSmemLimit = 232448;

// Shared memory for T tokens: rows of h's buffer, where the ring starts, and
// its stages.
template <int W, int NT> bool plan_smem(int T, int D, int I, int k, int* hcap, int* ring_at, int* stages) {
    const int64_t misc = up((int)sizeof(Misc), 128);
    const int64_t x = (int64_t)up(T * x_stride<W>(D), 128) + up(T * x_scales<W>(D), 128);
    const int64_t hrow = h_stride<W>(I) + h_scales<W>(I);
    // h's buffer takes x's place; at least the rows of one expert, at most
    // all of them, and beyond x only what leaves a ring of twelve stages
    const int64_t all = (int64_t)T * (k + 1);
    const int64_t room = std::max(x, std::min(all * hrow + 256, (int64_t)kSmemLimit - misc - 12 * 512 / Plan<W, NT>::box * Plan<W, NT>::stage));
    const int64_t cap = std::max<int64_t>(T, std::min(all, (room - 256) / hrow));
    const int64_t at = misc + std::max(x, cap * hrow + 256);
    if (at > kSmemLimit) return false;
    *hcap = (int)cap;
    *ring_at = up((int)at, 1024);
    *stages = std::min(kMaxStages, (kSmemLimit - *ring_at) / Plan<W, NT>::stage);
    return *stages >= 4;
}

// A matrix of `rows` rows of `bytes` as boxes of 8 rows and `box` bytes,
// laid out [line of `in` bytes][row][in], swizzled over a line.
template <int W, int NT> bool weight_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes) {
    constexpr int in = Tr<W>::in;
    const cuuint64_t dims[3] = {in, (cuuint64_t)rows, (cuuint64_t)(bytes / in)};
    const cuuint64_t strides[2] = {(cuuint64_t)bytes, in};
    const cuuint32_t box[3] = {in, 8, Plan<W, NT>::box / in}, es[3] = {1, 1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           in == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Scale bytes [rows, bytes], boxes of 8 rows and a stage's columns.
bool scale_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes) {
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {Plan<MOE_MXFP4, 1>::kc / 32, 8}, es[2] = {1, 1};
    return tc::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int W, int NT, bool ONE = false> cudaError_t launch(FewParams p, int num_sms, cudaStream_t s) {
    if (!plan_smem<W, NT>(p.T, p.D, p.I, p.k, &p.hcap, &p.ring_at, &p.stages)) return cudaErrorInvalidConfiguration;
    Maps maps = {};
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    const int64_t gr = (int64_t)(p.E + 1) * p.I, dr = (int64_t)(p.E + 1) * p.D;
    bool ok = weight_map<W, NT>(&maps.w[0], p.w_gate, gr, bytes_of<W>(p.D)) && weight_map<W, NT>(&maps.w[1], p.w_up, gr, bytes_of<W>(p.D)) &&
              weight_map<W, NT>(&maps.w[2], p.w_down, dr, bytes_of<W>(p.I));
    // scales by TMA where their rows are whole 16-byte pieces
    p.tma_scales = W == MOE_MXFP4 && p.D % 512 == 0 && p.I % 512 == 0;
    if (p.tma_scales)
        ok = ok && scale_map(&maps.s[0], p.s_gate, gr, p.D / 32) && scale_map(&maps.s[1], p.s_up, gr, p.D / 32) &&
             scale_map(&maps.s[2], p.s_down, dr, p.I / 32);
    if (!ok) return cudaErrorInvalidValue;
    const int bytes = p.ring_at + p.stages * Plan<W, NT>::stage;
    cudaError_t e = ensure_smem_attr((const void*)few_kernel<W, NT, ONE>, kSmemLimit);
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
    e = cudaLaunchKernelEx(&cfg, few_kernel<W, NT, ONE>, p, maps);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int W> cudaError_t launch_chunks(const FewParams& p, int num_sms, cudaStream_t s) {
    // As many tokens at a time as their x leaves room for a ring of
    // four stages (16 at D = 4096; wider rows take a few launches).  4 bits:
    // at most eight, since there the products of a second token tile cost
    // more than reading the weights again (16 tokens, D = 4096, I = 1024,
    // E = 128: 366 us in one launch, 282 in two; FP8 302 against 332).
    constexpr int kTiles = W == MOE_MXFP4 ? 1 : 2;
    const int launches = (p.T + 7) / 8;
    int per = W == MOE_MXFP4 ? (p.T + launches - 1) / launches : std::min(p.T, kFewMax), hcap, ring_at, stages;
    while (per > 1 && !(per > 8 ? plan_smem<W, kTiles> : plan_smem<W, 1>)(per, p.D, p.I, p.k, &hcap, &ring_at, &stages)) --per;
    for (int t0 = 0; t0 < p.T; t0 += per) {
        FewParams c = p;
        c.T = std::min(per, p.T - t0);
        c.tok0 = t0;
        c.plane = p.T * p.k;
        c.x = (const char*)p.x + (int64_t)t0 * p.D * (W == MOE_F32 ? 4 : 2);
        c.logits = p.logits + (int64_t)t0 * p.E;
        c.blob = p.blob + t0 * p.k;
        c.out = (char*)p.out + (int64_t)t0 * p.D * (p.out_elem == kF32 ? 4 : 2);
        const cudaError_t e = W == MOE_MXFP4 && c.T == 1 ? launch<W, 1, W == MOE_MXFP4>(c, num_sms, s) : c.T <= 8 ? launch<W, 1>(c, num_sms, s) : launch<W, kTiles>(c, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace few

// One token fits: its x and a ring of four stages in an SM's shared memory
// (all that a plan takes but fp32 rows of 43136 columns and more).
bool few_fits(int dtype, int down_f16, int D, int I, int k) {
    int hcap, ring_at, stages;
    switch (dtype) {
        case MOE_F32: return few::plan_smem<MOE_F32, 1>(1, D, I, k, &hcap, &ring_at, &stages);
        case MOE_BF16:
            return (down_f16 ? few::plan_smem<MOE_BF16, 1> : few::plan_smem<few::W_HILO, 1>)(1, D, I, k, &hcap, &ring_at, &stages);
        case MOE_FP8_E4M3_B128: return few::plan_smem<MOE_FP8_E4M3_B128, 1>(1, D, I, k, &hcap, &ring_at, &stages);
        default: return few::plan_smem<MOE_MXFP4, 1>(1, D, I, k, &hcap, &ring_at, &stages);
    }
}

cudaError_t launch_few(const FewParams& p, int num_sms, cudaStream_t s) {
    switch (p.dtype) {
        case MOE_F32: return few::launch_chunks<MOE_F32>(p, num_sms, s);
        case MOE_BF16: return p.down_f16 ? few::launch_chunks<MOE_BF16>(p, num_sms, s) : few::launch_chunks<few::W_HILO>(p, num_sms, s);
        case MOE_FP8_E4M3_B128: return few::launch_chunks<MOE_FP8_E4M3_B128>(p, num_sms, s);
        default: return few::launch_chunks<MOE_MXFP4>(p, num_sms, s);
    }
}

}  // namespace moe

// Products of rows grouped by expert on the tensor cores, bf16 with fp32 sums
// (moe_grouped_gemm and its gradients), and rows times 4-bit weights for many
// rows (moe_int4_gemm).  One kernel, D[f][i] = sum_c F(f, c) R(i, c):
//
//            f (MMA M, 128 a tile)   i (MMA N)      c               F lies   R lies
//   forward  features of w_g         rows of g      columns of x    along c  along c
//   dx       columns of w_g          rows of g      features of w_g along f  along c
//   dw       columns of x            columns of dy  rows of g       along f  along i
//
// f is what the output is contiguous along.  tcgen05 takes an operand that is
// contiguous along M or N as readily as one along K, so nothing is transposed:
// a stage holds 64 of c in 128-byte swizzled lines, of 64 c for each f or i,
// or of 64 f or i for each c.  The rows of a group are the MMA's N side in
// steps of 16, so a small group costs tensor time for its rows only.
//
// dw sums over a group's rows, which end anywhere: the lines of the last 16
// that lie past the end hold the next group's rows, and the MMA warp writes
// zeros over them in both operands (their values may be anything, and times
// zero need not be zero).  Columns past a matrix's edge are filled with zeros
// by TMA; w is mapped as [G][N][K], so that dx's sum ends with its own matrix.
//
// Measured (us; bytes or operations at the measured copy and GEMM rates in
// brackets).  16384 rows in 8 groups, 4096 x 4096: 338 to 347 (275) in a loop, 303 at
// the first calls after a pause: the power limit.  One CTA a tile took 369,
// with 73 % of the tensor pipe's cycles used and 4 stages of 48 KB on the way;
// pairs have 6 of 32.  64 ragged groups: forward of 4001 rows, 1024 x 4096, 100
// (86); dx of 16380 rows 131 (105); dw, fp32, 220 (185): HBM, at 5.6 to 5.8 of
// 6.7 TB/s.  2047 rows by 4096 x 4096 codes 57 (34): the MMAs (240 rows by 128
// features) use 55 % of the tensor pipe's cycles, the rest are waits for decoded
// stages, some 850 cycles each where the MMAs take 480.
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "groups.cuh"
#include "int4.cuh"
#include "internal.h"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu
}
namespace ptc {

using namespace tc;

// Where a stage's operands come from: TMA alone; or the lines of an
// operand that TMA cannot read (rows not aligned to 16 bytes) copied by warps;
// or the F operand's 4-bit codes turned into bf16 by them (bf16 or fp32
// scales), R by TMA or copied.
enum Feed { kTma = 0, kCopy = 1, kCodes16 = 2, kCodes32 = 3 };

constexpr int BF = 128, BK = 64, kMaxI = 256;  // f and c of a stage, i of a tile at most
constexpr int kLine = 128;                     // bytes
constexpr int kFBytes = BF * BK * 2;
constexpr int kMaxStages = 8;
// Epilogue warps, and groups of four warps that feed stages: a stage is a long
// way for one group, so four, and fewer epilogue warps for their registers.
constexpr int kFeedGroup = 4;
__host__ __device__ constexpr int epi_warps(int feed) { return feed == kTma ? 8 : 4; }
__host__ __device__ constexpr int feed_groups(int feed) { return feed == kTma ? 0 : 4; }
__host__ __device__ constexpr int threads_for(int feed) {  // (codes: and a warp that loads them)
    return 32 * (2 + epi_warps(feed) + kFeedGroup * feed_groups(feed) + (feed >= kCodes16 ? 1 : 0));
}
constexpr int kMaxSplit = 8;
constexpr int kRing = 4 * (kFBytes + kMaxI * BK * 2);
constexpr int kStWarp = 8 * 32 * 4;            // 8 row pairs x 32 features, two bf16 a word
// shared memory: ring, barriers, codes (BF rows of 32 bytes a slot, a slot a stage), epilogue staging, groups' table
constexpr int kOffBar = kRing;
constexpr int kCodeSlots = 4, kCodeBytes = BF * BK / 2;
constexpr int kOffCodes = kOffBar + 512;
__host__ __device__ constexpr int off_stage(int feed) { return kOffCodes + (feed >= kCodes16 ? kCodeSlots * kCodeBytes : 0); }
__host__ __device__ constexpr int off_table(int feed) { return off_stage(feed) + epi_warps(feed) * kStWarp; }
__host__ __device__ constexpr int smem_bytes(int feed) { return off_table(feed) + (int)sizeof(GroupTable); }
static_assert(smem_bytes(kTma) <= 232448 && smem_bytes(kCodes16) <= 232448, "shared memory plan exceeds 227 KB");
static_assert((3 * kMaxStages + 5 + 2 * kCodeSlots) * 8 + 8 <= 512, "barrier block overflows");

// What a cluster is for: nothing; a split of one unit's sum over its CTAs; a
// pair of CTAs that multiply 256 f by a tile's rows together (cta_group::2).
// Each of a pair holds 128 f and half of the rows of a stage, so that a stage
// takes 32 KB instead of 48 for the same time of MMAs: less to bring from L2,
// and six stages on the way instead of four.
enum Cluster { kSingle = 0, kSplit = 1, kPair = 2 };

struct Args {
    const int32_t* offsets;
    int rows, G, N, K;
    const bf16 *f, *r;  // operands F (w, or x for dw) and R
    int64_t ldf, ldr;
    Int4 w;             // F in 4 bits
    void* out;
    int out_elem, accumulate;
    int64_t ldo;
    uint32_t* err;
    int64_t spin_ns;
    int tile_i, stages, stage_bytes, split;
    int f_copy, r_copy;    // operand copied by the feed warps: 0 no, 1 by elements, 2 by pairs
};

// Descriptor of an operand contiguous along M or N, 128-byte swizzle: lines
// of 64 elements, eight lines (of eight c) 1024 bytes apart, the next 64
// elements 64 lines on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)((BK * kLine) >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// Loads; of a pair, bar may be the other CTA's (a cluster address).
template <bool PAIR> __device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    if (PAIR) tma_load_2d_pair(dst, map, bar, x, y);
    else tma_load_2d(dst, map, bar, x, y);
}
template <bool PAIR> __device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    if (!PAIR) {
        tma_load_3d(dst, map, bar, x, y, z);
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    }
}
// Arrival at another CTA's barrier, which orders no writes for that CTA.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

struct Unit {
    int g;
    int i0, n;   // first row (dw: column of dy) of the tile, and how many
    int f0;
    int c0, c1;  // range of the sum
};

template <int OP> __device__ __forceinline__ int f_size(const Args& p) { return OP == kProductFwd ? p.N : p.K; }

template <int OP, int UF> __device__ __forceinline__ Unit unit_at(const Args& p, int u, int FB, int NB, const GroupTable& t) {
    Unit r;
    const int rt = u / FB;
    r.f0 = (u - rt * FB) * UF;
    if (OP == kProductDw) {
        r.g = rt / NB;
        r.i0 = (rt - r.g * NB) * p.tile_i;
        r.n = min(p.tile_i, p.N - r.i0);
        r.c0 = t.first[r.g];
        r.c1 = t.last[r.g];
    } else {
        r.g = find_group_smem(t.tiles, p.G, rt);
        r.i0 = t.first[r.g] + (rt - t.tiles[r.g]) * p.tile_i;
        r.n = min(p.tile_i, t.last[r.g] - r.i0);
        r.c0 = 0;
        r.c1 = OP == kProductFwd ? p.K : p.N;
    }
    return r;
}
// Blocks of the sum that this rank of a split takes: [first, last).
__device__ __forceinline__ int2 my_blocks(const Unit& u, int rank, int split) {
    const int kb = (u.c1 - u.c0 + BK - 1) / BK;
    return make_int2((int)((int64_t)kb * rank / split), (int)((int64_t)kb * (rank + 1) / split));
}

// 32 features (this warp's lanes) x 32 rows, packed two rows a word (w[j]:
// rows 2j and 2j + 1 of feature `lane`), to out rows of 64 bytes.
__device__ __forceinline__ void store_block(uint8_t* st, const uint32_t* w, bf16* out, int64_t ldo, int rows, int cols) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) *(uint32_t*)(st + j * 128 + lane * 4) = w[8 * h + j];
        __syncwarp();
        const int pr = lane >> 2, q = lane & 3, row = 16 * h + 2 * pr;  // row pair, eight features
        const uint4 a = *(const uint4*)(st + pr * 128 + q * 32), b = *(const uint4*)(st + pr * 128 + q * 32 + 16);
        const uint4 lo = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410), __byte_perm(b.x, b.y, 0x5410),
                                    __byte_perm(b.z, b.w, 0x5410));
        const uint4 hi = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632), __byte_perm(b.x, b.y, 0x7632),
                                    __byte_perm(b.z, b.w, 0x7632));
        if (q * 8 < cols) {
            if (row < rows) *(uint4*)(out + (int64_t)row * ldo + q * 8) = lo;
            if (row + 1 < rows) *(uint4*)(out + (int64_t)(row + 1) * ldo + q * 8) = hi;
        }
        __syncwarp();
    }
}

// One element or (WIDTH 2) two, or zeros.  Volatile, so that a line's loads are
// not put off until the stores of the one before have its values: with them
// free to move a product of 16027 x 1645 x 1297 took 1044 us, so 202.
template <int WIDTH> __device__ __forceinline__ uint32_t load_if(const uint16_t* p, bool in) {
    uint32_t v;
    if (WIDTH == 2)
        asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n mov.b32 %0, 0;\n @q ld.global.b32 %0, [%1];\n}\n" : "=r"(v) : "l"(p), "r"((int)in));
    else
        asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n mov.b32 %0, 0;\n @q ld.global.u16 %0, [%1];\n}\n" : "=r"(v) : "l"(p), "r"((int)in));
    return v;
}
// Lines of an operand to shared memory at dst by a group of four warps, 64 at
// a time, all of a warp's sixteen in flight.  along_c: a line is 64 c of a row,
// c_left of them the matrix's, and rows_left rows are; else 64 rows (columns
// of the tensor) of one c.  What lies outside becomes zeros.  A lane takes two
// elements of a line: MODE 2, where pairs lie on 4 bytes, with one load.
template <int MODE>
__device__ __forceinline__ void copy_lines(uint32_t dst, const bf16* src, int64_t ld, bool along_c, int lines, int rows_left, int c_left,
                                           int c16, int warp, int lane) {
    constexpr int kEach = BK / kFeedGroup;
    const uint16_t* q = (const uint16_t*)src + warp * ld + 2 * lane;
    dst += warp * kLine + ((lane & 3) << 2);
    for (int l0 = 0; l0 < lines; l0 += BK) {
        const int in = along_c ? c_left : rows_left - l0;           // elements of a line
        const int some = along_c ? rows_left - l0 : c_left;         // lines that have any
        const bool lo = 2 * lane < in, hi = 2 * lane + 1 < in;
        const uint16_t* b = q + (along_c ? l0 * ld : (int64_t)l0);
        uint32_t v[kEach], w[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j, b += kFeedGroup * ld) {
            const bool line = warp + kFeedGroup * j < some;
            v[j] = load_if<MODE>(b, line && (MODE == 2 ? hi : lo));
            w[j] = load_if<1>(MODE == 2 ? b : b + 1, line && (MODE == 2 ? lo && !hi : hi));
        }
        const int put = along_c ? lines - l0 : c16;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int l = warp + kFeedGroup * j;
            if (l >= put) continue;
            const uint32_t a = dst + (l0 + kFeedGroup * j) * kLine + (((lane >> 2) ^ (l & 7)) << 4);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(MODE == 1 ? v[j] | w[j] << 16 : v[j] | w[j]) : "memory");
        }
    }
}

// Eight codes' values, rounded to bf16 once: a choice.  The tensor cores take
// bf16 on both sides, and a value is code - zero times the scale, 12 bits with a
// bf16 scale.  In two parts, which would be exact, a product would be twice the
// MMAs and stores to shared memory, and those bound it (2047 rows, 4096 x 4096: the
// outputs are 0.0022 of their rms off 64 bits, 0.0017 from their own rounding
// alone).  Few rows, bound by the codes' bytes, multiply the codes and keep all
// bits (product_few.cu).  s: the scale's bits; TIES: it may be one of int4_on_ties.
template <int FEED, bool TIES> __device__ __forceinline__ uint4 values8(uint32_t w, __nv_bfloat162 z, uint32_t s) {
    uint32_t o[4];
    int4_pairs(w, z, o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 d = *(const __nv_bfloat162*)&o[j];
        __nv_bfloat162 v;
        if (FEED == kCodes16) {
            const uint32_t ss = s * 0x10001u;
            v = __hmul2(d, *(const __nv_bfloat162*)&ss);
        } else {
            const float2 x = __bfloat1622float2(d);
            const float f = __uint_as_float(s);
            v = TIES ? __floats2bfloat162_rn(int4_value(x.x, f), int4_value(x.y, f)) : __floats2bfloat162_rn(x.x * f, x.y * f);
        }
        o[j] = *(const uint32_t*)&v;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The line of 64 codes in q, two halves of one scale and zero point each; swap:
// which 16 bytes of the line the swizzle puts first.
template <int FEED, bool TIES>
__device__ __forceinline__ void put_values(uint32_t row, int swap, const uint4 (&q)[2], const uint32_t (&zp)[2], const uint32_t (&sc)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {q[h].x, q[h].y, q[h].z, q[h].w};
        const __nv_bfloat162 z = int4_zero((int)zp[h]);
#pragma unroll
        for (int j = 0; j < 4; ++j) st_shared16(row + (((4 * h + j) ^ swap) << 4), values8<FEED, TIES>(w[j], z, sc[h]));
    }
}

template <int OP, int FEED, int CL>
__global__ void __launch_bounds__(threads_for(FEED), 1)
    product_tc_kernel(const __grid_constant__ CUtensorMap tm_f, const __grid_constant__ CUtensorMap tm_f16,
                      const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_r16, const Args p) {
    constexpr bool kFAlongC = OP == kProductFwd, kRAlongC = OP != kProductDw;
    constexpr int kEpi = epi_warps(FEED), kHalves = kEpi / 4;  // warps for each lane quarter
    constexpr bool SPLIT = CL == kSplit, PAIR = CL == kPair;
    static_assert(!PAIR || FEED == kTma, "pairs load by TMA alone");
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = (uint64_t*)(smem + kOffBar);
    const int S = p.stages;
    const uint32_t smem0 = smem_u32(smem);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kMaxStages);
    const uint32_t tfull0 = smem_u32(bars + 2 * kMaxStages), tempty0 = tfull0 + 16, drain = tfull0 + 32;
    const uint32_t tail0 = drain + 8, cfull0 = tail0 + 8 * kMaxStages, cempty0 = cfull0 + 8 * kCodeSlots;  // codes
    uint32_t* tmem_slot = (uint32_t*)(bars + 3 * kMaxStages + 5 + 2 * kCodeSlots);
    volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
    GroupTable& tab = *(GroupTable*)(smem + off_table(FEED));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool f_tma = FEED == kTma || (FEED == kCopy && !p.f_copy), r_tma = FEED == kTma || !p.r_copy;
    if (threadIdx.x == 0) {
        // (pair, dw: the leader's are told by the other CTA's loads as well)
        const int feeders = (f_tma || r_tma ? 1 : 0) + (FEED == kTma ? 0 : kFeedGroup) + (PAIR && OP == kProductDw ? 1 : 0);
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, feeders);
            mbar_init(empty0 + 8 * s, 1);
            mbar_init(tail0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, PAIR ? 2 * kEpi : kEpi);
        }
        for (int s = 0; s < kCodeSlots; ++s) {
            mbar_init(cfull0 + 8 * s, 1);
            mbar_init(cempty0 + 8 * s, kFeedGroup);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (PAIR && warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();  // what an earlier kernel wrote
    if (warp == 2) group_table(tab, p.offsets, p.G, p.rows, OP == kProductDw ? kMaxI : p.tile_i);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // both CTAs' barriers and tensor memory exist before either uses the other's
    tc_fence_after();
    pdl_release();  // (once tensor memory is ours)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    constexpr int kUnitF = PAIR ? 2 * BF : BF;
    const int F = f_size<OP>(p), FB = (F + kUnitF - 1) / kUnitF, NB = (p.N + p.tile_i - 1) / p.tile_i;
    // (a split has a cluster for each unit that ascending offsets can give)
    const int most = SPLIT ? (int)gridDim.x / p.split : 0x7FFFFFFF;
    const int units = min((OP == kProductDw ? p.G * NB : tab.tiles[p.G]) * FB, most);
    // Units of this CTA: u0, u0 + step, ...  Split: a cluster takes one unit or none.
    const int rank = SPLIT ? (int)cluster_rank() : 0, cl = SPLIT ? p.split : 1;
    const int crank = PAIR ? (int)cluster_rank() : 0, per = PAIR ? 2 : cl;  // of a pair: 0 leads (issues the MMAs)
    const int u0 = (int)blockIdx.x / per, step = (int)gridDim.x / per;
    const int64_t lim = p.spin_ns;
    // A wait for a unit's last block takes as long as the unit's sum, and that of dw goes over all rows of a group: 2 s, the
    // limit of a block's wait, are 220 million rows of 9 x 9 (0.6 us a block; up to 1.6 where wide operands are copied).
    // So it has ten times that for each of its blocks beside.
    auto unit_lim = [&](int2 kb) { return lim + (int64_t)(kb.y - kb.x) * 16000; };
    auto wait = [&](uint32_t bar, uint32_t parity, int where, int64_t limit) {
        const bool ok = warp_wait(bar, parity, limit, abort_flag, p.err, where);
        if (PAIR && !ok && elect_one()) raise_abort_pair(abort_flag, (uint32_t)crank);
        return ok;
    };
    auto at_unit = [&](int u) {
        Unit un = unit_at<OP, kUnitF>(p, u, FB, NB, tab);
        if (PAIR) un.f0 += crank * BF;
        return un;
    };

    if (warp == 0) {
        // -------------------------------------------------- TMA producer
        if (f_tma || r_tma) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = u0; u < units && ok; u += step) {
                const Unit un = at_unit(u);
                const int2 kb = my_blocks(un, rank, cl);
                // sixteens of i that this CTA loads, from i0 on
                const int n16 = __shfl_sync(0xffffffffu, PAIR ? (un.n + 31) >> 5 : (un.n + 15) >> 4, 0), slabs = (n16 + 3) >> 2;
                const int i0 = __shfl_sync(0xffffffffu, un.i0 + crank * n16 * 16, 0), f0 = __shfl_sync(0xffffffffu, un.f0, 0);
                const int g = __shfl_sync(0xffffffffu, un.g, 0);
                for (int k = kb.x; k < kb.y; ++k) {
                    ok = wait(empty0 + 8 * stage, phase ^ 1, 61, lim);
                    if (!ok) break;
                    const int c = __shfl_sync(0xffffffffu, un.c0 + k * BK, 0);
                    // dw: sixteens of this block's rows; the others read whole blocks, zeros past the edge
                    const int c16 = OP == kProductDw ? __shfl_sync(0xffffffffu, min(4, (un.c1 - c + 15) >> 4), 0) : 4;
                    if (elect_one()) {
                        uint32_t fb = full0 + 8 * stage;
                        const uint32_t fs = smem0 + stage * p.stage_bytes, rs = fs + kFBytes;
                        // boxes of 64 rows, then of 16 (of three, 64 once more: what they bring is ignored)
                        const int n64 = (n16 + 1) >> 2, rows = max(n16, 4 * n64) * 16;
                        const int rlines = kRAlongC ? rows : slabs * c16 * 16, flines = kFAlongC ? BF : 2 * c16 * 16;
                        const uint32_t bytes = (f_tma ? flines * kLine : 0) + (r_tma ? rlines * kLine : 0);
                        if (!PAIR) {
                            mbar_expect_tx(fb, bytes);
                        } else {
                            // Both CTAs' loads count at the leader.  dw's last block, where zeros have to be written
                            // over lines: the other's at its own barrier, and its MMA warp tells the leader.
                            const bool ragged = OP == kProductDw && un.c1 - c < BK && ((un.c1 - c) & 15);
                            if (crank == 0) {
                                mbar_expect_tx(fb, ragged ? bytes : 2 * bytes);
                            } else if (ragged) {
                                fb = tail0 + 8 * stage;
                                mbar_expect_tx(fb, bytes);
                            } else if (OP == kProductDw) {
                                mbar_arrive_remote(mapa_shared(fb, 0));
                            }
                            if (!ragged) fb = mapa_shared(fb, 0);
                            else fb = mapa_shared(fb, (uint32_t)crank);
                        }
                        if (f_tma) {
                            if (OP == kProductFwd) {
                                load3<PAIR>(fs, &tm_f, fb, c, f0, g);
                            } else if (OP == kProductDx) {
                                load3<PAIR>(fs, &tm_f, fb, f0, c, g);
                                load3<PAIR>(fs + BK * kLine, &tm_f, fb, f0 + 64, c, g);
                            } else {
                                for (int s = 0; s < 2; ++s) {
                                    if (c16 == 4) load2<PAIR>(fs + s * BK * kLine, &tm_f, fb, f0 + 64 * s, c);
                                    else
                                        for (int j = 0; j < c16; ++j)
                                            load2<PAIR>(fs + s * BK * kLine + j * 16 * kLine, &tm_f16, fb, f0 + 64 * s, c + 16 * j);
                                }
                            }
                        }
                        if (r_tma) {
                            if (kRAlongC) {
                                for (int j = 0; j < n64; ++j) load2<PAIR>(rs + j * 64 * kLine, &tm_r, fb, c, i0 + j * 64);
                                for (int j = 4 * n64; j < n16; ++j) load2<PAIR>(rs + j * 16 * kLine, &tm_r16, fb, c, i0 + j * 16);
                            } else {
                                for (int s = 0; s < slabs; ++s) {
                                    if (c16 == 4) load2<PAIR>(rs + s * BK * kLine, &tm_r, fb, i0 + 64 * s, c);
                                    else
                                        for (int j = 0; j < c16; ++j)
                                            load2<PAIR>(rs + s * BK * kLine + j * 16 * kLine, &tm_r16, fb, i0 + 64 * s, c + 16 * j);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) sleep_ns(200000);  // copies already issued land before the CTA leaves
        }
    } else if (warp == 1) {
        // --------------------------------------------------- MMA issuer
        // dw: zeros over the lines of a last block's last sixteen that lie past the end.
        auto clear = [&](uint32_t fs, int left, int rslabs) {
            const int slabs = 2 + rslabs, each = (16 - (left & 15)) * 8;  // 16-byte pieces of a slab
            for (int e = lane; e < slabs * each; e += 32) {
                const int s = e / each;
                st_shared16(fs + s * BK * kLine + left * kLine + (e - s * each) * 16, make_uint4(0, 0, 0, 0));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        };
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0, tail_phase = 0;  // (a bit a stage)
        bool ok = true;
        for (int u = u0; u < units && ok; u += step) {
            const Unit un = at_unit(u);
            const int2 kb = my_blocks(un, rank, cl);
            if (kb.x == kb.y) continue;  // nothing to sum: the epilogue knows
            const int n = __shfl_sync(0xffffffffu, PAIR ? (un.n + 31) & ~31 : (un.n + 15) & ~15, 0);
            const int rslabs = ((PAIR ? n / 2 : n) + 63) / 64;
            if (PAIR && crank) {  // only the other CTA's last block of dw is of concern here
                if (OP != kProductDw) break;
                const int left = (un.c1 - un.c0) & (BK - 1);
                stage = (stage + kb.y - 1) % S;
                if (left & 15) {
                    ok = wait(tail0 + 8 * stage, tail_phase >> stage & 1, 66, unit_lim(kb));
                    if (!ok) break;
                    tail_phase ^= 1u << stage;
                    clear(smem0 + stage * p.stage_bytes, left, rslabs);
                    if (elect_one()) mbar_arrive_cluster(mapa_shared(full0 + 8 * stage, 0));
                    __syncwarp();
                }
                stage = (stage + 1) % S;
                continue;
            }
            const uint32_t id = idesc_bf16(PAIR ? 2 * BF : BF, n) | (kFAlongC ? 0u : 1u << 15) | (kRAlongC ? 0u : 1u << 16);
            ok = wait(tempty0 + 8 * acc, acc_phase ^ 1, 62, lim);
            if (!ok) break;
            const uint32_t d = tmem + acc * kMaxI;
            for (int k = kb.x; k < kb.y; ++k) {
                ok = wait(full0 + 8 * stage, phase, 63, lim);
                if (!ok) break;
                const uint32_t fs = smem0 + stage * p.stage_bytes, rs = fs + kFBytes;
                const int left = un.c1 - un.c0 - k * BK;
                const int steps = __shfl_sync(0xffffffffu, min(4, (left + 15) >> 4), 0);
                if (OP == kProductDw && left < BK && (left & 15)) {
                    if (PAIR) asm volatile("fence.acq_rel.cluster;" ::: "memory");  // the other CTA's zeros
                    clear(fs, left, rslabs);
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t fd = kFAlongC ? umma_desc(fs) : desc_mn(fs), rd = kRAlongC ? umma_desc(rs) : desc_mn(rs);
                    constexpr uint64_t fstep = (kFAlongC ? 32 : 16 * kLine) >> 4, rstep = (kRAlongC ? 32 : 16 * kLine) >> 4;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        if (PAIR) umma_bf16_pair(d, fd + kk * fstep, rd + kk * rstep, id, k != kb.x || kk != 0);
                        else umma_bf16(d, fd + kk * fstep, rd + kk * rstep, id, k != kb.x || kk != 0);
                    }
                    if (PAIR) umma_commit_pair(empty0 + 8 * stage);
                    else umma_commit(empty0 + 8 * stage);
                    if (k + 1 == kb.y) {
                        if (PAIR) umma_commit_pair(tfull0 + 8 * acc);
                        else umma_commit(tfull0 + 8 * acc);
                    }
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
        // everything issued is done before tensor memory is freed
        if (!PAIR || crank == 0) {
            if (elect_one()) {
                if (PAIR) umma_commit_pair(drain);
                else umma_commit(drain);
            }
            __syncwarp();
            volatile int never = 0;
            mbar_wait(drain, 0, 1000000000LL, &never);
        }
    } else if (FEED >= kCodes16 && warp == threads_for(FEED) / 32 - 1) {
        // ------------------------------------------------- loads of codes
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0; u < units && ok; u += step) {
            const Unit un = at_unit(u);
            const int2 kb = my_blocks(un, rank, cl);
            const int row = __shfl_sync(0xffffffffu, un.g * p.N + un.f0, 0);
            for (int k = kb.x; k < kb.y; ++k) {
                ok = warp_wait(cempty0 + 8 * slot, phase ^ 1, lim, abort_flag, p.err, 65);
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect_tx(cfull0 + 8 * slot, kCodeBytes);
                    tma_load_2d(smem0 + kOffCodes + slot * kCodeBytes, &tm_f, cfull0 + 8 * slot, k * (BK / 2), row);
                }
                __syncwarp();
                if (++slot == kCodeSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) sleep_ns(200000);
    } else if (FEED != kTma && warp >= 2 + kEpi) {
        // -------------------------------------------- copied or coded operands
        // Groups of four warps fill stages in turn, so that one's latency (a
        // wait, loads, a proxy fence, an arrival) passes beside the others'.
        constexpr int kGroups = feed_groups(FEED);
        const int fw = (warp - 2 - kEpi) & (kFeedGroup - 1), mine = (warp - 2 - kEpi) / kFeedGroup;
        const int t = (threadIdx.x - 32 * (2 + kEpi)) & (32 * kFeedGroup - 1);
        int64_t done = 0;  // blocks of the units before
        uint32_t turn = 0;  // this group's
        bool ok = true;
        for (int u = u0; u < units && ok; u += step) {
            const Unit un = at_unit(u);
            const int2 kb = my_blocks(un, rank, cl);
            // codes: thread t takes the line (64 codes, a scale or two) of feature t
            const int64_t wrow = (int64_t)un.g * p.N + un.f0 + t;
            const bool in = un.f0 + t < p.N;
            const int nbk = (p.K + p.w.group - 1) / p.w.group;
            uint32_t sc[2], zp[2];  // as loaded: converting would wait for the load
            auto fetch = [&](int k) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = k * BK + 32 * h;
                    if (h && p.w.group > 32 && c < p.K) {  // one for both halves
                        sc[1] = sc[0];
                        zp[1] = zp[0];
                        continue;
                    }
                    sc[h] = zp[h] = 0;  // (past the edge)
                    if (!in || k >= kb.y || c >= p.K) continue;
                    const int64_t at = wrow * nbk + c / p.w.group;
                    sc[h] = FEED == kCodes16 ? ((const uint16_t*)p.w.scales)[at] : ((const uint32_t*)p.w.scales)[at];
                    zp[h] = 8;
                    if (p.w.zeros) zp[h] = p.w.zeros[at];
                }
            };
            const int skip = (mine - (int)(done % kGroups) + kGroups) % kGroups;  // to this group's first block
            const int64_t at0 = done + skip;
            int stage = (int)(at0 % S);
            uint32_t phase = (uint32_t)(at0 / S) & 1;
            done += kb.y - kb.x;
            if (FEED >= kCodes16) fetch(kb.x + skip);
            for (int k = kb.x + skip; k < kb.y; k += kGroups) {
                uint4 q[2];
                if (FEED >= kCodes16) {
                    static_assert(FEED < kCodes16 || kGroups == kCodeSlots, "a group reads one slot");
                    ok = __all_sync(0xffffffffu, mbar_wait(cfull0 + 8 * mine, turn & 1, lim, abort_flag));
                    if (!ok) break;
                    ++turn;
                    // 32 bytes a line, their halves exchanged by TMA in every other four lines
                    const uint8_t* line = smem + kOffCodes + mine * kCodeBytes + t * 32;
                    q[0] = *(const uint4*)(line + ((t >> 2) & 1) * 16);
                    q[1] = *(const uint4*)(line + (~(t >> 2) & 1) * 16);
                }
                bool ties = false;
                if (FEED == kCodes32)
                    ties = __any_sync(0xffffffffu, int4_on_ties(__uint_as_float(sc[0])) || (p.w.group == 32 && int4_on_ties(__uint_as_float(sc[1]))));
                ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * stage, phase ^ 1, lim, abort_flag));
                if (!ok) break;
                const int c = un.c0 + k * BK, left = un.c1 - c, c16 = min(4, (left + 15) >> 4) * 16;
                const uint32_t fs = smem0 + stage * p.stage_bytes, rs = fs + kFBytes;
                if (FEED >= kCodes16) {
                    const uint32_t row = fs + t * kLine;
                    if (ties) put_values<FEED, true>(row, t & 7, q, zp, sc);
                    else put_values<FEED, false>(row, t & 7, q, zp, sc);
                    __syncwarp();
                    // Only now, when the codes have been used: an arrival does not order loads that are on their way
                    // with TMA's writes, and right behind the loads it let the next codes overwrite some.
                    if (lane == 0) mbar_arrive(cempty0 + 8 * mine);
                    fetch(k + kGroups);
                } else if (p.f_copy) {
                    const bf16* src = OP == kProductFwd   ? p.f + ((int64_t)un.g * p.N + un.f0) * p.ldf + c
                                      : OP == kProductDx ? p.f + ((int64_t)un.g * p.N + c) * p.ldf + un.f0
                                                         : p.f + (int64_t)c * p.ldf + un.f0;
                    if (p.f_copy == 2) copy_lines<2>(fs, src, p.ldf, kFAlongC, BF, F - un.f0, left, c16, fw, lane);
                    else copy_lines<1>(fs, src, p.ldf, kFAlongC, BF, F - un.f0, left, c16, fw, lane);
                }
                if (p.r_copy) {
                    const bf16* src = kRAlongC ? p.r + (int64_t)un.i0 * p.ldr + c : p.r + (int64_t)c * p.ldr + un.i0;
                    const int lines = kRAlongC ? (un.n + 15) & ~15 : ((un.n + 63) & ~63);
                    if (p.r_copy == 2) copy_lines<2>(rs, src, p.ldr, kRAlongC, lines, un.n, left, c16, fw, lane);
                    else copy_lines<1>(rs, src, p.ldr, kRAlongC, lines, un.n, left, c16, fw, lane);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(full0 + 8 * stage);
                stage += kGroups;
                if (stage >= S) {
                    stage -= S;
                    phase ^= 1;
                }
            }
        }
    }
    // ---------------------------------------------------------- epilogue
    // Lanes are f, columns i.
    const int ew = warp - 2, sub = warp & 3, half = ew >> 2;  // lane quarter, column half
    const bool epi = ew >= 0 && ew < kEpi;
    if (!SPLIT && epi) {
        uint8_t* st = smem + off_stage(FEED) + ew * kStWarp;
        const bool vec = F % 8 == 0 && p.ldo % 8 == 0 && ((uintptr_t)p.out & 15) == 0;
        const bool add = OP == kProductDw && p.accumulate;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = u0; u < units; u += step) {
            const Unit un = at_unit(u);
            const bool any = un.c1 > un.c0;
            const uint32_t taddr = tmem + acc * kMaxI + ((uint32_t)(sub * 32) << 16);
            const uint32_t te = tempty0 + 8 * acc;
            if (any) {
                const bool ok = mbar_wait(tfull0 + 8 * acc, acc_phase, unit_lim(my_blocks(un, rank, cl)), abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0 && !*abort_flag) {
                        record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 64, blockIdx.x, u);
                        *abort_flag = 1;
                        if (PAIR) raise_abort_pair(abort_flag, (uint32_t)crank);
                    }
                    break;
                }
                tc_fence_after();
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            } else if (add) {
                continue;
            }
            const int f = un.f0 + sub * 32, cols = F - f;  // this warp's f inside the matrix
            const int64_t row0 = OP == kProductDw ? (int64_t)un.g * p.N + un.i0 : (int64_t)un.i0;
            // this warp's 32-row blocks: of two halves 0, 2, 4, 6 or 1, 3, 5, 7
#pragma unroll 1
            for (int c = half * 32; c < un.n; c += 32 * kHalves) {
                uint32_t v[32];
                if (any) {
                    tmem_ld32(taddr + c, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0;
                }
                const int rows = un.n - c;
                const int64_t at = (row0 + c) * p.ldo + f;
                if (p.out_elem == kF32) {
                    float* o = (float*)p.out + at + lane;
                    if (lane < cols) {
                        if (add) {
                            const float* q = o;
#pragma unroll
                            for (int j = 0; j < 32; ++j, q += p.ldo)
                                if (j < rows) v[j] = __float_as_uint(*q + __uint_as_float(v[j]));
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j, o += p.ldo)
                            if (j < rows) *o = __uint_as_float(v[j]);
                    }
                } else if (vec && !add) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                        pk[j] = *(const uint32_t*)&h;
                    }
                    store_block(st, pk, (bf16*)p.out + at, p.ldo, rows, cols);
                } else if (lane < cols) {
                    bf16* o = (bf16*)p.out + at + lane;
                    if (add) {
                        const bf16* q = o;
#pragma unroll
                        for (int j = 0; j < 32; ++j, q += p.ldo)
                            if (j < rows) v[j] = __float_as_uint(to_f32(*q) + __uint_as_float(v[j]));
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j, o += p.ldo)
                        if (j < rows) *o = __float2bfloat16_rn(__uint_as_float(v[j]));
                }
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    // (what this orders are loads from tensor memory, which are complete; a release for the cluster
                    // would wait for the stores above)
                    if (PAIR) mbar_arrive_remote(mapa_shared(te, 0));
                    else mbar_arrive(te);
                }
            }
        }
    }
    if (SPLIT) {
        // One unit a cluster.  Rank q sums rows q, q + split, ... of the tile
        // in blocks of four: every rank sends it its partial sums, [rank][slot
        // of four rows][feature], into the ring, which is idle by then.
        __syncwarp();
        cluster_sync();  // every CTA's loads and MMAs are done
        const bool has = u0 < units;
        const Unit un = has ? at_unit(u0) : Unit{};
        const int2 kb = my_blocks(un, rank, cl);
        const int quads = (un.n + 3) >> 2, slots = (quads + cl - 1) / cl;  // four-row slots, of each rank
        const uint32_t part = (uint32_t)(slots * BF * 16);                 // bytes a rank sends another
        if (has && epi) {
            tc_fence_after();  // the accumulator was committed before the barrier
            const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16);
            const uint32_t mine = smem0 + rank * part + (uint32_t)((sub * 32 + lane) * 16);
#pragma unroll 1
            for (int c = half * 16; c < un.n; c += 16 * kHalves) {
                uint32_t v[16];
                if (kb.x < kb.y) {
                    tmem_ld16(taddr + c, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int qd = c / 4 + j;
                    if (qd < quads) {
                        const float4 x = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]), __uint_as_float(v[4 * j + 2]),
                                                     __uint_as_float(v[4 * j + 3]));
                        st_cluster(mapa_shared(mine + (uint32_t)(qd / cl) * BF * 16, (uint32_t)(qd % cl)), x);
                    }
                }
            }
            tc_fence_before();
        }
        __syncwarp();
        cluster_sync();
        const bool add = OP == kProductDw && p.accumulate;
        if (has && epi && !(add && un.c0 == un.c1)) {
            const int e = threadIdx.x - 64, feat = un.f0 + (e & 127);
            const int64_t row0 = OP == kProductDw ? (int64_t)un.g * p.N + un.i0 : (int64_t)un.i0;
            for (int i = e >> 7; i < slots; i += kHalves) {
                const int row = (i * cl + rank) * 4;
                if (row >= un.n) break;
                float s[4] = {0, 0, 0, 0};
                for (int k = 0; k < cl; ++k) {
                    const float4 x = *(const float4*)(smem + k * part + i * BF * 16 + (e & 127) * 16);
                    s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
                }
                if (feat < F) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (row + j < un.n) {
                            const int64_t at = (row0 + row + j) * p.ldo + feat;
                            if (p.out_elem == kF32) {
                                float* o = (float*)p.out + at;
                                *o = add ? *o + s[j] : s[j];
                            } else {
                                bf16* o = (bf16*)p.out + at;
                                *o = __float2bfloat16_rn(add ? to_f32(*o) + s[j] : s[j]);
                            }
                        }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // no arrival or MMA of the other CTA is on its way here
    tc_fence_after();
    if (PAIR) {
        if (warp == 1) tmem_dealloc_pair(tmem, 512);
        return;
    }
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// bf16 [d2][d1][d0] (d2 = 0: two dimensions), boxes of a 128-byte line by box1.
bool line_map(CUtensorMap* m, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t ld, int box1) {
    if (((uintptr_t)base & 15) || ld % 8) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2}, strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(ld * d1) * 2};
    const cuuint32_t box[3] = {BK, (cuuint32_t)box1, 1}, es[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Codes, boxes of 32 bytes of BF rows.
bool code_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes) {
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {BK / 2, BF}, es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// How the feed warps would copy an operand.
int copy_mode(const void* base, int64_t ld) { return ((uintptr_t)base & 3) == 0 && ld % 2 == 0 ? 2 : 1; }

struct Maps {
    CUtensorMap f, f16, r, r16;
};

template <int OP, int FEED, int CL> cudaError_t launch(const Maps& m, const Args& a, int grid, cudaStream_t s) {
    cudaError_t e = ensure_smem_attr((const void*)product_tc_kernel<OP, FEED, CL>, smem_bytes(FEED));
    if (e != cudaSuccess) return e;
    e = launch_kernel(product_tc_kernel<OP, FEED, CL>, dim3(grid), dim3(threads_for(FEED)), smem_bytes(FEED), s,
                      CL == kSplit ? a.split : CL == kPair ? 2 : 1, m.f, m.f16, m.r, m.r16, a);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Tiles, stages, split and grid; the launch.
template <int OP> cudaError_t plan_and_launch(const Maps& m, Args& a, int feed, int num_sms, cudaStream_t s) {
    // i of a tile: as many as the groups fill (F is read once per tile), fewer
    // where they do not, for more stages in flight.
    const int64_t avg = OP == kProductDw ? a.N : cdiv(a.rows, a.G);
    const int F = OP == kProductFwd ? a.N : a.K;
    const int64_t fb = cdiv(F, BF);
    auto units = [&](int ti) {  // at most
        return (OP == kProductDw ? a.G * cdiv(a.N, ti) : cdiv(a.rows, ti) + std::min(a.G - 1, a.rows)) * fb;
    };
    a.tile_i = avg > 128 ? 256 : avg > (OP == kProductDw ? 64 : 32) ? 128 : 64;
    while (a.tile_i > 64 && units(a.tile_i) * 2 <= num_sms) a.tile_i /= 2;  // (few tiles: smaller ones on more SMs)
    if (OP != kProductDw && a.G == 1 && a.tile_i == 256) {
        // One matrix: as many tiles as the same number of rounds holds, of equal size.
        const int64_t tiles = cdiv(units(256), num_sms) * num_sms / fb;
        if (tiles > 0) a.tile_i = (int)std::min<int64_t>(256, cdiv(cdiv(a.rows, tiles), 16) * 16);
    }
    // dw: a group's rows, at most (an average would leave the largest to one CTA)
    const int64_t kb = cdiv(OP == kProductFwd ? a.K : OP == kProductDx ? a.N : a.rows, BK);
    a.split = 1;
    while (a.split < kMaxSplit && units(a.tile_i) * a.split * 2 <= num_sms && kb >= 4 * a.split) a.split *= 2;
    // Pairs: where they leave no more than one in eight of the f tiles empty, and there is a unit for each.  dw
    // with few rows a group is bound by its epilogue, which two CTAs wait for: 64 groups of 256 rows, 1024 x 4096,
    // fp32 dw 193 us (pairs 238), of 512 rows 296 (239); bf16 dw, 256 rows 138 (132).
    const bool pair = feed == kTma && a.split == 1 && (fb % 2 == 0 || fb >= 8) && units(a.tile_i) >= num_sms &&
                      (OP != kProductDw || (a.tile_i >= 128 && a.rows >= (a.out_elem == kF32 ? 384 : 128) * (int64_t)a.G));
    a.stage_bytes = kFBytes + (int)cdiv(a.tile_i, 64) * 64 * BK * 2 / (pair ? 2 : 1);
    a.stages = std::min(kMaxStages, kRing / a.stage_bytes);
    if (pair) {
        const int64_t n = units(a.tile_i) / fb * cdiv(fb, 2);
        return launch<OP, kTma, kPair>(m, a, 2 * (int)std::min<int64_t>(n, num_sms / 2), s);
    }
    const int grid = a.split > 1 ? (int)units(a.tile_i) * a.split : (int)std::min<int64_t>(units(a.tile_i), num_sms);
#define MOE_PTC(FEED) (a.split > 1 ? launch<OP, FEED, kSplit>(m, a, grid, s) : launch<OP, FEED, kSingle>(m, a, grid, s))
    if (feed == kTma) return MOE_PTC(kTma);
    if constexpr (OP == kProductFwd) {
        if (feed == kCodes16) return MOE_PTC(kCodes16);
        if (feed == kCodes32) return MOE_PTC(kCodes32);
    }
    return MOE_PTC(kCopy);
#undef MOE_PTC
}

}  // namespace ptc

cudaError_t launch_product_tc(const GroupProduct& g, int num_sms, cudaStream_t stream) {
    using namespace ptc;
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    Maps m = {};
    Args a = {};
    a.offsets = g.offsets;
    a.rows = g.rows;
    a.G = g.G;
    a.N = g.N;
    a.K = g.K;
    a.f = (const bf16*)g.b;
    a.r = (const bf16*)g.a;
    a.ldf = g.op == kProductDw ? g.ldb : g.K;
    a.ldr = g.lda;
    a.out = g.out;
    a.out_elem = g.out_elem;
    a.accumulate = g.accumulate;
    a.ldo = g.ldo;
    a.err = g.err;
    a.spin_ns = g.spin_ns;
    const int64_t r0 = g.op == kProductFwd ? g.K : g.N;  // columns of R
    // one row: its stride is of no account, and must not keep TMA from it
    if (g.rows == 1) {
        a.ldr = cdiv(r0, 8) * 8;
        if (g.op == kProductDw) a.ldf = cdiv(g.K, 8) * 8;
    }
    // (no rows, dw: the maps are not read from, only zeros are written)
    if (g.rows == 0) {
        a.f_copy = a.r_copy = 1;
    } else {
        if (g.op == kProductDw) {
            if (!line_map(&m.f, g.b, g.K, g.rows, 0, a.ldf, 64) || !line_map(&m.f16, g.b, g.K, g.rows, 0, a.ldf, 16))
                a.f_copy = copy_mode(g.b, a.ldf);
        } else if (!line_map(&m.f, g.b, g.K, g.N, g.G, g.K, g.op == kProductFwd ? BF : 64)) {
            a.f_copy = copy_mode(g.b, g.K);
        }
        if (!line_map(&m.r, g.a, r0, g.rows, 0, a.ldr, 64) || !line_map(&m.r16, g.a, r0, g.rows, 0, a.ldr, 16))
            a.r_copy = copy_mode(g.a, a.ldr);
    }
    const int feed = a.f_copy || a.r_copy ? kCopy : kTma;
    if (g.op == kProductFwd) return plan_and_launch<kProductFwd>(m, a, feed, num_sms, stream);
    if (g.op == kProductDx) return plan_and_launch<kProductDx>(m, a, feed, num_sms, stream);
    return plan_and_launch<kProductDw>(m, a, feed, num_sms, stream);
}

cudaError_t launch_int4_tc(const Int4Product& g, int num_sms, cudaStream_t stream) {
    using namespace ptc;
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    Maps m = {};
    Args a = {};
    a.offsets = g.offsets;
    a.rows = g.rows;
    a.G = g.G;
    a.N = g.N;
    a.K = g.K;
    a.w = g.w;
    a.r = (const bf16*)g.x;
    a.ldr = g.rows == 1 ? g.K : g.ldx;
    a.out = g.out;
    a.out_elem = g.out_elem;
    a.ldo = g.ldo;
    a.err = g.err;
    a.spin_ns = g.spin_ns;
    if (!code_map(&m.f, g.w.codes, (int64_t)g.G * g.N, g.K / 2)) return cudaErrorNotSupported;
    if (!line_map(&m.r, g.x, g.K, g.rows, 0, a.ldr, 64) || !line_map(&m.r16, g.x, g.K, g.rows, 0, a.ldr, 16)) a.r_copy = copy_mode(g.x, a.ldr);
    return plan_and_launch<kProductFwd>(m, a, g.w.scale_elem == kF32 ? kCodes32 : kCodes16, num_sms, stream);
}

}  // namespace moe

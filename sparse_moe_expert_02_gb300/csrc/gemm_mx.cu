// Product of two microscaled 4-bit matrices (moe_mx_gemm), dense or grouped:
//   out[r][n] = sum_k a[r][k] * b_g[n][k]   for the rows r of group g.
//
// tcgen05.mma kind::mxf4 takes both operands as E2M1 codes and multiplies
// each 32-column block by the product of its two E8M0 scales itself, so the
// kernel feeds it what memory holds.  The weights are the MMA's M side (128
// output features a tile) and the rows its N side, rounded up to 16, so a
// group of a few rows costs tensor time for a few rows.  256 columns of K a
// stage (a 128-byte swizzled line per row: 16 KB of weights and up to 32 KB
// of rows); the rows of a tile, and with them the stages in the ring, are
// chosen by the launcher from the rows a group has on average.
//
// The scales' home is tensor memory, in chunks of 128 rows x 4 blocks: lane =
// row % 32, word = row / 32, byte = block, which is not how rows of scale
// bytes lie in memory; four warps read the scale bytes (two stages of a row a
// load, a weight row and two rows a thread, two loads ahead), write them to
// shared memory in that order, and the MMA thread copies them on with
// tcgen05.cp ahead of their MMAs.  Six slots of scales (at most as many as
// stages), in shared and in tensor memory: a slot's way from the MMAs that
// free it to those that use it again takes some 1200 cycles.
//
// Measured: 8192 x 4096 x 4096 61 us (4.5 PFLOP/s) under the power limit.  Of
// the MMA warp's 106,000 cycles (seven tiles; the mean is 6.7) 37,000 are waits
// for a stage's operands and scales, 5,000 for an accumulator, the rest issue,
// with 57,000 the MMAs' own.  64 ragged groups of 4001 rows, 1024 x 4096
// weights, 36 us (150 MB: 22 at the copy bandwidth): 18,000 of 51,000 cycles
// are waits for stages, and the CTAs with five units instead of four take
// 63,000.  7 rows, 4096 x 4096, 5.8 us, latency.
//
// 448 threads: warp 0 TMA, warp 1 tensor memory + MMA, warps 2-5 scales,
// warps 6-13 epilogue (two per lane quarter, half of the tile's rows each).
// Tiles of up to 128 rows have two accumulators; one of 256 rows leaves no
// room for a second beside the scales, so the epilogue packs its columns into
// registers, gives the accumulator back, and stores while the next tile's
// MMAs run.
//
// Few tiles (a few rows against one matrix: N / 128 of them): the K range is
// split over a cluster's CTAs, which exchange slices of their partial tiles
// through distributed shared memory and add them in rank order, so the
// result does not vary.
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu
}
namespace mxg {

using namespace tc;

constexpr int BF = 128;                        // features of a tile (MMA M)
constexpr int kMaxRows = 256;                  // rows of a tile at most (MMA N)
constexpr int kKB = 128;                       // bytes of K a stage: 256 codes
constexpr int kBlk = 2 * kKB / kMxBlock;       // 8 scale bytes of a row
constexpr int kMaxStages = 8;
constexpr int kWBytes = BF * kKB;
constexpr int kSfSlots = 6;
constexpr int kSfChunk = 512;                  // 128 rows x 4 blocks
constexpr int kSfBytes = (BF + kMaxRows) / 128 * 2 * kSfChunk;
constexpr int kScaleWarps = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kScaleWarps + kEpiWarps);
constexpr int kAccCols = 256, kSfCols = kSfBytes / 128;  // tensor-memory columns (128 lanes x 4 B; scales repeat per quarter)
constexpr int kMaxG = 1025;
constexpr int kMaxSplit = 8;
constexpr int kAhead = 2;                      // scale loads in flight, of two stages each
// shared memory: ring, then (at kOffSf) scales, epilogue staging, barriers, the groups' tile prefix and first rows
constexpr int kRing = 4 * (kWBytes + kMaxRows * kKB);
constexpr int kOffSf = kRing;
constexpr int kOffStage = kOffSf + kSfSlots * kSfBytes;
constexpr int kStWarp = 8 * 32 * 4;            // 8 row pairs x 32 features, two bf16 a word
constexpr int kOffBar = kOffStage + kEpiWarps * kStWarp;
constexpr int kOffTab = kOffBar + 256;
constexpr int kSmem = kOffTab + 2 * (kMaxG + 1) * 4;
static_assert(kSmem <= 232448, "shared memory plan exceeds 227 KB");
static_assert(kAccCols + kSfSlots * kSfCols <= 512, "tensor memory plan");
static_assert((2 * kMaxStages + 5) * 8 + 8 <= 256, "barrier block overflows");

// Instruction descriptor of kind::mxf4: E2M1 operands, both K-major, E8M0
// scales, n rows; sf: which half of the scale words (0 or 2).
__device__ __forceinline__ uint32_t idesc(int n, int sf) {
    return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(BF >> 4) << 24) |
           ((uint32_t)sf << 29);
}
__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
// One chunk of scales, shared memory to tensor memory (all four quarters):
// 32 rows of 16 bytes, eight-row groups 128 bytes apart, no swizzle.
__device__ __forceinline__ void copy_sf(uint32_t tmem, uint32_t saddr) {
    const uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

struct Plan {
    int tile_rows;  // rows of a tile: 16 .. 256
    int stages, stage_bytes;
    int accs;       // accumulators: 1 or 2
    int split;      // CTAs of a cluster that share a tile's K
};

struct Unit {
    int g, row0, rows, f0;  // group, first row of the tile, its rows, first feature
};
// pre: prefix of the groups' row tiles, then each group's first row; in
// shared memory: the offsets themselves are some 1000 cycles away, which the
// MMA warp would wait for at every tile.
__device__ __forceinline__ Unit unit_at(const MxGemm& p, const Plan& q, int u, int FB, const int32_t* pre) {
    Unit r;
    const int rt = u / FB;
    r.f0 = (u - rt * FB) * BF;
    r.g = 0;
    int lo = 0, hi = p.rows, t = rt;
    if (p.offsets) {
        r.g = find_group_smem(pre, p.G, rt);
        t = rt - pre[r.g];
        lo = pre[kMaxG + 1 + r.g];
        hi = pre[kMaxG + 2 + r.g];  // above lo where the group has a tile
    }
    r.row0 = lo + t * q.tile_rows;
    r.rows = min(q.tile_rows, hi - r.row0);
    return r;
}

// The sixteen scale bytes of a row from block b0, two stages' worth (blocks
// past the row's end: scale 1; their codes are zeros).  VEC: bytes that rows
// are aligned to.
template <int VEC> __device__ __forceinline__ uint4 load_scales(const uint8_t* row, int b0, int blocks) {
    uint32_t w[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if constexpr (VEC == 16) {
        return b0 < blocks ? *(const uint4*)(row + b0) : make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (VEC == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (b0 + 4 * j < blocks) w[j] = *(const uint32_t*)(row + b0 + 4 * j);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (b0 + i < blocks) w[i / 4] = (w[i / 4] & ~(255u << (8 * (i & 3)))) | (uint32_t)row[b0 + i] << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 features (this warp's lanes) x 32 rows, packed two rows a word (w[j]:
// rows 2j and 2j + 1 of feature `lane`), to out rows of 64 bytes.  rows,
// cols: what is inside the tile; vec: 16-byte stores are possible.
__device__ __forceinline__ void store_block(uint8_t* st, const uint32_t* w, bf16* out, int64_t ldo, int rows, int cols, bool vec) {
    const int lane = threadIdx.x & 31;
    if (!vec) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h = *(const __nv_bfloat162*)&w[j];
            if (lane < cols && 2 * j < rows) out[(int64_t)(2 * j) * ldo + lane] = h.x;
            if (lane < cols && 2 * j + 1 < rows) out[(int64_t)(2 * j + 1) * ldo + lane] = h.y;
        }
        return;
    }
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

template <int VEC, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_r64,
                   const __grid_constant__ CUtensorMap tm_r16, const MxGemm p, const Plan pl) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = (uint64_t*)(smem + kOffBar);
    const int S = pl.stages, slots = min(kSfSlots, S);
    const uint32_t smem0 = smem_u32(smem);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kMaxStages);
    const uint32_t tfull0 = smem_u32(bars + 2 * kMaxStages), tempty0 = tfull0 + 16, drain = tfull0 + 32;
    uint32_t* tmem_slot = (uint32_t*)(bars + 2 * kMaxStages + 5);
    volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
    int32_t* pre = (int32_t*)(smem + kOffTab);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int FB = (p.N + BF - 1) / BF, KB = (p.K / 2 + kKB - 1) / kKB;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1 + kScaleWarps);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();  // what an earlier kernel wrote
    if (p.offsets && warp == 2) {  // prefix of the groups' row tiles, 32 groups at a time
        int base = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            int n = 0;
            if (g < p.G) {
                const int lo = min(max(p.offsets[g], 0), p.rows), hi = min(max(p.offsets[g + 1], lo), p.rows);
                n = (hi - lo + pl.tile_rows - 1) / pl.tile_rows;
                pre[kMaxG + 1 + g] = lo;
            }
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (g < p.G) pre[g] = base + inc - n;
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            pre[p.G] = base;
            pre[kMaxG + 1 + p.G] = min(max(p.offsets[p.G], 0), p.rows);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_release();  // (once tensor memory is ours)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // Units of this CTA: u0, u0 + step, ...; k-blocks [kb0, kb1) of each.  Split: a cluster takes one
    // unit (or none: the grid covers a bound on their number).
    const int units = (p.offsets ? pre[p.G] : (p.rows + pl.tile_rows - 1) / pl.tile_rows) * FB;
    const int rank = SPLIT ? (int)cluster_rank() : 0, cl = SPLIT ? pl.split : 1;
    const int u0 = (int)blockIdx.x / cl, step = (int)gridDim.x / cl;
    const int KB2 = (KB + 1) / 2;  // split at even blocks: a load of scales is two
    const int kb0 = SPLIT ? 2 * (KB2 * rank / pl.split) : 0, kb1 = SPLIT ? min(KB, 2 * (KB2 * (rank + 1) / pl.split)) : KB;
    const int64_t my_stages = u0 < units ? (int64_t)((units - 1 - u0) / step + 1) * (kb1 - kb0) : 0;
    const int64_t lim = p.spin_ns;

    if (warp == 0) {
        // -------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0; u < units && ok; u += step) {
            const Unit un = unit_at(p, pl, u, FB, pre);
            // whole 64-row boxes, then 16-row boxes (rows past the tile are read and ignored)
            const int n16 = __shfl_sync(0xffffffffu, (un.rows + 15) >> 4, 0), n64 = n16 >> 2, rest = n16 & 3;
            const int wrow = __shfl_sync(0xffffffffu, un.g * p.N + un.f0, 0);
            const int row0 = __shfl_sync(0xffffffffu, un.row0, 0);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = warp_wait(empty0 + 8 * stage, phase ^ 1, lim, abort_flag, p.err, 51);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t fb = full0 + 8 * stage, base = smem0 + stage * pl.stage_bytes;
                    mbar_expect_tx(fb, kWBytes + n16 * 16 * kKB);
                    tma_load_2d(base, &tm_w, fb, kb * kKB, wrow);
                    for (int i = 0; i < n64; ++i) tma_load_2d(base + kWBytes + i * 64 * kKB, &tm_r64, fb, kb * kKB, row0 + i * 64);
                    for (int i = 0; i < rest; ++i)
                        tma_load_2d(base + kWBytes + (n64 * 64 + i * 16) * kKB, &tm_r16, fb, kb * kKB, row0 + n64 * 64 + i * 16);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) sleep_ns(200000);  // copies already issued land before the CTA leaves
    } else if (warp == 1) {
        // --------------------------------------------------- MMA issuer
        // One wait a stage (its barrier counts the operands' bytes and the
        // scale warps): the issue of a stage takes about as long as its MMAs.
        int stage = 0, slot = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        const bool wide = pl.tile_rows > 128;
        const uint32_t rstep = wide ? 8 : 4;
        for (int u = u0; u < units && ok; u += step) {
            const Unit un = unit_at(p, pl, u, FB, pre);
            const int n = __shfl_sync(0xffffffffu, (un.rows + 15) & ~15, 0);
            const uint32_t id0 = idesc(n, 0), id2 = idesc(n, 2);
            ok = warp_wait(tempty0 + 8 * acc, acc_phase ^ 1, lim, abort_flag, p.err, 52);
            if (!ok) break;
            const uint32_t d = tmem + acc * 128;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = warp_wait(full0 + 8 * stage, phase, lim, abort_flag, p.err, 53);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    // scale columns: two k halves of the weights, then of the rows (a half's columns for 256
                    // rows lie at 8 + 8 half, for 128 at 8 + 4 half)
                    const uint32_t sf = smem0 + kOffSf + slot * kSfBytes, sfw = tmem + kAccCols + slot * kSfCols, sfr = sfw + 8;
#pragma unroll
                    for (int c = 0; c < 4; ++c) copy_sf(sfw + 4 * c, sf + c * kSfChunk);
                    if (wide) {
                        copy_sf(sfw + 16, sf + 4 * kSfChunk);
                        copy_sf(sfw + 20, sf + 5 * kSfChunk);
                    }
                    const uint64_t wd = umma_desc(smem0 + stage * pl.stage_bytes);
                    const uint64_t rd = umma_desc(smem0 + stage * pl.stage_bytes + kWBytes);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_mxf4(d, wd + (uint64_t)(kk * 2), rd + (uint64_t)(kk * 2), kk & 1 ? id2 : id0, sfw + 4 * (kk >> 1),
                                        sfr + rstep * (kk >> 1), kb != kb0 || kk != 0);
                    umma_commit(empty0 + 8 * stage);
                    if (kb + 1 == kb1) umma_commit(tfull0 + 8 * acc);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++slot == slots) slot = 0;
            }
            if (++acc == pl.accs) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (elect_one()) umma_commit(drain);  // everything issued is done before tensor memory is freed
        __syncwarp();
        volatile int never = 0;
        mbar_wait(drain, 0, 1000000000LL, &never);
    } else if (warp < 2 + kScaleWarps) {
        // ------------------------------------------------------- scales
        // Thread r: weight row r, rows r and 128 + r of the tile, sixteen
        // bytes (two stages) a load; the next kAhead loads of a row are in
        // flight in registers (their latency beside the operands' traffic is
        // some 2500 cycles).  Two stages are written at a time: a wait, a
        // proxy fence and an arrival cost a few hundred cycles, as much as
        // half a stage's MMAs.  The slots are free when the MMAs of the
        // stages `slots` before are done: the stage barriers tell (the ring
        // has at least that many stages).
        const int r = threadIdx.x - 64, blocks = p.K / kMxBlock;
        const int64_t wrows = (int64_t)p.G * p.N;
        const int nk = kb1 - kb0, pairs = (nk + 1) / 2;  // loads of a unit
        const bool wide = pl.tile_rows > 128;
        const uint8_t *rw = nullptr, *r0 = nullptr, *r1 = nullptr;
        int fu = u0, fp = 0;  // the load to issue next
        uint4 q[kAhead][3];
        auto fetch = [&](uint4 (&v)[3]) {
            if (fu >= units) return;
            if (fp == 0) {
                const Unit un = unit_at(p, pl, fu, FB, pre);
                rw = p.b_scale + min((int64_t)un.g * p.N + un.f0 + r, wrows - 1) * blocks;
                r0 = p.a_scale + (int64_t)min(un.row0 + r, p.rows - 1) * blocks;
                r1 = p.a_scale + (int64_t)min(un.row0 + r + 128, p.rows - 1) * blocks;
            }
            const int b0 = kb0 * kBlk + fp * 2 * kBlk;
            v[0] = load_scales<VEC>(rw, b0, blocks);
            v[1] = load_scales<VEC>(r0, b0, blocks);
            if (wide) v[2] = load_scales<VEC>(r1, b0, blocks);
            if (++fp == pairs) {
                fp = 0;
                fu += step;
            }
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(q[i]);
        int slot = 0, left = nk;  // left: stages of the unit still to be written
        int64_t written = 0;
        uint8_t* dst0 = smem + kOffSf + (r & 31) * 16 + (r >> 5) * 4;
        int stage = 0, wstage = 0;  // ring stage being written, and of the stage `slots` before it with its phase
        uint32_t wphase = 0;
        auto write = [&](uint32_t w0, uint32_t w1, uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
            uint8_t* dst = dst0 + slot * kSfBytes;
            *(uint32_t*)(dst) = w0;
            *(uint32_t*)(dst + kSfChunk) = w1;
            if (wide) {
                *(uint32_t*)(dst + 2 * kSfChunk) = a0;
                *(uint32_t*)(dst + 3 * kSfChunk) = b0;
                *(uint32_t*)(dst + 4 * kSfChunk) = a1;
                *(uint32_t*)(dst + 5 * kSfChunk) = b1;
            } else {
                *(uint32_t*)(dst + 2 * kSfChunk) = a0;
                *(uint32_t*)(dst + 3 * kSfChunk) = a1;
            }
            if (++slot == slots) slot = 0;
        };
        auto tell = [&]() {
            if (lane == 0) mbar_arrive(full0 + 8 * stage);
            if (++stage == S) stage = 0;
        };
        auto put2 = [&](const uint4 (&v)[3]) -> bool {
            const int two = left > 1 ? 2 : 1;
            for (int i = 0; i < two; ++i) {
                if (written++ < slots) continue;
                // (the MMAs finish in order: of two stages the second is waited for)
                if (i + 1 == two) {
                    const bool ok = mbar_wait(empty0 + 8 * wstage, wphase, lim, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) return false;
                }
                if (++wstage == S) {
                    wstage = 0;
                    wphase ^= 1;
                }
            }
            write(v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y);
            if (two == 2) write(v[0].z, v[0].w, v[1].z, v[1].w, v[2].z, v[2].w);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            tell();
            if (two == 2) tell();
            left -= two;
            if (left == 0) left = nk;
            return true;
        };
        const int64_t total = nk > 0 ? my_stages / nk * pairs : 0;
        bool go = true;
        for (int64_t i = 0; i < total && go; i += kAhead) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i + j >= total || !go) break;
                go = put2(q[j]);
                fetch(q[j]);
            }
        }
    }
    // ---------------------------------------------------------- epilogue
    // Lanes are features, columns rows.
    const int ew = warp - 2 - kScaleWarps, sub = warp & 3, half = ew >> 2;  // lane quarter, column half
    if (!SPLIT && ew >= 0) {
        uint8_t* st = smem + kOffStage + ew * kStWarp;
        const bool vec = p.N % 8 == 0 && p.ldo % 8 == 0 && ((uintptr_t)p.out & 15) == 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = u0; u < units; u += step) {
            const Unit un = unit_at(p, pl, u, FB, pre);
            const bool ok = mbar_wait(tfull0 + 8 * acc, acc_phase, lim, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0 && !*abort_flag) {
                    record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 54, blockIdx.x, u);
                    *abort_flag = 1;
                }
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem + acc * 128 + ((uint32_t)(sub * 32) << 16);
            const uint32_t te = tempty0 + 8 * acc;
            if (++acc == pl.accs) {
                acc = 0;
                acc_phase ^= 1;
            }
            const int f = un.f0 + sub * 32, cols = p.N - f;  // features of this warp inside the matrix
            // this half's 32-row blocks: 0, 2, 4, 6 or 1, 3, 5, 7
            if (p.out_elem == kF32) {
#pragma unroll 1
                for (int c = half * 32; c < un.rows; c += 64) {
                    uint32_t v[32];
                    tmem_ld32(taddr + c, v);
                    tmem_wait_ld();
                    float* o = (float*)p.out + (int64_t)(un.row0 + c) * p.ldo + f + lane;
                    if (lane < cols) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c + j < un.rows) o[(int64_t)j * p.ldo] = __uint_as_float(v[j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(te);
                continue;
            }
            uint32_t pk[4][16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = half * 32 + i * 64;
                if (c < un.rows) {
                    uint32_t v[32];
                    tmem_ld32(taddr + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                        pk[i][j] = *(const uint32_t*)&h;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(te);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = half * 32 + i * 64;
                if (c < un.rows)
                    store_block(st, pk[i], (bf16*)p.out + (int64_t)(un.row0 + c) * p.ldo + f, p.ldo, un.rows - c, cols, vec);
            }
        }
    }
    if (SPLIT) {
        // One unit a cluster.  Rank q sums rows q, q + split, ... of the tile
        // in blocks of four: every rank sends it its partial sums, [rank][slot
        // of four rows][feature], into the ring, which is idle by then.
        __syncwarp();
        cluster_sync();  // every CTA's loads, MMAs and scale copies are done
        const bool has = u0 < units;
        const Unit un = has ? unit_at(p, pl, u0, FB, pre) : Unit{};
        const int quads = (un.rows + 3) >> 2, per = (quads + pl.split - 1) / pl.split;  // four-row slots, of each rank
        const uint32_t part = (uint32_t)(per * BF * 16);                                // bytes a rank sends another
        if (has && ew >= 0) {
            tc_fence_after();  // the accumulator was committed before the barrier
            const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16);
            const uint32_t mine = smem0 + rank * part + (uint32_t)((sub * 32 + lane) * 16);
#pragma unroll 1
            for (int c = half * 16; c < un.rows; c += 32) {
                uint32_t v[16];
                tmem_ld16(taddr + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int qd = c / 4 + j;
                    if (qd < quads) {
                        const float4 x = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]), __uint_as_float(v[4 * j + 2]),
                                               __uint_as_float(v[4 * j + 3]));
                        st_cluster(mapa_shared(mine + (uint32_t)(qd / pl.split) * BF * 16, (uint32_t)(qd % pl.split)), x);
                    }
                }
            }
            tc_fence_before();
        }
        __syncwarp();
        cluster_sync();
        if (has && ew >= 0) {
            const int f = threadIdx.x - 32 * (2 + kScaleWarps), feat = un.f0 + (f & 127);
            for (int i = f >> 7; i < per; i += 2) {
                const int row = (i * pl.split + rank) * 4;
                if (row >= un.rows) break;
                float s[4] = {0, 0, 0, 0};
                for (int k = 0; k < pl.split; ++k) {
                    const float4 x = *(const float4*)(smem + k * part + i * BF * 16 + (f & 127) * 16);
                    s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
                }
                if (feat < p.N) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (row + j < un.rows) {
                            const int64_t at = (int64_t)(un.row0 + row + j) * p.ldo + feat;
                            if (p.out_elem == kF32) ((float*)p.out)[at] = s[j];
                            else ((bf16*)p.out)[at] = __float2bfloat16_rn(s[j]);
                        }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Codes [rows, bytes], boxes of one 128-byte swizzled line by box_rows.
bool code_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {kKB, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap w, r64, r16;
};
template <int VEC, bool SPLIT> cudaError_t launch(const MxGemm& g, const Maps& m, const Plan& pl, int grid, cudaStream_t s) {
    cudaError_t e = ensure_smem_attr((const void*)gemm_mx_kernel<VEC, SPLIT>, kSmem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(gemm_mx_kernel<VEC, SPLIT>, dim3(grid), dim3(kThreads), kSmem, s, SPLIT ? pl.split : 1, m.w, m.r64, m.r16, g, pl);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mxg

cudaError_t launch_gemm_mx(const MxGemm& g, int num_sms, cudaStream_t stream) {
    using namespace mxg;
    Maps m;
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    if (!code_map(&m.w, g.b, (int64_t)g.G * g.N, g.K / 2, BF) || !code_map(&m.r64, g.a, g.rows, g.K / 2, 64) ||
        !code_map(&m.r16, g.a, g.rows, g.K / 2, 16))
        return cudaErrorInvalidValue;
    Plan pl = {};
    // Rows of a tile: 256 where the groups fill it (the MMA's N side; the
    // weights are read once per tile), fewer where they do not, for more
    // stages of weights in flight and a second accumulator.
    const int64_t avg = cdiv(g.rows, g.G);
    pl.tile_rows = avg > 128 ? 256 : avg > 32 ? 128 : 64;
    pl.stage_bytes = kWBytes + pl.tile_rows * kKB;
    pl.stages = std::min(kMaxStages, kRing / pl.stage_bytes);
    pl.accs = pl.tile_rows > 128 ? 1 : 2;
    pl.split = 1;
    const int64_t units = (cdiv(g.rows, pl.tile_rows) + (g.offsets && g.G > 1 ? g.G : 0)) * cdiv(g.N, BF);  // at most
    const int KB = (int)cdiv(g.K / 2, kKB);
    while (pl.split < kMaxSplit && units * pl.split * 2 <= num_sms && KB >= 4 * pl.split) pl.split *= 2;
    const int grid = pl.split > 1 ? (int)units * pl.split : (int)std::min<int64_t>(units, num_sms);
    const int blocks = g.K / kMxBlock;
    const uintptr_t al = (uintptr_t)g.a_scale | (uintptr_t)g.b_scale;
#define MOE_MX(V) (pl.split > 1 ? launch<V, true>(g, m, pl, grid, stream) : launch<V, false>(g, m, pl, grid, stream))
    if (blocks % 16 == 0 && al % 16 == 0) return MOE_MX(16);
    if (blocks % 4 == 0 && al % 4 == 0) return MOE_MX(4);
    return MOE_MX(1);
#undef MOE_MX
}

}  // namespace moe

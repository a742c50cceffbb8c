// Product of two microscaled 4-bit matrices (moe_mx_gemm), dense or grouped:
//   out[r][n] = sum_k a[r][k] * b_g[n][k]   for the rows r of group g.
//
// tcgen05.mma kind::mxf4 takes both operands as E2M1 codes and multiplies
// each 32-column block by the product of its two E8M0 scales itself, so the
// kernel feeds it what memory holds.  A 128 x 256 tile, 256 columns of K a
// stage (a 128-byte swizzled line per row: 16 KB of A, 32 KB of B), four
// stages.  The scales' home is tensor memory, in chunks of 128 rows x 4
// blocks: lane = row % 32, word = row / 32, byte = block, which is not how
// rows of scale bytes lie in memory; four warps read the scale bytes (two
// stages of a row a load, a row of A and two of B a thread, two loads ahead),
// write them to shared memory in that order, and the MMA thread copies them
// on with tcgen05.cp, a stage ahead of its MMAs.  Each stage has its own 24
// columns of scales, reused when the stage is, so the stage barriers order
// the copies too.
//
// 448 threads: warp 0 TMA, warp 1 tensor memory + MMA, warps 2-5 scales,
// warps 6-13 epilogue (two per lane quarter, 128 columns each).  The
// accumulator and the scales leave no room for a second 256-column
// accumulator: the epilogue packs its columns into registers, gives the
// accumulator back, and stores while the next tile's MMAs run.
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
namespace mxg {

using namespace tc;

constexpr int BM = 128, BN = 256;
constexpr int kKB = 128;                       // bytes of K a stage: 256 codes
constexpr int kBlk = 2 * kKB / kMxBlock;       // 8 scale bytes of a row
constexpr int kStages = 4;
constexpr int kABytes = BM * kKB, kBBytes = BN * kKB;
constexpr int kSfChunk = 512;                  // 128 rows x 4 blocks
constexpr int kSfBytes = (BM + BN) / 128 * 2 * kSfChunk;
constexpr int kScaleWarps = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kScaleWarps + kEpiWarps);
constexpr int kAccCols = 256, kSfCols = kSfBytes / 128;  // tensor-memory columns (128 lanes x 4 B; scales repeat per quarter)
constexpr int kMaxG = 1025;
constexpr int kStRow = 64;                     // epilogue staging: 32 bf16 columns a row
// shared memory: ring, scales, staging, barriers, tile prefix
constexpr int kOffB = kStages * kABytes;
constexpr int kOffSf = kOffB + kStages * kBBytes;
constexpr int kOffStage = kOffSf + kStages * kSfBytes;
constexpr int kOffBar = kOffStage + kEpiWarps * 32 * kStRow;
constexpr int kOffTab = kOffBar + 256;
constexpr int kSmem = 1024 + kOffTab + (kMaxG + 1) * 4;
static_assert(kSmem <= 232448, "shared memory plan exceeds 227 KB");
static_assert(kSfCols == 24 && kAccCols + kStages * kSfCols <= 512, "tensor memory plan");

// Instruction descriptor of kind::mxf4: E2M1 operands, both K-major, E8M0
// scales; sf: which half of the scale words (0 or 2).
__device__ __forceinline__ uint32_t idesc(int sf) {
    return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(BM >> 4) << 24) |
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

struct Unit {
    int g, row0, rows, n0;  // group, first row of the tile, its rows, first column
};
// pre: prefix of the groups' row tiles
__device__ __forceinline__ Unit unit_at(const MxGemm& p, int u, int NB, const int32_t* pre) {
    Unit r;
    const int rt = u / NB;
    r.n0 = (u - rt * NB) * BN;
    r.g = 0;
    int lo = 0, hi = p.rows, t = rt;
    if (p.offsets) {
        r.g = find_group_smem(pre, p.G, rt);
        t = rt - pre[r.g];
        lo = min(max(__ldg(p.offsets + r.g), 0), p.rows);
        hi = min(max(__ldg(p.offsets + r.g + 1), lo), p.rows);
    }
    r.row0 = lo + t * BM;
    r.rows = min(BM, hi - r.row0);
    return r;
}

// The sixteen scale bytes of a row from block b0, two stages' worth (blocks
// past the row's end: scale 1; their codes are zeros).  VEC: bytes that rows
// are aligned to.
template <int VEC> __device__ __forceinline__ uint4 load_scales(const uint8_t* row, int b0, int blocks) {
    uint32_t w[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if constexpr (VEC == 16) {
        return __ldg((const uint4*)(row + b0));
    } else if constexpr (VEC == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (b0 + 4 * j < blocks) w[j] = __ldg((const uint32_t*)(row + b0 + 4 * j));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (b0 + i < blocks) w[i / 4] = (w[i / 4] & ~(255u << (8 * (i & 3)))) | (uint32_t)__ldg(row + b0 + i) << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int VEC>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const MxGemm p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = (uint64_t*)(smem + kOffBar);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages), sfull0 = smem_u32(bars + 2 * kStages);
    const uint32_t tfull = smem_u32(bars + 3 * kStages), tempty = smem_u32(bars + 3 * kStages + 1), drain = smem_u32(bars + 3 * kStages + 2);
    uint32_t* tmem_slot = (uint32_t*)(bars + 3 * kStages + 3);
    volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
    int32_t* pre = (int32_t*)(smem + kOffTab);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NB = (p.N + BN - 1) / BN, KB = (p.K / 2 + kKB - 1) / kKB;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(sfull0 + 8 * s, kScaleWarps);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, kEpiWarps);
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (p.offsets && warp == 2) {  // prefix of the groups' row tiles, 32 groups at a time
        int base = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            int n = 0;
            if (g < p.G) {
                const int lo = min(max(__ldg(p.offsets + g), 0), p.rows), hi = min(max(__ldg(p.offsets + g + 1), lo), p.rows);
                n = (hi - lo + BM - 1) / BM;
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
        if (lane == 0) pre[p.G] = base;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int units = (p.offsets ? pre[p.G] : (p.rows + BM - 1) / BM) * NB;
    const int64_t lim = p.spin_ns;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit un = unit_at(p, u, NB, pre);
                for (int kb = 0; kb < KB; ++kb) {
                    ok = mbar_wait(empty0 + 8 * stage, phase ^ 1, lim, abort_flag);
                    if (!ok) {
                        record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 51, blockIdx.x, u);
                        *abort_flag = 1;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * stage;
                    mbar_expect_tx(fb, kABytes + kBBytes);
                    tma_load_2d(smem_u32(smem + stage * kABytes), &tm_a, fb, kb * kKB, un.row0);
                    tma_load_2d(smem_u32(smem + kOffB + stage * kBBytes), &tm_b, fb, kb * kKB, un.g * p.N + un.n0);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) sleep_ns(200000);  // copies already issued land before the CTA leaves
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ----------------------------------------------- MMA issuer
            // A stage's scales are copied before the MMAs of the stage before
            // it are issued, so that the copies run beside them.
            int stage = 0, cstage = 0;
            uint32_t phase = 0, cphase = 0, acc_phase = 0;
            bool ok = true;
            int64_t copies = units > (int)blockIdx.x ? (int64_t)((units - 1 - blockIdx.x) / gridDim.x + 1) * KB : 0;  // left to make
            auto copy_scales = [&]() {
                if (copies-- <= 0 || !ok) return;
                ok = mbar_wait(sfull0 + 8 * cstage, cphase, lim, abort_flag);
                if (!ok) {
                    record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 55, blockIdx.x, 0);
                    *abort_flag = 1;
                    return;
                }
                tc_fence_after();
                const uint32_t sf = smem_u32(smem + kOffSf + cstage * kSfBytes), t = tmem + kAccCols + cstage * kSfCols;
#pragma unroll
                for (int c = 0; c < 6; ++c) copy_sf(t + 4 * c, sf + c * kSfChunk);
                if (++cstage == kStages) {
                    cstage = 0;
                    cphase ^= 1;
                }
            };
            copy_scales();
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                ok = mbar_wait(tempty, acc_phase ^ 1, lim, abort_flag);
                if (!ok) {
                    record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 52, blockIdx.x, u);
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after();
                for (int kb = 0; kb < KB; ++kb) {
                    copy_scales();
                    ok = ok && mbar_wait(full0 + 8 * stage, phase, lim, abort_flag);
                    if (!ok) {
                        record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 53, blockIdx.x, u);
                        *abort_flag = 1;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sfa = tmem + kAccCols + stage * kSfCols, sfb = sfa + 8;
                    const uint64_t ad = umma_desc(smem_u32(smem + stage * kABytes));
                    const uint64_t bd = umma_desc(smem_u32(smem + kOffB + stage * kBBytes));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_mxf4(tmem, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc((kk & 1) * 2), sfa + 4 * (kk >> 1),
                                  sfb + 8 * (kk >> 1), (kb | kk) != 0);
                    umma_commit(empty0 + 8 * stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                umma_commit(tfull);
                acc_phase ^= 1;
            }
            umma_commit(drain);  // everything issued is done before tensor memory is freed
            volatile int never = 0;
            mbar_wait(drain, 0, 1000000000LL, &never);
        }
    } else if (warp < 2 + kScaleWarps) {
        // ------------------------------------------------------- scales
        // Thread r: row r of A, rows r and 128 + r of B, sixteen bytes (two
        // stages) a load; the next two loads of a row are in flight in
        // registers ahead of the stages being written.
        const int r = threadIdx.x - 64, blocks = p.K / kMxBlock;
        const int64_t brows = (int64_t)p.G * p.N;
        const int pairs = (KB + 1) / 2;  // loads of a unit
        const uint8_t *ra = nullptr, *rb0 = nullptr, *rb1 = nullptr;
        int fu = blockIdx.x, fp = 0;  // the load to issue next
        uint4 q[2][3];
        auto fetch = [&](uint4 (&v)[3]) {
            if (fu >= units) return;
            if (fp == 0) {
                const Unit un = unit_at(p, fu, NB, pre);
                ra = p.a_scale + (int64_t)min(un.row0 + r, p.rows - 1) * blocks;
                const int64_t b = (int64_t)un.g * p.N + un.n0 + r;
                rb0 = p.b_scale + min(b, brows - 1) * blocks;
                rb1 = p.b_scale + min(b + 128, brows - 1) * blocks;
            }
            v[0] = load_scales<VEC>(ra, fp * 2 * kBlk, blocks);
            v[1] = load_scales<VEC>(rb0, fp * 2 * kBlk, blocks);
            v[2] = load_scales<VEC>(rb1, fp * 2 * kBlk, blocks);
            if (++fp == pairs) {
                fp = 0;
                fu += gridDim.x;
            }
        };
        fetch(q[0]);
        fetch(q[1]);
        int stage = 0, left = KB;  // stages left of the unit being written
        uint32_t phase = 0;
        const int64_t total = units > (int)blockIdx.x ? (int64_t)((units - 1 - blockIdx.x) / gridDim.x + 1) * pairs : 0;
        // chunk: k half of A; then for each k half the two 128-row halves of B
        uint8_t* dst0 = smem + kOffSf + (r & 31) * 16 + (r >> 5) * 4;
        auto put = [&](uint32_t a0, uint32_t a1, uint32_t b00, uint32_t b01, uint32_t b10, uint32_t b11) -> bool {
            const bool ok = mbar_wait(empty0 + 8 * stage, phase ^ 1, lim, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) return false;
            uint8_t* dst = dst0 + stage * kSfBytes;
            *(uint32_t*)(dst) = a0;
            *(uint32_t*)(dst + kSfChunk) = a1;
            *(uint32_t*)(dst + 2 * kSfChunk) = b00;
            *(uint32_t*)(dst + 3 * kSfChunk) = b10;
            *(uint32_t*)(dst + 4 * kSfChunk) = b01;
            *(uint32_t*)(dst + 5 * kSfChunk) = b11;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull0 + 8 * stage);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
            return true;
        };
        auto put2 = [&](const uint4 (&v)[3]) -> bool {
            if (!put(v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y)) return false;
            if (--left > 0) {
                if (!put(v[0].z, v[0].w, v[1].z, v[1].w, v[2].z, v[2].w)) return false;
                --left;
            }
            if (left <= 0) left = KB;
            return true;
        };
        for (int64_t i = 0; i < total; i += 2) {
            if (!put2(q[0])) break;
            fetch(q[0]);
            if (i + 1 < total) {
                if (!put2(q[1])) break;
                fetch(q[1]);
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        const int ew = warp - 2 - kScaleWarps, sub = warp & 3, half = ew >> 2;  // lane quarter, column half
        uint8_t* st = smem + kOffStage + ew * 32 * kStRow;
        const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16) + half * 128;
        const int row = sub * 32 + lane;
        uint32_t acc_phase = 0;
        const bool vec = p.N % 8 == 0 && p.ldo % 8 == 0 && ((uintptr_t)p.out & 15) == 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            const Unit un = unit_at(p, u, NB, pre);
            const bool ok = mbar_wait(tfull, acc_phase, lim, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0 && !*abort_flag) {
                    record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 54, blockIdx.x, u);
                    *abort_flag = 1;
                }
                break;
            }
            acc_phase ^= 1;
            tc_fence_after();
            const int n0 = un.n0 + half * 128;
            if (p.out_elem == kF32) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld32(taddr + c * 32, v);
                    tmem_wait_ld();
                    float* o = (float*)p.out + (int64_t)(un.row0 + row) * p.ldo + n0 + c * 32;
                    if (row < un.rows) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (n0 + c * 32 + j < p.N) o[j] = __uint_as_float(v[j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty);
                continue;
            }
            uint32_t pk[64];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld32(taddr + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    pk[c * 16 + j] = *(const uint32_t*)&h;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty);
            bf16* out = (bf16*)p.out + (int64_t)un.row0 * p.ldo;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int col = n0 + c * 32;
                if (vec) {
                    // through shared memory: rows of 64 bytes, 16-byte pieces swizzled over the rows
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *(uint4*)(st + lane * kStRow + ((q ^ ((lane >> 1) & 3)) * 16)) =
                            make_uint4(pk[c * 16 + 4 * q], pk[c * 16 + 4 * q + 1], pk[c * 16 + 4 * q + 2], pk[c * 16 + 4 * q + 3]);
                    __syncwarp();
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int rr = 8 * it + (lane >> 2), q = lane & 3;
                        const uint4 v = *(const uint4*)(st + rr * kStRow + ((q ^ ((rr >> 1) & 3)) * 16));
                        if (sub * 32 + rr < un.rows && col + q * 8 < p.N) *(uint4*)(out + (int64_t)(sub * 32 + rr) * p.ldo + col + q * 8) = v;
                    }
                    __syncwarp();
                } else if (row < un.rows) {
                    const bf16* h = (const bf16*)(pk + c * 16);
                    bf16* o = out + (int64_t)row * p.ldo + col;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (col + j < p.N) o[j] = h[j];
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

template <int VEC> cudaError_t launch(const MxGemm& g, const CUtensorMap& a, const CUtensorMap& b, int grid, cudaStream_t s) {
    const cudaError_t e = ensure_smem_attr((const void*)gemm_mx_kernel<VEC>, kSmem);
    if (e != cudaSuccess) return e;
    gemm_mx_kernel<VEC><<<grid, kThreads, kSmem, s>>>(a, b, g);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace mxg

cudaError_t launch_gemm_mx(const MxGemm& g, int num_sms, cudaStream_t stream) {
    using namespace mxg;
    CUtensorMap a, b;
    if (!tc::encode_fn()) return cudaErrorNotSupported;
    if (!code_map(&a, g.a, g.rows, g.K / 2, BM) || !code_map(&b, g.b, (int64_t)g.G * g.N, g.K / 2, BN)) return cudaErrorInvalidValue;
    const int64_t units = (cdiv(g.rows, BM) + (g.offsets ? g.G : 0)) * cdiv(g.N, BN);  // at most
    const int grid = (int)std::min<int64_t>(units, num_sms);
    const int blocks = g.K / kMxBlock;
    const uintptr_t al = (uintptr_t)g.a_scale | (uintptr_t)g.b_scale;
    if (blocks % 16 == 0 && al % 16 == 0) return launch<16>(g, a, b, grid, stream);
    if (blocks % 4 == 0 && al % 4 == 0) return launch<4>(g, a, b, grid, stream);
    return launch<1>(g, a, b, grid, stream);
}

}  // namespace moe

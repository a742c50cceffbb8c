// The products of product_few.cu where K is a multiple of 128 and x and the
// weights are aligned to 16 bytes.
//
// There the weights, and a unit's scales and zero points, come to shared
// memory by bulk copies, issued by a warp of their own some stages ahead: with
// loads to registers a warp's waits for x, or for words of other lanes, were
// waits for the weights behind them too.  Lanes then read their words where
// they want them, so that nothing is exchanged.  x of the next 128 columns is
// loaded as soon as an MMA is done with this one's.
//   bf16: a stage is 16 rows of 1024 columns, a copy each, to rows a bank's
//   width apart; a warp takes 128 columns of each.
//   4 bits: a stage is a unit, all columns of 16 rows, or of 64 where they are
//   short.  The rows lie in one piece, but a copy of each, to rows a bank's
//   width apart, is worth its 100 cycles of the TMA unit for long ones.
//
// Measured: 64 groups of 8 rows, 1024 x 4096 bf16 (537 MB), 78 us, 6.9 TB/s;
// 13 rows over 8 groups 12.7 (8.3 at the copy's rate: of some 420 units an SM
// has two or three).  Codes, groups of 128 columns, 64 groups of a row: 49 us at
// 1024 x 4096, 51 at 4096 x 1024 (72 with tiles of 16 features).  80 rows over
// 128 groups, 1024 x 4096 with zero points in groups of 64 columns, 34 to 36 us
// (11 to 13 at the copy's rate): the loads alone take 20 of them; decoding and
// multiplying take 250 instructions a chunk of 16 x 128 codes and warp, 58 % of
// the ALU pipe's cycles, and do not hide the loads in full.  One token by 4096 x
// 4096 codes: 5.9 us a call from Python, latency.
#include <algorithm>

#include "few_rows.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace few_rows {

namespace {

using namespace tc;

constexpr int kMaxStages = 8, kDenseCols = 1024;
constexpr int kAllThreads = kThreads + 32;  // and the loading warp

struct Shape {
    int stages, stage_bytes, pitch;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, int bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// First column, within a chunk, of the eight in word i of lane t.
template <int LG> __device__ __forceinline__ int col_of(int i, int t) {
    return LG == 7 ? 32 * t + 8 * i : LG == 6 ? 64 * (i >> 1) + 16 * t + 8 * (i & 1) : 32 * i + 8 * t;
}

template <int LG, typename T, typename TS, int SUB>
__global__ void __launch_bounds__(kAllThreads, 2) product_few_bulk_kernel(const Args p, const Shape q) {
    extern __shared__ __align__(128) uint8_t ring[];
    constexpr int F = kF * SUB, kBufs = SUB == 1 ? 2 : 1;
    __shared__ Tables<F, kBufs> tab;
    __shared__ uint64_t bars[2 * kMaxStages];
    __shared__ volatile int abort_flag;
    constexpr bool kCoded = LG != 0, kAhead = sizeof(T) == 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages;
    if (threadIdx.x == 0) {
        for (int s = 0; s < q.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kWarps);
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    const int FB = (p.N + F - 1) / F, units = build_tables<F>(tab, p), step = gridDim.x;
    if ((int)blockIdx.x >= units) return;
    const int nb = kCoded ? p.K >> (kCoded ? LG : 7) : 0, chunks = p.K / kChunk;
    const int per_unit = kCoded ? 1 : (p.K + kDenseCols - 1) / kDenseCols;  // stages
    int stage = 0;
    uint32_t phase = 0;
    auto advance = [&]() {
        if (++stage == q.stages) {
            stage = 0;
            phase ^= 1;
        }
    };

    if (warp == kWarps) {
        // ----------------------------------------------------------- loads
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += step) {
            const Unit un = unit_at<F>(u, FB, p.G, tab);
            const int rows = min(F, p.N - un.f0);
            const int64_t row = (int64_t)un.g * p.N + un.f0;
            for (int i = 0; i < per_unit; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * stage, phase ^ 1, p.spin_ns, &abort_flag));
                if (!ok) break;
                const uint32_t bar = full0 + 8 * stage, dst = smem_u32(ring) + stage * q.stage_bytes;
                if constexpr (kCoded) {
                    const int sb = rows * nb * (int)sizeof(TS), zb = p.q.zeros ? rows * nb : 0;
                    const uint32_t sd = dst + F * q.pitch;
                    if (lane == 0) mbar_expect_tx(bar, rows * (p.K / 2) + sb + zb);
                    __syncwarp();
                    if (q.pitch != p.K / 2) {
                        for (int r = lane; r < rows; r += 32) bulk_load(dst + r * q.pitch, p.q.codes + (row + r) * (p.K / 2), p.K / 2, bar);
                    } else if (lane == 0) {
                        bulk_load(dst, p.q.codes + row * (p.K / 2), rows * (p.K / 2), bar);
                    }
                    if (lane == 1) bulk_load(sd, (const TS*)p.q.scales + row * nb, sb, bar);
                    if (lane == 2 && zb) bulk_load(sd + F * nb * (int)sizeof(TS), p.q.zeros + row * nb, zb, bar);
                } else {
                    const int bytes = 2 * min(kDenseCols, p.K - i * kDenseCols);
                    if (lane == 0) mbar_expect_tx(bar, rows * bytes);
                    __syncwarp();
                    if (lane < rows) bulk_load(dst + lane * q.pitch, p.w + (row + lane) * p.K + i * kDenseCols, bytes, bar);
                }
                __syncwarp();
                advance();
            }
        }
        if (!ok) sleep_ns(200000);  // copies already issued land before the block leaves
        return;
    }

    // This warp's chunks of a unit: first, first + every, ... below end.
    const int first = kCoded ? chunks * warp / kWarps : warp, every = kCoded ? 1 : kWarps;
    const int end = kCoded ? chunks * (warp + 1) / kWarps : chunks;
    Parts<T> x[kAhead ? 4 : 1];
    const int xt = col_of<LG>(0, t);
    auto x_at = [&](const Unit& un, int r) {  // rows past the tile: the last one's, their sums are not stored
        return (const T*)p.x + (int64_t)(un.row0 + min(r, un.n - 1)) * p.ldx + xt;
    };
    Unit cur = unit_at<F>(blockIdx.x, FB, p.G, tab);
    const T* x0 = x_at(cur, g);
    if (kAhead && first < end) {
#pragma unroll
        for (int i = 0; i < (kAhead ? 4 : 1); ++i) load_x<true>(x0 + first * kChunk + col_of<LG>(i, 0), x[i]);
    }
    int buf = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units; u += step, buf ^= kBufs - 1) {
        const bool more = u + step < units;
        const Unit nxt = more ? unit_at<F>(u + step, FB, p.G, tab) : cur;
        const T* xn = x_at(nxt, g);
        float acc[SUB][4] = {};
        int k = first;
        for (int st = 0; st < per_unit; ++st) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(full0 + 8 * stage, phase, p.spin_ns, &abort_flag));
            if (!ok) break;
            const uint8_t* base = ring + stage * q.stage_bytes;
            const int stop = kCoded ? end : min(end, (st + 1) * kWarps);
            for (; k < stop; k += every) {
                const T* xk = x0 + k * kChunk;
                const T* ahead = k + every < end ? xk + every * kChunk : more ? xn + first * kChunk : xk;  // next columns
                if constexpr (!kCoded) {
                    const uint8_t* r0 = base + g * q.pitch + (k - st * kWarps) * kChunk * 2 + 16 * t;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 a4 = *(const uint4*)(r0 + 64 * j), e4 = *(const uint4*)(r0 + 8 * q.pitch + 64 * j);
                        const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, e[4] = {e4.x, e4.y, e4.z, e4.w};
                        mma8(*(float(*)[1][4])acc[0], a, e, x[j].v);
                        load_x<true>(ahead + 32 * j, x[j]);
                    }
                } else {
                    constexpr int kGroups = 1 << (7 - LG), kWords = 4 / kGroups;  // column groups of a chunk, words of each
#pragma unroll
                    for (int sub = 0; sub < SUB; ++sub) {
                        Chunk<LG, TS> v;
                        uint32_t w[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int row = 16 * sub + g + 8 * h, at = row * nb + k * kGroups;
                            const uint8_t* r = base + row * q.pitch + k * (kChunk / 2) + (LG == 7 ? 16 : LG == 6 ? 8 : 4) * t;
                            if constexpr (LG == 7) {
                                *(uint4*)w[h] = *(const uint4*)r;
                            } else if constexpr (LG == 6) {
                                *(uint2*)w[h] = *(const uint2*)r;
                                *(uint2*)(w[h] + 2) = *(const uint2*)(r + 32);
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j) w[h][j] = *(const uint32_t*)(r + 16 * j);
                            }
                            const uint8_t* s = base + F * q.pitch + at * (int)sizeof(TS);
                            constexpr int kBytes = kGroups * (int)sizeof(TS);
                            if constexpr (kBytes == 2) v.s[h][0] = *(const uint16_t*)s;
                            else if constexpr (kBytes == 4) v.s[h][0] = *(const uint32_t*)s;
                            else if constexpr (kBytes == 8) *(uint2*)v.s[h] = *(const uint2*)s;
                            else *(uint4*)v.s[h] = *(const uint4*)s;
                            v.z[h] = 0x08080808u;
                            if (p.q.zeros) {
                                const uint8_t* z = base + F * q.pitch + F * nb * (int)sizeof(TS) + at;
                                v.z[h] = kGroups == 1 ? *z : kGroups == 2 ? *(const uint16_t*)z : *(const uint32_t*)z;
                            }
                        }
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) {
                            float sum[Parts<T>::n][4] = {};
#pragma unroll
                            for (int j = 0; j < kWords; ++j) {
                                const int wi = gr * kWords + j, col = col_of<LG>(wi, 0);
                                uint32_t a[4], e[4];
                                int4_pairs(w[0][wi], zero_pair(v.z[0], gr), a);
                                int4_pairs(w[1][wi], zero_pair(v.z[1], gr), e);
                                Parts<T>& xj = x[kAhead ? wi : 0];
                                if (!kAhead) load_x<true>(xk + col, xj);
                                mma8(sum, a, e, xj.v);
                                if (kAhead && sub == SUB - 1) load_x<true>(ahead + col, xj);
                            }
                            const float sc[2] = {scale_of(v, 0, gr), scale_of(v, 1, gr)};
                            add_scaled(acc[sub], sum, sc);
                        }
                    }
                }
            }
            // What was loaded has been used (an arrival would not order loads on their way with the copies' writes).
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub)
                asm volatile("" ::"f"(acc[sub][0]), "f"(acc[sub][1]), "f"(acc[sub][2]), "f"(acc[sub][3]) : "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * stage);
            advance();
        }
        if (!ok) {
            if (lane == 0) {
                record_error(p.err, MOE_ERR_DEVICE_TIMEOUT, 71, blockIdx.x, u);
                abort_flag = 1;
            }
        }
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) put_part<F>(tab.part[buf][warp] + 16 * sub, acc[sub], g, t);
        sync_compute();
        finish<LG, T, F>(p, tab.part[buf], cur, nb);
        if (kBufs == 1) sync_compute();
        cur = nxt;
        x0 = xn;
    }
}

template <int LG, typename T, typename TS, int SUB> cudaError_t launch_bulk(const Args& a, int num_sms, cudaStream_t s) {
    constexpr int F = kF * SUB, kStatic = (int)sizeof(Tables<F, SUB == 1 ? 2 : 1>) + 512, kSm = 227 * 1024;
    Shape q;
    int rest = 0;
    if (LG) {
        const int nb = a.K >> (LG ? LG : 7), sb = nb * (int)sizeof(TS), zb = a.q.zeros ? nb : 0;
        if (((uintptr_t)a.q.scales | (uintptr_t)a.q.zeros) & 15) return cudaErrorNotSupported;
        if (a.N % F && (sb % 16 || zb % 16)) return cudaErrorNotSupported;  // a tile's scales start and end on 16 bytes
        rest = F * (sb + zb);
        if (a.K > (1 << 17)) return cudaErrorNotSupported;  // (beyond any ring)
    }
    // Rows a bank's width apart where a copy each does not cost more than their conflicts: 80 rows of 128 experts, 4096
    // columns 34 us, in one copy 36 to 39; 64 rows of 64 experts, 1024 columns 78 and 72.
    constexpr int kPad[8] = {64, 0, 0, 0, 0, 16, 32, 64};
    q.pitch = LG == 0 ? kDenseCols * 2 + kPad[0] : a.K < 2048 ? a.K / 2 : (a.K / 2 + 127) / 128 * 128 + kPad[LG];
    q.stage_bytes = (F * q.pitch + rest + 127) / 128 * 128;
    // two blocks an SM where two stages of each fit, else one
    const int blocks = 2 * q.stage_bytes <= kSm / 2 - kStatic - 1024 ? 2 : 1;
    q.stages = std::min(kMaxStages, (kSm / blocks - kStatic - 1024) / q.stage_bytes);
    if (q.stages < 2) return cudaErrorNotSupported;
    const int64_t tiles = cdiv(a.rows, kRows) + (a.offsets ? std::min(a.G - 1, a.rows) : 0), units = tiles * cdiv(a.N, F);  // at most
    cudaError_t e = ensure_smem_attr((const void*)product_few_bulk_kernel<LG, T, TS, SUB>, q.stages * q.stage_bytes);
    if (e != cudaSuccess) return e;
    e = launch_kernel(product_few_bulk_kernel<LG, T, TS, SUB>, dim3((unsigned)std::min<int64_t>(units, blocks * num_sms)), dim3(kAllThreads),
                      q.stages * q.stage_bytes, s, 1, a, q);
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}
// Tiles of 64 features where K is short, so that a unit's fixed cost (some 240
// instructions a warp, two barriers) is a smaller part of it, and there are
// several for each block all the same.
template <int LG, typename T, typename TS> cudaError_t launch_tiles(const Args& a, int num_sms, cudaStream_t s) {
    const int64_t tiles = cdiv(a.rows, kRows) + (a.offsets ? std::min(a.G - 1, a.rows) : 0);  // at most
    if constexpr (sizeof(T) == 2) {
        if (a.K <= 1024 && tiles * cdiv(a.N, 4 * kF) >= 8 * num_sms) {
            const cudaError_t e = launch_bulk<LG, T, TS, 4>(a, num_sms, s);
            if (e != cudaErrorNotSupported) return e;
        }
    }
    return launch_bulk<LG, T, TS, 1>(a, num_sms, s);
}
template <int LG> cudaError_t launch_coded_bulk(const Args& a, int elem, int num_sms, cudaStream_t s) {
    if (elem == kF32) return a.q.scale_elem == kF32 ? launch_tiles<LG, float, float>(a, num_sms, s) : launch_tiles<LG, float, bf16>(a, num_sms, s);
    return a.q.scale_elem == kF32 ? launch_tiles<LG, bf16, float>(a, num_sms, s) : launch_tiles<LG, bf16, bf16>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_few_bulk(const Args& a, int LG, int elem, int num_sms, cudaStream_t s) {
    const int64_t row = a.rows > 1 ? a.ldx * (elem == kF32 ? 4 : 2) : 0;
    if (a.K % kChunk || ((uintptr_t)a.x & 15) || row % 16) return cudaErrorNotSupported;
    if (LG == 0) return launch_bulk<0, bf16, bf16, 1>(a, num_sms, s);
    if (LG == 5) return launch_coded_bulk<5>(a, elem, num_sms, s);
    if (LG == 6) return launch_coded_bulk<6>(a, elem, num_sms, s);
    return launch_coded_bulk<7>(a, elem, num_sms, s);
}

}  // namespace few_rows
}  // namespace moe

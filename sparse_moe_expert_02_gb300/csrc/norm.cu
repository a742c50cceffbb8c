// Norms before and after a block (moe_norm_pre, moe_norm_post).
//
//   N(v)  = (v - mu) / sqrt(mean((v - mu)^2) + eps) * (w + w_offset) + b,
//           mu = mean(v) (LayerNorm) or 0 (RMSNorm)
//   pre:    n  = N(x)
//   post:   r' = res_scale * r + branch_scale * g * N(y)
//           n' = N_next(r' as stored)
//
// A row is held in registers as fp32, 8 or 16 elements a thread, so that every
// tensor passes once: the statistics are sums over the registers (the
// variance is taken about the mean, not from a sum of squares), and the next
// norm reads r' before it leaves them, rounded as it is stored.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float load_p(const void* p, int is_bf16, int64_t i) {
    return is_bf16 ? __bfloat162float(((const bf16*)p)[i]) : ((const float*)p)[i];
}

// Row access, VEC elements at a time.  VEC = 8: 16-byte accesses (two for
// fp32); thread i of the row takes vector i (PER = 16: and i + nthr).  VEC = 1: any
// alignment, elements i, i + nthr, ...
template <int VEC, int PER> struct Row {
    static constexpr int kChunks = PER / VEC;
    __device__ static int col(int c, int i, int nthr) { return (c * nthr + i) * VEC; }
};

// Eight bf16 as they lie in a 16-byte piece.
__device__ __forceinline__ void unpack8(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// KEEP: by way of L1, for what other rows read too.  Not through the read-only
// path in either case: these kernels start while the one before them, which may
// write what they read, ends (common.cuh, programmatic dependent launch).
template <bool KEEP, typename T> __device__ __forceinline__ T load(const T* p) {
    if constexpr (KEEP) return *p;
    else return __ldcg(p);
}
template <int VEC, bool KEEP = false, typename T> __device__ __forceinline__ void load_vec(const T* p, float* v) {
    if constexpr (VEC == 1) {
        v[0] = to_f32(load<KEEP>(p));
    } else if constexpr (sizeof(T) == 2) {
        unpack8(load<KEEP>((const uint4*)p), v);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 q = load<KEEP>((const float4*)p + h);
            v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
        }
    }
}
// Two values as a bf16 pair (one conversion).
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&h;
}
// Store; v becomes what was stored.
template <int VEC, typename T> __device__ __forceinline__ void store_vec(T* p, float* v) {
    if constexpr (VEC == 1) {
        const T h = from_f32<T>(v[0]);
        *p = h;
        v[0] = to_f32(h);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack2(v[2 * i], v[2 * i + 1]);
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        ((float4*)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        ((float4*)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
// VEC values of a parameter vector (w, b, a per-channel gate), either type.
template <int VEC> __device__ __forceinline__ void load_par(const void* p, int is_bf16, int64_t i, float* v) {
    if (is_bf16) load_vec<VEC, true>((const bf16*)p + i, v);
    else load_vec<VEC, true>((const float*)p + i, v);
}

// Sum over the nthr threads of a row (nthr = 32, or the whole block).  turn
// counts the block's sums: two buffers in turn, so one barrier a sum.
__device__ __forceinline__ float row_sum(float s, int nthr, float (*red)[32], int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (nthr == 32) return s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* r = red[turn & 1];
    ++turn;
    if (lane == 0) r[warp] = s;
    __syncthreads();
    s = lane < (nthr >> 5) ? r[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// v <- N(v) for this thread's elements of the row.
template <int VEC, int PER>
__device__ __forceinline__ void normalise(float* v, const NormParams& n, int i, int nthr, int D, float (*red)[32], int& turn) {
    constexpr int C = Row<VEC, PER>::kChunks;
    if (n.kind == MOE_NORM_NONE) return;
    float mu = 0.0f;
    if (n.kind == MOE_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < PER; ++e) s += v[e];  // elements past D are zero
        mu = row_sum(s, nthr, red, turn) / (float)D;
    }
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (Row<VEC, PER>::col(c, i, nthr) < D) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[c * VEC + e] - mu;
                v[c * VEC + e] = d;
                s = fmaf(d, d, s);
            }
        }
    }
    const float rstd = rsqrtf(row_sum(s, nthr, red, turn) / (float)D + n.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC, PER>::col(c, i, nthr);
        if (col >= D) continue;
        float w[VEC];
        if (n.w) {
            load_par<VEC>(n.w, n.p_bf16, col, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[c * VEC + e] *= rstd * (w[e] + n.w_offset);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[c * VEC + e] *= rstd;
        }
        if (n.b) {
            load_par<VEC>(n.b, n.p_bf16, col, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[c * VEC + e] += w[e];
        }
    }
}

// One row per nthr threads; nthr = 32 (several rows a block) or the block.
template <int VEC, int PER, int MAXT, typename XT, typename OT>
__global__ void __launch_bounds__(MAXT) norm_pre_kernel(const NormParams n, const XT* __restrict__ x, int64_t ld_x, int T,
                                                    int D, OT* __restrict__ out, int64_t ld_out, int nthr) {
    pdl_wait_then_release();
    __shared__ float red[2][32];
    int turn = 0;
    constexpr int C = Row<VEC, PER>::kChunks;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / nthr) + threadIdx.x / nthr;
    const int i = threadIdx.x % nthr;
    if (t >= T) return;  // whole warps: nthr = 32 here
    float v[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC, PER>::col(c, i, nthr);
        if (col < D) load_vec<VEC>(x + t * ld_x + col, v + c * VEC);
    }
    normalise<VEC, PER>(v, n, i, nthr, D, red, turn);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC, PER>::col(c, i, nthr);
        if (col < D) store_vec<VEC>(out + t * ld_out + col, v + c * VEC);
    }
}

__device__ __forceinline__ float gate_value(float g, int sigmoid) { return sigmoid ? 1.0f / (1.0f + expf(-g)) : g; }

// The rest of row t once y (in v) and r are in registers.
template <int VEC, int PER, typename RT, typename NT>
__device__ __forceinline__ void post_row(const PostParams& p, int64_t t, int i, int nthr, float* v, float* r, RT* out, NT* next,
                                         float (*red)[32], int& turn) {
    constexpr int C = Row<VEC, PER>::kChunks;
    const int D = p.D;
    normalise<VEC, PER>(v, p.norm, i, nthr, D, red, turn);
    const float scale = p.branch_scale * (p.gate_by == MOE_GATE_TOKEN ? gate_value(load_p(p.gate, p.gate_bf16, t), p.gate_sigmoid) : 1.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC, PER>::col(c, i, nthr);
        if (col >= D) continue;
        if (p.gate_by == MOE_GATE_CHANNEL || p.gate_by == MOE_GATE_FULL) {
            float g[VEC];
            load_par<VEC>(p.gate, p.gate_bf16, (p.gate_by == MOE_GATE_FULL ? t * p.ld_gate : 0) + col, g);
            if (p.gate_sigmoid) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[e] = gate_value(g[e], 1);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[c * VEC + e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[c * VEC + e] = fmaf(scale, v[c * VEC + e], p.res_scale * r[c * VEC + e]);
        store_vec<VEC>(out + t * p.ld_out + col, r + c * VEC);
    }
    if (p.next.kind == MOE_NORM_NONE) return;
    normalise<VEC, PER>(r, p.next, i, nthr, D, red, turn);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC, PER>::col(c, i, nthr);
        if (col < D) store_vec<VEC>(next + t * p.ld_next + col, r + c * VEC);
    }
}

template <int VEC, int PER, int MAXT, typename YT, typename RT, typename NT>
__global__ void __launch_bounds__(MAXT) norm_post_kernel(const PostParams p, const YT* __restrict__ y, const RT* res, RT* out,
                                                     NT* __restrict__ next, int nthr) {
    pdl_wait_then_release();
    __shared__ float red[2][32];
    int turn = 0;
    constexpr int C = Row<VEC, PER>::kChunks;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / nthr) + threadIdx.x / nthr;
    const int i = threadIdx.x % nthr;
    if (t >= p.T) return;
    float v[PER], r[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] = r[e] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = Row<VEC, PER>::col(c, i, nthr);
        if (col < p.D) {
            load_vec<VEC>(y + t * p.ld_y + col, v + c * VEC);
            load_vec<VEC>(res + t * p.ld_res + col, r + c * VEC);
        }
    }
    post_row<VEC, PER>(p, t, i, nthr, v, r, out, next, red, turn);
}

// Many rows of bf16: a block takes row after row, and each thread copies its
// own elements of the next rows into shared memory while it works on this one
// (cp.async: the copies are the thread's own, so nothing but the sums waits
// for other threads).  Without it a block has its loads in flight only until
// its first sum: 8192 x 4096 with gate and next norm 69.3 us; with it 58.4
// (4.6 TB/s).  Rows of fp32 do without: a lane's eight elements are two pieces
// of a 32-byte sector then, fetched by two copies, and 8192 x 4096 fp32 took
// 157 us with the ring, 105 without (pre 79 and 43).
constexpr int kAhead = 2;  // rows in flight (three: 65.4 us, fewer blocks fit)

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
// This thread's elements of a row: 16-byte pieces [piece][thread].
template <int PER> __device__ __forceinline__ void copy_row(uint4* dst, const bf16* row, int i, int nthr, int D) {
#pragma unroll
    for (int c = 0; c < PER / 8; ++c) {
        const int col = (c * nthr + i) * 8;
        if (col < D) copy16(dst + c * nthr, row + col);
    }
}
template <int PER> __device__ __forceinline__ void take_row(const uint4* src, float* v, int i, int nthr, int D) {
#pragma unroll
    for (int c = 0; c < PER / 8; ++c) {
        if ((c * nthr + i) * 8 < D) {
            unpack8(src[c * nthr], v + c * 8);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[c * 8 + k] = 0.0f;
        }
    }
}

template <int PER, int MAXT, typename NT>
__global__ void __launch_bounds__(MAXT) norm_post_rows_kernel(const PostParams p, const bf16* __restrict__ y, const bf16* res, bf16* out,
                                                              NT* __restrict__ next) {
    pdl_wait_then_release();
    extern __shared__ uint4 ring[];
    __shared__ float red[2][32];
    int turn = 0;
    const int nthr = blockDim.x, i = threadIdx.x;
    const int half = PER / 8 * nthr;  // 16-byte pieces of a row
    auto start = [&](int64_t t, int slot) {
        if (t < p.T) {
            uint4* dst = ring + 2 * slot * half + i;
            copy_row<PER>(dst, y + t * p.ld_y, i, nthr, p.D);
            copy_row<PER>(dst + half, res + t * p.ld_res, i, nthr, p.D);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) start((int64_t)blockIdx.x + (int64_t)a * gridDim.x, a);
    int slot = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        float v[PER], r[PER];
        take_row<PER>(ring + 2 * slot * half + i, v, i, nthr, p.D);
        take_row<PER>(ring + (2 * slot + 1) * half + i, r, i, nthr, p.D);
        start(t + (int64_t)kAhead * gridDim.x, slot);
        if (++slot == kAhead) slot = 0;
        post_row<8, PER>(p, t, i, nthr, v, r, out, next, red, turn);
    }
}

template <int PER, int MAXT, typename OT>
__global__ void __launch_bounds__(MAXT) norm_pre_rows_kernel(const NormParams n, const bf16* __restrict__ x, int64_t ld_x, int T, int D,
                                                             OT* __restrict__ out, int64_t ld_out) {
    pdl_wait_then_release();
    extern __shared__ uint4 ring[];
    __shared__ float red[2][32];
    int turn = 0;
    const int nthr = blockDim.x, i = threadIdx.x;
    const int row_pieces = PER / 8 * nthr;
    auto start = [&](int64_t t, int slot) {
        if (t < T) copy_row<PER>(ring + slot * row_pieces + i, x + t * ld_x, i, nthr, D);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) start((int64_t)blockIdx.x + (int64_t)a * gridDim.x, a);
    int slot = 0;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        float v[PER];
        take_row<PER>(ring + slot * row_pieces + i, v, i, nthr, D);
        start(t + (int64_t)kAhead * gridDim.x, slot);
        if (++slot == kAhead) slot = 0;
        normalise<8, PER>(v, n, i, nthr, D, red, turn);
#pragma unroll
        for (int c = 0; c < PER / 8; ++c) {
            const int col = Row<8, PER>::col(c, i, nthr);
            if (col < D) store_vec<8>(out + t * ld_out + col, v + c * 8);
        }
    }
}

// Elements of a thread: eight (one token, before programmatic launches: 3.8 us
// against 4.6 with sixteen), or sixteen where the rows alone fill the GPU and a thread's fixed work (two
// sums) counts (from four rows an SM), or where eight would need more than 1024
// threads.
int row_per(int T, int D) { return D > 8 * kMaxThreads || (T >= 608 && D >= 1024) ? 16 : 8; }
// Threads of a row: a whole number of warps.
int row_threads(int D, int per) { return (int)(32 * cdiv(cdiv(D, per), 32)); }

bool vec_ok(const void* p, int64_t ld, int bytes) {
    return p == nullptr || (((uintptr_t)p & 15) == 0 && (ld * bytes) % 16 == 0);
}
bool par_ok(const NormParams& n) { return vec_ok(n.w, 0, 1) && vec_ok(n.b, 0, 1); }

// The row-after-row kernels' grid, or 0 where they do not apply: rows of one
// warp, too few rows for every block to have several, or rows too long for the
// ring (above 14336 columns after a block).
int rows_grid(int T, int nthr, int ring_bytes) {
    constexpr int kSms = 152, kSmem = 226 * 1024;
    if (nthr < 64 || ring_bytes > kSmem / 2) return 0;
    const int blocks = std::min({2048 / nthr, 65536 / (64 * nthr), kSmem / (ring_bytes + 1280)});
    return T >= 3 * kSms * blocks ? kSms * blocks : 0;
}
template <typename K> cudaError_t allow_smem(K* k, int bytes) { return ensure_smem_attr((const void*)k, bytes); }

}  // namespace

bool norm_supported(int D) { return D <= 16 * kMaxThreads; }

cudaError_t launch_norm_pre(const NormParams& n, const void* x, int x_elem, int64_t ld_x, int T, int D, void* out,
                            int out_elem, int64_t ld_out, cudaStream_t stream) {
    const int per = row_per(T, D), nthr = row_threads(D, per), rows = nthr == 32 ? 4 : 1;
    const dim3 grid((unsigned)cdiv(T, rows)), block(nthr * rows);
    const bool vec = D % 8 == 0 && vec_ok(x, ld_x, x_elem == kF32 ? 4 : 2) &&
                     vec_ok(out, ld_out, out_elem == kF32 ? 4 : 2) && par_ok(n);
    const int ring = kAhead * nthr * per * 2, many = vec && x_elem == kBF16 ? rows_grid(T, nthr, ring) : 0;
    cudaError_t e = cudaSuccess;
#define MOE_PRE_P(PER, MAXT, XT, OT)                                                                                   \
    do {                                                                                                         \
        if (many) {                                                                                              \
            if ((e = allow_smem(norm_pre_rows_kernel<PER, MAXT, OT>, ring)) != cudaSuccess) return e;            \
            e = launch_kernel(norm_pre_rows_kernel<PER, MAXT, OT>, dim3(many), dim3(nthr), ring, stream, 1, n, (const bf16*)x, ld_x, T, D, (OT*)out, ld_out); \
        } else if (vec) {                                                                                        \
            e = launch_kernel(norm_pre_kernel<8, PER, MAXT, XT, OT>, dim3(grid), dim3(block), 0, stream, 1, n, (const XT*)x, ld_x, T, D, (OT*)out, ld_out, nthr); \
        } else {                                                                                                 \
            e = launch_kernel(norm_pre_kernel<1, PER, MAXT, XT, OT>, dim3(grid), dim3(block), 0, stream, 1, n, (const XT*)x, ld_x, T, D, (OT*)out, ld_out, nthr); \
        }                                                                                                        \
    } while (0)
#define MOE_PRE(XT, OT)                          \
    do {                                         \
        if (per == 8) MOE_PRE_P(8, 1024, XT, OT);            \
        else if (nthr <= 512) MOE_PRE_P(16, 512, XT, OT);    \
        else MOE_PRE_P(16, 1024, XT, OT);                    \
    } while (0)
    if (x_elem == kF32) {
        if (out_elem == kF32) MOE_PRE(float, float);
        else MOE_PRE(float, bf16);
    } else {
        if (out_elem == kF32) MOE_PRE(bf16, float);
        else MOE_PRE(bf16, bf16);
    }
#undef MOE_PRE
#undef MOE_PRE_P
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_norm_post(const PostParams& p, cudaStream_t stream) {
    const int per = row_per(p.T, p.D), nthr = row_threads(p.D, per), rows = nthr == 32 ? 4 : 1;
    const dim3 grid((unsigned)cdiv(p.T, rows)), block(nthr * rows);
    auto bytes = [](int elem) { return elem == kF32 ? 4 : 2; };
    const bool has_next = p.next.kind != MOE_NORM_NONE;
    const bool vec = p.D % 8 == 0 && vec_ok(p.y, p.ld_y, bytes(p.y_elem)) && vec_ok(p.res, p.ld_res, bytes(p.r_elem)) &&
                     vec_ok(p.out, p.ld_out, bytes(p.r_elem)) && par_ok(p.norm) && par_ok(p.next) &&
                     (!has_next || vec_ok(p.next_out, p.ld_next, bytes(p.n_elem))) &&
                     (p.gate_by == MOE_GATE_NONE || p.gate_by == MOE_GATE_TOKEN ||
                      vec_ok(p.gate, p.gate_by == MOE_GATE_FULL ? p.ld_gate : 0, p.gate_bf16 ? 2 : 4));
    // (8192 x 512 with gate and next norm: 13.4 us row after row, 10.9 not; 16384 x 1024: 30.8 and 34.1)
    const bool rows_pay = p.y_elem == kBF16 && p.r_elem == kBF16 && p.D >= 1024;
    const int ring = kAhead * nthr * per * 4, many = vec && rows_pay ? rows_grid(p.T, nthr, ring) : 0;
    cudaError_t e = cudaSuccess;
#define MOE_POST_P(PER, MAXT, YT, RT, NT)                                                                              \
    do {                                                                                                         \
        if (many) {                                                                                              \
            if ((e = allow_smem(norm_post_rows_kernel<PER, MAXT, NT>, ring)) != cudaSuccess) return e;           \
            e = launch_kernel(norm_post_rows_kernel<PER, MAXT, NT>, dim3(many), dim3(nthr), ring, stream, 1, p, (const bf16*)p.y, (const bf16*)p.res, \
                                                                                 (bf16*)p.out, (NT*)p.next_out); \
        } else if (vec) {                                                                                        \
            e = launch_kernel(norm_post_kernel<8, PER, MAXT, YT, RT, NT>, dim3(grid), dim3(block), 0, stream, 1, p, (const YT*)p.y, (const RT*)p.res, (RT*)p.out, \
                                                                             (NT*)p.next_out, nthr);             \
        } else {                                                                                                 \
            e = launch_kernel(norm_post_kernel<1, PER, MAXT, YT, RT, NT>, dim3(grid), dim3(block), 0, stream, 1, p, (const YT*)p.y, (const RT*)p.res, (RT*)p.out, \
                                                                             (NT*)p.next_out, nthr);             \
        }                                                                                                        \
    } while (0)
#define MOE_POST(YT, RT, NT)                          \
    do {                                              \
        if (per == 8) MOE_POST_P(8, 1024, YT, RT, NT);            \
        else if (nthr <= 512) MOE_POST_P(16, 512, YT, RT, NT);    \
        else MOE_POST_P(16, 1024, YT, RT, NT);                    \
    } while (0)
#define MOE_POST_N(YT, RT)                                       \
    do {                                                         \
        if (p.n_elem == kF32) MOE_POST(YT, RT, float);           \
        else MOE_POST(YT, RT, bf16);                             \
    } while (0)
    if (p.y_elem == kF32) {
        if (p.r_elem == kF32) MOE_POST_N(float, float);
        else MOE_POST_N(float, bf16);
    } else {
        if (p.r_elem == kF32) MOE_POST_N(bf16, float);
        else MOE_POST_N(bf16, bf16);
    }
#undef MOE_POST_N
#undef MOE_POST
#undef MOE_POST_P
    count_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

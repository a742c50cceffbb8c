// Issue and waits of whole warps, for the kernels whose TMA and MMA warps run
// their loops with all lanes.
#pragma once

#include "tc_ptx.cuh"

namespace moe {
namespace tc {

__device__ __forceinline__ void st_cluster(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// One lane of the (converged) warp.  The TMA and MMA warps run their loops
// with all lanes and issue under this: the loop's values are then uniform,
// in the registers that the instructions take them from.  Issued from a
// single lane's own branch instead, an MMA costs 171 cycles whatever its
// size; so, 128 at 256 rows, 64 at 128.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.b32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p != 0;
}
// A bounded wait of the whole warp; the first to fail records where.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int64_t lim, volatile int* abort_flag, uint32_t* err, int where) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, lim, abort_flag));
    if (!ok && elect_one() && !*abort_flag) {
        record_error(err, MOE_ERR_DEVICE_TIMEOUT, where, blockIdx.x, 0);
        *abort_flag = 1;
    }
    return ok;
}

}  // namespace tc
}  // namespace moe

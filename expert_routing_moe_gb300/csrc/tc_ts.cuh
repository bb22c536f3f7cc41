// tc_ts.cuh -- what kernels share whose products have an operand in TMEM: the
// product, the wait for what was stored there, and waits of whole warps.
#pragma once

#include "common.cuh"
#include "tmap.h"

namespace moe {

__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16 (bf16 inputs, fp32 accumulate).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// A wait that is mostly over when it begins: the loop with the time limit stays out of the way.
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, moe_dev_status* st, int site) {
    return mbar_wait(bar, parity, abort_flag, st, site);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, moe_dev_status* st, int site) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    return __all_sync(kFull, wait_long(bar, parity, abort_flag, st, site));
}

}  // namespace moe

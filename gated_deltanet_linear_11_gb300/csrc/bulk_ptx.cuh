// bulk_ptx.cuh -- bulk copies into shared memory and bounded waits for them.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace gdn {

// Asynchronous copy of `bytes` (a multiple of 16; both addresses 16-byte aligned) from
// global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(tc::smem_u32(dst)), "l"(src), "r"(bytes), "r"(tc::smem_u32(bar)) : "memory");
}

constexpr uint64_t kCopyWaitNs = 2000000000ull;   // 2 s bound on any single wait

// mbarrier.try_wait with a hint of how long the thread may be suspended (20 us): a waiting
// warp then stays off the issue slots instead of polling.
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity), "r"(20000u) : "memory");
    return ok != 0;
}

// Wait for an mbarrier phase; false when it has not completed within the bound.
__device__ __forceinline__ bool wait_copy(uint64_t *bar, uint32_t parity) {
    if (try_wait_long(bar, parity)) return true;
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    do {
        if (try_wait_long(bar, parity)) return true;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    } while (t - t0 < kCopyWaitNs);
    return false;
}

// Two floats rounded to a bf16 pair (lo in the low half).
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace gdn

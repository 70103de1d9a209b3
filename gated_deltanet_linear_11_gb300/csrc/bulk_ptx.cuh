// bulk_ptx.cuh -- bulk copies into shared memory, bounded waits for them, and paired fp32
// and bf16 operations.
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

// Waits for an mbarrier phase; false when the bound has passed, or when *abort is set
// (another thread has given up; may be null).  SLEEP_NS = 0 polls, for waits on a kernel's
// critical chain; otherwise the warp sleeps between polls and leaves the issue slots to the
// others.  The clock is read every 64 polls only.
template <int SLEEP_NS>
__device__ __forceinline__ bool wait_bounded_poll(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0, t;
    for (uint32_t i = 1;; ++i) {
        if (SLEEP_NS > 0) __nanosleep(SLEEP_NS);
        if (tc::mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (abort && *abort) return false;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
            if (t0 == 0) t0 = t;
            if (t - t0 > kCopyWaitNs) return false;
        }
    }
}
__device__ __forceinline__ bool wait_copy(uint64_t *bar, uint32_t parity) {
    return wait_bounded_poll<0>(bar, parity, nullptr);
}

// Two fp32 operations in one instruction, rounded like the single ones.
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)),
          "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return d;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)),
          "l"(*reinterpret_cast<const unsigned long long *>(&b)),
          "l"(*reinterpret_cast<const unsigned long long *>(&c)));
    return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)),
          "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return d;
}

// Two floats rounded to a bf16 pair (lo in the low half).
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace gdn

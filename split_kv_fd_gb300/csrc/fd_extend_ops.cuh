// fd_extend_ops.cuh -- what the attention of new tokens asks of the hardware
// beside fd_device.cuh and fd_tc.cuh: a wait for phases that are mostly over,
// packed additions, and tensor-core issue by one lane of a converged warp.
#pragma once

#include "fd_device.cuh"
#include "fd_tc.cuh"

namespace fd {

// Bounded wait by a whole warp for a phase that is often complete already:
// one try first, and the clock is read only when that fails (a read of
// %globaltimer costs about as much as a short wait).
__device__ __forceinline__ bool mbar_wait_bounded_soon(uint32_t bar, uint32_t parity, uint32_t hint_ns,
                                                       const unsigned long long &limit_ns)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const unsigned long long t0 = global_ns();
        for (unsigned i = 0; i < WAIT_LIMIT_POLLS; ++i) {
            if (mbar_try_wait_hint(bar, parity, hint_ns)) {
                ok = true;
                break;
            }
            if (global_ns() - t0 > limit_ns)
                break;
        }
    }
    return __all_sync(FULL_MASK, ok);
}

// Two independent round-to-nearest fp32 additions (PTX add.rn.f32x2).
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// tc_mma_ss, tc_mma_ts and tc_commit by the one thread whose `pred` is set,
// as straight-line code: the other lanes of the warp run past it, so that the
// operands stay in uniform registers (inside a divergent branch each would be
// moved there one by one).
__device__ __forceinline__ void tc_mma_ss_if(uint32_t pred, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc), "r"(pred)
        : "memory");
}

__device__ __forceinline__ void tc_mma_ts_if(uint32_t pred, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc), "r"(pred)
        : "memory");
}

__device__ __forceinline__ void tc_commit_if(uint32_t pred, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(pred)
        : "memory");
}

// 1 in one lane of a converged warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

}  // namespace fd

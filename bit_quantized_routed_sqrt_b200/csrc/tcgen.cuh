// tcgen.cuh -- bounded barrier waits and wrappers of TMA loads and tcgen05 instructions
// (sm_100a inline PTX) shared by the tensor-core kernels.
#pragma once
#include <cuda.h>
#include "common.cuh"
#include "mbar.cuh"

namespace ds4 {

// Bounded wait for the completion of the barrier phase of the given parity (about two
// seconds); false on timeout (recorded) or when another role of the CTA gave up.  Roles off
// the critical path pass backoff_ns, so that while they wait they leave the issue slots to
// the dequantising warps.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort, int *status,
                                          int *dbg = nullptr, int who = 0, uint32_t iter = 0,
                                          unsigned backoff_ns = 0) {
    long long t0 = 0;
    for (int i = 0;; ++i) {
        if (mbar_try_spin(bar, parity)) return true;
        if (backoff_ns) __nanosleep(backoff_ns);
        if ((i & 15) == 15) {
            if (*abort) return false;
            const long long now = clock64();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > 4000000000ll) {
                set_status(status, ST_ETIMEOUT);
                if (dbg && atomicCAS(dbg, 0, 100 + who) == 0) {
                    dbg[1] = (int)iter;
                    dbg[2] = (int)parity;
                    dbg[3] = (int)(bar & 0xFFFF);
                    dbg[6] = blockIdx.x;
                    dbg[7] = threadIdx.x;
                }
                *abort = 1;
                return false;
            }
        }
    }
}
// Wait for copies or MMAs already issued by this CTA (they complete without any other
// role's help), ignoring the abort flag; bounded by about half a second.
__device__ __forceinline__ bool mbar_drain(uint32_t bar, uint32_t parity, int *status) {
    const long long t0 = clock64();
    for (int i = 0;; ++i) {
        if (mbar_try_spin(bar, parity)) return true;
        if ((i & 15) == 15 && clock64() - t0 > 1000000000ll) {
            set_status(status, ST_ETIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace ds4

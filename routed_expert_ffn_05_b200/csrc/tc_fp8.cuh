// tcgen05 helpers of the FP8 matrix products: the E4M3 MMA, tensor-memory loads
// tied to their wait, and a bounded wait that polls before it looks at a clock.
#pragma once

#include "tc.cuh"

namespace moe {

// D[M][N] (+)= A[M][K] . B[N][K]^T with K = 32 E4M3 elements, fp32 accumulate
// in TMEM; A and B in shared memory (descriptors).
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same for a pair of CTAs (cluster ranks 2 i and 2 i + 1), M = 256: each CTA
// holds 128 rows of A, half of the rows of B and 128 rows of D (all N columns),
// at the same shared and tensor-memory addresses. Issued by the even CTA only.
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives once on `bar` of both CTAs when the pair's MMAs issued so far by this
// thread have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// Tensor-memory allocation of a pair: one warp of each CTA calls these.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// TMA tile load (no multicast) into this CTA's shared memory, completing on the
// barrier at the cluster address `bar` of this CTA or its pair.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const void *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// Arrival on an mbarrier of another CTA of the cluster. CTA scope: it hands
// tensor memory on, whose loads have been waited for, and no other data
// (a release at cluster scope took about 900 cycles more, measured).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Instruction descriptor of kind::f8f6f4 with E4M3 A and B (format 0, both
// K-major) and an fp32 accumulator (D format 1).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// Thread i of the warp reads TMEM lane (lane field of taddr) + i, 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Waits for the warp's tensor-memory loads, tied to the registers a load fills:
// nothing that uses them can be scheduled ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}

// True for one lane of a converged warp. The compiler then knows that one thread
// runs what follows, so the operands of TMA and tcgen05 instructions (uniform
// registers) need no loop over the active lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A bounded wait with an abort flag (see mbar_wait) for the waits inside a K
// loop; barrier and flag by their shared-memory addresses. Its shape matters:
// with the first try outside the loop and a flag instead of returns, a wait that
// is already satisfied measured 57 cycles on this part; a loop around the first
// try, or returns inside it, 120 to 300 (one try alone: 47). The clock and the
// abort flag are looked at every 256 tries.
__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_poll_at(uint32_t bar, uint32_t parity, uint32_t abort, uint64_t limit_ns) {
    bool ok = mbar_try_wait_at(bar, parity);
    int n = 0;
    uint64_t t0 = 0;
#pragma unroll 1
    while (!ok && n >= 0) {
        ok = mbar_try_wait_at(bar, parity);
        if ((++n & 255) == 0) {
            const uint64_t now = globaltimer_ns();
            if (n == 256) t0 = now;
            uint32_t stop;
            asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(stop) : "r"(abort) : "memory");
            if (stop || now - t0 > limit_ns) n = -1;
        }
    }
    return ok;
}
__device__ __forceinline__ bool mbar_poll(uint64_t *bar, uint32_t parity, const volatile int *abort, uint64_t limit_ns) {
    return mbar_poll_at(smem_u32(bar), parity, smem_u32(const_cast<const int *>(abort)), limit_ns);
}

}  // namespace moe

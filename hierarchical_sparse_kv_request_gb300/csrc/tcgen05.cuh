// tcgen05.cuh -- the fifth-generation tensor core from inline PTX: tensor
// memory, matrix descriptors, MMA issue, and mbarriers with bounded waits.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace hs {

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// One thread of a converged warp, always the same.  MMAs are issued under this
// rather than under a lane test: the compiler then keeps their descriptors in
// uniform registers (measured, M = N = 64: 32 cycles an MMA against 45).
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "elect.sync _|p, 0xffffffff;\n"
                 "selp.u32 %0, 1, 0, p;\n"
                 "}"
                 : "=r"(ok));
    return ok != 0;
}

// ---- mbarriers ---------------------------------------------------------------

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrives, and `bytes` more have to come before the phase ends.
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 "selp.u32 %0, 1, 0, p;\n"
                 "}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// The long part of a wait, kept out of line: the attention kernel's loops have
// to stay in the instruction cache.
__device__ __noinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int *gave_up)
{
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try(bar, parity)) return true;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (*gave_up || t - t0 > 1000000000ull) {
            *gave_up = 1;
            return false;
        }
    }
}

// Wait for the phase with this parity, for at most about a second; false if
// it did not come or another thread of the CTA gave up (*gave_up).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up)
{
    return mbar_try(bar, parity) || mbar_wait_long(bar, parity, gave_up);
}

// This thread's shared-memory writes become visible to the tensor core.
__device__ __forceinline__ void fence_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory -------------------------------------------------------------

// Whole warp: all 512 columns; the address goes to *at (shared memory).
__device__ __forceinline__ void tmem_alloc_all(uint32_t at)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(at) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free_all(uint32_t tmem)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define HS_R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define HS_I4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
#define HS_REGS32                                                                    \
    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"    \
    "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}"

// 16 lanes x 64 columns: v[4 * j + {0, 1}] is row lane / 4, columns 8 * j +
// 2 * (lane % 4) + {0, 1}; v[4 * j + {2, 3}] the same columns of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t at, uint32_t (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 " HS_REGS32 ", [%32];"
                 : HS_R4(v, 0), HS_R4(v, 4), HS_R4(v, 8), HS_R4(v, 12), HS_R4(v, 16), HS_R4(v, 20),
                   HS_R4(v, 24), HS_R4(v, 28)
                 : "r"(at));
}

__device__ __forceinline__ void tmem_st_16x64(uint32_t at, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.16x256b.x8.b32 [%32], " HS_REGS32 ";" ::HS_I4(v, 0), HS_I4(v, 4),
                 HS_I4(v, 8), HS_I4(v, 12), HS_I4(v, 16), HS_I4(v, 20), HS_I4(v, 24), HS_I4(v, 28), "r"(at)
                 : "memory");
}

// The same for 8 and for 32 columns.
__device__ __forceinline__ void tmem_ld_16x8(uint32_t at, uint32_t (&v)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];" : HS_R4(v, 0) : "r"(at));
}

__device__ __forceinline__ void tmem_st_16x32(uint32_t at, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::HS_I4(v, 0),
                 HS_I4(v, 4), HS_I4(v, 8), HS_I4(v, 12), "r"(at)
                 : "memory");
}

// ---- MMA ----------------------------------------------------------------------

// Shared-memory matrix descriptor, 128-byte swizzle (tiles of 8 rows of 128
// bytes, 1024-byte aligned).  K-major: sbo is the distance between groups of
// 8 rows, lbo unused.  MN-major (rows of 64 consecutive M/N elements, one
// per k): sbo is the distance between groups of 8 k, lbo between blocks of 64
// M/N elements.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16 with f32 accumulators: bf16 or f16
// operands (both the same), B K-major or MN-major, A K-major.
__host__ __device__ constexpr uint32_t mma_desc(int M, int N, bool bf16, bool b_mn_major)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D (tensor memory) = A B (+ D if accumulate); one thread.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
                 "}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

// The same with A in tensor memory: for M = 64, row i in lane 32 (i / 16) + i %
// 16, columns of two 16-bit values each.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
                 "}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

// Arrive on the mbarrier once every MMA this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace hs

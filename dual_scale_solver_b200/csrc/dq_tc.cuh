// dq_tc.cuh — the tcgen05, TMEM and mbarrier instructions that the prompt
// attention kernel is written in, one wrapper each (fp16 operands, one CTA).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dq_device.cuh"

namespace dq {
namespace tc {

constexpr uint64_t kWaitLimitNs = 1000000000ull;   // a wait gives up after 1 s

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// ---- mbarriers
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t addr, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; "
                 "selp.u32 %0, 1, 0, p; }"
                 : "=r"(done) : "r"(addr), "r"(parity) : "memory");
    return done != 0;
}
// Bounded wait for the phase of the given parity.  False if another thread of
// the CTA gave up, or (raising the device flag and the CTA's abort flag) if
// this wait ran past its limit.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, volatile int *abort,
                                         unsigned int *status) {
    const uint32_t addr = smem_addr(b);
    if (bar_test(addr, parity)) return true;
    const uint64_t t0 = now_ns();
    while (true) {
        if (bar_test(addr, parity)) return true;
        if (*abort) return false;
        if (now_ns() - t0 > kWaitLimitNs) break;
    }
    *abort = 1;
    atomicOr(status, STATUS_TIMEOUT);
    return false;
}

// ---- ordering
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// this thread's shared-memory stores before later tensor-core reads
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// arrive on the barrier once this thread's earlier MMAs are done
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_addr(bar)) : "memory");
}

// One lane of a converged warp (the same one each time).  MMAs and commits are
// issued under it by a warp that computes their operands together, so that
// they stay in uniform registers.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// ---- operands.  Tiles of fp16 in shared memory are blocks of 64 contiguous
// elements (128 bytes, 128-byte swizzle) by rows, 8-row groups 1024 bytes
// apart.
// Rows along M or N, the contiguous dimension along K (K-major).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Rows along K, the contiguous dimension along N (MN-major); `block` bytes
// from one block of 64 N to the next.
__device__ __forceinline__ uint64_t desc_n_major(uint32_t addr, uint32_t block) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}
// fp16 x fp16 -> float32, M x N; b_n_major: B is MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_n_major) {
    return (1u << 4) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}
// A from TMEM
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}

// ---- TMEM: 32 consecutive 32-bit columns of this thread's lane
#define DQ_TC_W32(c, r)                                                                                \
    c((r)[0]), c((r)[1]), c((r)[2]), c((r)[3]), c((r)[4]), c((r)[5]), c((r)[6]), c((r)[7]), c((r)[8]), \
        c((r)[9]), c((r)[10]), c((r)[11]), c((r)[12]), c((r)[13]), c((r)[14]), c((r)[15]),             \
        c((r)[16]), c((r)[17]), c((r)[18]), c((r)[19]), c((r)[20]), c((r)[21]), c((r)[22]),            \
        c((r)[23]), c((r)[24]), c((r)[25]), c((r)[26]), c((r)[27]), c((r)[28]), c((r)[29]),            \
        c((r)[30]), c((r)[31])
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
        "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : DQ_TC_W32("=r", r) : "r"(addr));
}
// the registers of earlier loads are valid after it (and not used before it)
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : DQ_TC_W32("+r", r) :: "memory");
}
// 8 columns
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :: "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_store_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
template <uint32_t COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t *base) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(base)), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <uint32_t COLS>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(COLS) : "memory");
}

}  // namespace tc
}  // namespace dq

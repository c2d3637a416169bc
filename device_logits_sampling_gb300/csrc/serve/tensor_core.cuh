// Barriers in shared memory, tensor memory and the 5th-generation tensor cores: what the kernels that use them share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace arcs {

constexpr int kWaits = 1 << 24;  // tries of a wait before it gives up

__device__ __forceinline__ uint32_t shared_of(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_of(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_of(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_of(b)), "r"(bytes) : "memory");
}
// Waits for the phase; gives up after kWaits tries, or when another role has.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, uint32_t* failed) {
    const uint32_t p = shared_of(b);
    for (int i = 0; i < kWaits; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(p), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 1023) == 1023 && *static_cast<volatile uint32_t*>(failed)) return false;
    }
    *static_cast<volatile uint32_t*>(failed) = 1;
    return false;
}
// The same by a warp, all lanes together.
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, uint32_t* failed) {
    return __all_sync(0xFFFFFFFFu, bar_wait(b, parity, failed));
}
// One look at the barrier, whose answer may come while other work is issued.
__device__ __forceinline__ uint32_t bar_done(uint64_t* b, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(shared_of(b)), "r"(parity)
                 : "memory");
    return done;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit_to(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(shared_of(b)) : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Both operands in shared memory.
__device__ __forceinline__ void mma_f16_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Contiguous bytes into shared memory; both addresses and the count are multiples of 16.
__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(shared_of(bar))
                 : "memory");
}
// Read-only bytes that are used once: nothing of them stays in L1, which is what shared memory leaves of it.
__device__ __forceinline__ uint4 load_past_l1(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// Plain stores to shared memory before what the tensor cores read.
__device__ __forceinline__ void fence_operands() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
#define ARC_REGS8(x, o) "r"(x[o]), "r"(x[o + 1]), "r"(x[o + 2]), "r"(x[o + 3]), "r"(x[o + 4]), "r"(x[o + 5]), "r"(x[o + 6]), "r"(x[o + 7])
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        ARC_REGS8(x, 0), ARC_REGS8(x, 8)
        : "memory");
}
#undef ARC_REGS8
#define ARC_OUT8(x, o) "=r"(x[o]), "=r"(x[o + 1]), "=r"(x[o + 2]), "=r"(x[o + 3]), "=r"(x[o + 4]), "=r"(x[o + 5]), "=r"(x[o + 6]), "=r"(x[o + 7])
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : ARC_OUT8(x, 0), ARC_OUT8(x, 8)
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : ARC_OUT8(x, 0), ARC_OUT8(x, 8), ARC_OUT8(x, 16), ARC_OUT8(x, 24)
        : "r"(at)
        : "memory");
}
#undef ARC_OUT8
// The wait, with the loaded registers as its own: nothing that reads them comes before it.
#define ARC_BOTH8(x, o) "+r"(x[o]), "+r"(x[o + 1]), "+r"(x[o + 2]), "+r"(x[o + 3]), "+r"(x[o + 4]), "+r"(x[o + 5]), "+r"(x[o + 6]), "+r"(x[o + 7])
__device__ __forceinline__ void tmem_wait_load32(uint32_t (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : ARC_BOTH8(x, 0), ARC_BOTH8(x, 8), ARC_BOTH8(x, 16), ARC_BOTH8(x, 24)
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_load16(uint32_t (&x)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : ARC_BOTH8(x, 0), ARC_BOTH8(x, 8) : : "memory");
}
#undef ARC_BOTH8
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float half_of(uint64_t v, int i) {
    return __uint_as_float(static_cast<uint32_t>(i ? v >> 32 : v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// K-major operand in shared memory, rows of 128 bytes in swizzled groups of
// eight: start address, 1,024 bytes from group to group, 128-byte swizzle.
__device__ __forceinline__ uint64_t operand_at(uint32_t shared) {
    return static_cast<uint64_t>((shared & 0x3FFFFu) >> 4) | (uint64_t{1} << 16) | (uint64_t{1024 >> 4} << 32) |
           (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// The same memory read along the other dimension (groups of eight rows are the inner dimension): `block` bytes from 64
// values of the outer dimension to the next 64.
__device__ __forceinline__ uint64_t operand_across(uint32_t shared, uint32_t block) {
    return static_cast<uint64_t>((shared & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(block >> 4) << 16) |
           (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

}  // namespace arcs

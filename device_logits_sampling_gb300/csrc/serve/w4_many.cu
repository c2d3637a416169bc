// 9 .. 256 rows of x times 4-bit weights, on the 5th-generation tensor cores.
//
// Mathematics.  128 weight rows are the long side of a product (operand A), up
// to 128 rows of x the other (B, in shared memory).  A code masked out of its
// word is the fp16 subnormal q * 2^-24 (one nibble up: 16 q * 2^-24, with x
// divided by 16 beforehand); the zero point is subtracted in the same form,
// exactly, and x is fp16 after a power-of-two scaling of each row.  Group
// scales stay out of the products: each group's fp32 sum is read back and
// multiplied by its scale in fp32.
//
// Where things lie.  A never touches shared memory: a thread owns one weight
// row, unpacks 128 values of it into 64 registers and stores them to tensor
// memory, which is where the product reads A.  The order of the inner
// dimension inside a product is free, so the unpacked pairs stay as the masks
// give them and x is laid out to match, once a call, by a small kernel that
// also swizzles it: a stage of x is one contiguous bulk copy.  A group's sums
// lie in tensor memory with the weight row as the lane, so its scale is one
// number a thread and the running sums are the thread's registers.
//
// Roles of a block: one or two groups of four warps add up group sums (and store
// the output), each its share of the columns; two or four groups of four copy and
// unpack weights, taking turns; a warp issues the products and one copies x.  They meet at barriers in shared memory: rings of unpacked A, of x and of group
// sums, so that copying, unpacking, multiplying and adding up overlap across
// groups and tiles.  Few tiles: the inner dimension is split over a cluster
// whose blocks add each other's sums through distributed shared memory.
//
// Every wait has a limit; a block whose wait runs out writes NaN.
//
// Bounds and figures (129,280 x 4,096, groups of 128).  256 rows: 184 us, 1,470
// TFLOP/s, 78% of the measured bf16 rate; what is left is the round from a
// group's sums back to the product that takes their place, about 1,600 clocks
// over three slots.  128 rows: 118 us, the adders' share.  16 rows: 82 us, 3.4
// TB/s; a block of 128 x 128 takes 700 clocks of adding and unpacking against
// 350 of memory time.  Measured and left: products predicated on the thread's
// index rather than elect.sync (222 us at 16 rows), one lane polling for a warp
// (no change), 256 rows as two passes (427 us), outputs stored with their
// factors loaded one by one (295 us).
#include <atomic>
#include <climits>
#include <cstdint>
#include <cstring>

#include "launch_util.cuh"
#include "serve_util.cuh"
#include "w4_many.cuh"

namespace arcs {
namespace {

constexpr int kInner = 128;    // inner values of a block of A and x
constexpr int kRawStage = 32 * 128;  // bytes of a warp's raw stage: 32 rows of 256 codes
constexpr int kWaits = 1 << 24;

// N: rows of x of a product (16, 32, 64 or 128). H: products that share A: 2
// for more than 128 rows, so that weights are unpacked once for 256 of them.
template <int N, int H>
struct Many {
    // 64 columns and more are added up by two groups of warps, each half of the columns: one took 1,100 clocks
    // for the 128 sums of a row, the products 512
    static constexpr int kAdders = N >= 64 ? 2 : 1;
    // few columns: unpacking is what a block waits for, so four groups of warps do it
    static constexpr int kUnpackers = N <= 32 ? 4 : 2;
    static constexpr int kThreads = (kAdders + kUnpackers + 1) * 128;
    static constexpr int kCols = N * H / kAdders;        // columns of a group of warps
    // registers of a thread once the roles part, of 96 at the launch of 640 threads (5 * 96 = 480)
    static constexpr int kAddRegs = H == 2 ? 160 : 128, kUnpackRegs = H == 2 ? 64 : 88, kIssueRegs = H == 2 ? 32 : 40;
    static_assert(kAdders == 1 || 2 * kAddRegs + 2 * kUnpackRegs + kIssueRegs <= 480, "registers of the launch");
    static constexpr int kSums = H == 2 ? 3 : N == 128 ? 2 : 4;  // ring of group sums, N columns each
    static constexpr int kA = H == 2 ? 2 : 4;            // ring of unpacked A, 64 columns each
    static constexpr int kX = H == 2 ? 2 : N == 128 ? 3 : 4;     // ring of x
    static constexpr int kRaw = H == 2 ? 2 : N == 128 || N <= 32 ? 3 : 4;  // a warp's ring of raw weights
    static constexpr int kColumns = 512;                 // tensor memory taken
    static constexpr int kXHalf = N * kInner * 2, kXBytes = H * kXHalf;
    static constexpr int kRawBytes = 4 * kUnpackers * kRaw * kRawStage;
    static constexpr int kJoin = H * N * 128 * 4;        // over the rings, at the end
    static constexpr int kRings = kX * kXBytes + kRawBytes;
    static constexpr int kSmem = (kRings > kJoin ? kRings : kJoin) + 1024;
};

struct Bars {
    uint64_t a_full[4], a_empty[4];
    uint64_t x_full[4], x_empty[4];
    uint64_t s_full[4], s_empty[4];
    uint64_t drained;  // the products issued before a wait ran out
    uint32_t tmem;
    uint32_t failed;
    float back[256];  // each row of x's factor
};

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
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int C>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(C) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
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

// K-major operand in shared memory, rows of 128 bytes in swizzled groups of
// eight: start address, 1,024 bytes from group to group, 128-byte swizzle.
__device__ __forceinline__ uint64_t operand_at(uint32_t shared) {
    return static_cast<uint64_t>((shared & 0x3FFFFu) >> 4) | (uint64_t{1} << 16) | (uint64_t{1024 >> 4} << 32) |
           (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <class T>
__device__ __forceinline__ T as_output(float v);
template <>
__device__ __forceinline__ float as_output<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 as_output<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half as_output<__half>(float v) { return __float2half_rn(v); }

// A weight row's sums for C rows of x: 32 rows of a warp are neighbours in y.
template <class T, int C>
__device__ __forceinline__ void store_sums(const ManyArgs& a, const float* back, const uint64_t (&y)[C / 2], int m0, int64_t n) {
    T* out = static_cast<T*>(a.y) + m0 * a.y_stride + n;
    const int left = a.rows - m0;
    if (left >= C) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            *out = as_output<T>(half_of(y[i / 2], i & 1) * 0x1p24f * back[m0 + i]);
            out += a.y_stride;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (i < left) *out = as_output<T>(half_of(y[i / 2], i & 1) * 0x1p24f * back[m0 + i]);
            out += a.y_stride;
        }
    }
}

// The products of all items, by one thread: for each block of 128 inner values
// its groups, each into the next slot of the ring of sums. False where a wait ran out.
template <int N, int H, int G>
__device__ __forceinline__ bool issue_products(Bars& bars, uint32_t x_ring, uint32_t tmem, uint32_t tmem_a, int first, int step,
                                               int items, int nb) {
    using M = Many<N, H>;
    constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(N / 8) << 17) | (8u << 24);
    constexpr int kSteps = G / 16;
    const uint64_t x0 = operand_at(x_ring);
    uint32_t buf = 0, buf_phase = 0, xs = 0, xs_phase = 0, slot = 0, slot_phase = 1;
    // a look at a barrier takes 240 clocks beside the copies and loads of the other warps, even at a finished
    // phase: the next block's are under way while this block's products are issued
    uint32_t a_ready = 0, x_ready = 0, s_ready = 0;
    for (int item = first; item < items; item += step)
        for (int b = 0; b < nb; ++b) {
            if (!a_ready && !bar_wait(&bars.a_full[buf], buf_phase, &bars.failed)) return false;
            if (!x_ready && !bar_wait(&bars.x_full[xs], xs_phase, &bars.failed)) return false;
            // addresses count 16 bytes
            const uint64_t x_at = x0 + xs * (M::kXBytes / 16);
            const uint32_t a_at = tmem_a + buf * 64;
#pragma unroll
            for (int gh = 0; gh < kInner / G * H; ++gh) {
                const int g = gh / H, h = gh % H;
                if (!s_ready && !bar_wait(&bars.s_empty[slot], slot_phase, &bars.failed)) return false;
                fence_after();
                const uint32_t d = tmem + slot * N;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int kk = g * kSteps + k;  // of the block's eight
                    mma_f16(d, a_at + kk * 8, x_at + h * (M::kXHalf / 16) + (kk >> 2) * (N * 128 / 16) + (kk & 3) * 2, idesc, k != 0);
                }
                commit_to(&bars.s_full[slot]);
                if (++slot == M::kSums) {
                    slot = 0;
                    slot_phase ^= 1;
                }
                s_ready = bar_done(&bars.s_empty[slot], slot_phase);
            }
            commit_to(&bars.a_empty[buf]);
            commit_to(&bars.x_empty[xs]);
            if (++buf == M::kA) {
                buf = 0;
                buf_phase ^= 1;
            }
            if (++xs == M::kX) {
                xs = 0;
                xs_phase ^= 1;
            }
            a_ready = bar_done(&bars.a_full[buf], buf_phase);
            x_ready = bar_done(&bars.x_full[xs], xs_phase);
        }
    return true;
}

// ------------------------------------------------------------------ x
// One block for each row (and each row of padding): fp16, scaled by a power of
// two to [2^14, 2^15), in the order of the unpacked pairs: a word of eight
// codes k0 .. k7 gives (k0, k4), (k2, k6) and, times 16, (k1, k5), (k3, k7).
template <int DT>
__global__ void __launch_bounds__(256) many_x_kernel(const __grid_constant__ ManyArgs a) {
    __shared__ uint32_t red[8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row = blockIdx.x, tid = threadIdx.x;
    const int block_rows = a.columns, half = row / block_rows, in = row % block_rows;
    const bool real = row < a.rows;
    const char* x = static_cast<const char*>(a.x) + row * a.x_stride * 2;
    const int units = a.ins / 8, all = a.blocks * (kInner / 8);
    float top = 0.0f;
    if (real)
        for (int u = tid; u < units; u += 256) {
            float v[8];
            load8<DT>(x + u * 16, a.x_vec, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float z = fabsf(v[i]);
                if (z <= 3.4028235e38f) top = fmaxf(top, z);  // the largest finite one
            }
        }
    const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, red[i]);
    const int ex = static_cast<int>(m >> 23) - 127;
    const int e = m == 0 ? 0 : (14 - ex > 120 ? 120 : 14 - ex);
    const float up = exp2i(e);
    if (tid == 0) a.x_back[row] = exp2i(-e);
    uint8_t* const out = static_cast<uint8_t*>(a.x_ready) + static_cast<size_t>(half) * a.blocks * block_rows * (kInner * 2);
    for (int u = tid; u < all; u += 256) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (real && u < units) load8<DT>(x + u * 16, a.x_vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= up;
        const __half2 h[4] = {__floats2half2_rn(v[0], v[4]), __floats2half2_rn(v[2], v[6]),
                              __floats2half2_rn(v[1] * 0.0625f, v[5] * 0.0625f),
                              __floats2half2_rn(v[3] * 0.0625f, v[7] * 0.0625f)};
        // 64 values of all rows, 128 bytes a row, its 16-byte chunks swizzled by the row
        const size_t at = (static_cast<size_t>(u >> 3) * block_rows + in) * 128 + (((u & 7) ^ (in & 7)) * 16);
        *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(h);
    }
}

// ------------------------------------------------------------------ products
template <int N, int H>
__global__ void __launch_bounds__(Many<N, H>::kThreads, 1) many_kernel(const __grid_constant__ ManyArgs a) {
    using M = Many<N, H>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ Bars bars;
    uint8_t* const dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
    constexpr int kUnpack = M::kAdders * 4, kIssue = kUnpack + 4 * M::kUnpackers;  // first warps of the roles
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x) % a.cluster;
    const int first = static_cast<int>(blockIdx.x) / a.cluster, step = static_cast<int>(gridDim.x) / a.cluster;
    const int items = a.tiles;
    // blocks of the inner dimension that this block takes
    const int b0 = static_cast<int>(static_cast<int64_t>(a.blocks) * rank / a.cluster);
    const int nb = static_cast<int>(static_cast<int64_t>(a.blocks) * (rank + 1) / a.cluster) - b0;
    const int per = kInner / a.group;  // groups of a block
    uint8_t* const x_ring = dyn;
    uint8_t* const raw_ring = dyn + M::kX * M::kXBytes;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            bar_init(&bars.a_full[i], 4);
            bar_init(&bars.a_empty[i], 1);
            bar_init(&bars.x_full[i], 1);
            bar_init(&bars.x_empty[i], 1);
            bar_init(&bars.s_full[i], 1);
            bar_init(&bars.s_empty[i], H == 2 ? 4 : 4 * M::kAdders);
        }
        bar_init(&bars.drained, 1);
        bars.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kIssue) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_of(&bars.tmem)),
                     "n"(M::kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem, tmem_a = tmem + M::kSums * N;

    if (warp >= kUnpack && warp < kIssue) {
        // ---- unpack: a thread for each weight row; the U groups take blocks in turn, counted over all items, so
        // that none waits for a buffer more than one use behind another.  A raw stage holds two of a group's
        // blocks: 64 bytes of each row, and 64 bytes 64 U further on.
        constexpr int U = M::kUnpackers;
        static_assert(U <= M::kA, "a group's next block must not be two uses of a buffer past its last");
        if constexpr (M::kAdders == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(M::kUnpackRegs));
        const int w = warp & 3, turn = (warp - kUnpack) >> 2;
        const uint32_t ring = shared_of(raw_ring) + (warp - kUnpack) * M::kRaw * kRawStage;
        const uint8_t* const ring_p = raw_ring + (warp - kUnpack) * M::kRaw * kRawStage;
        const int end = (b0 + nb) * kInner < a.ins ? (b0 + nb) * kInner : a.ins;
        const int cc = lane & 7;  // the lane's chunk, of the rows lane / 8, + 4, ...
        const uint32_t copy_to = ring + (lane >> 3) * 128 + ((cc ^ (lane >> 3)) * 16);
        int c_item = first, c_block = turn, c_stage = 0;  // the next raw stage's item and first block
        auto issue = [&]() {
            while (c_block >= nb && c_item < items) {  // the group's next block, of a later item
                c_block = (c_block - nb) & (U - 1);
                c_item += step;
            }
            if (c_item < items) {
                const int64_t n0 = static_cast<int64_t>(c_item) * 128 + w * 32 + (lane >> 3);
                const int b = c_block + (cc >> 2) * U;
                const int k = (b0 + b) * kInner + (cc & 3) * 32;  // first inner value of the lane's chunk
                const bool inner = b < nb && k < end;
                const char* src = static_cast<const char*>(a.q) + n0 * a.row_bytes + k / 2;
                const uint32_t to = copy_to + c_stage * kRawStage;
                const bool whole = inner && n0 + 28 < a.outs;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // (a row four further on changes the third bit of its permutation)
                    const bool on = whole || (inner && n0 + 4 * i < a.outs);
                    copy16((to ^ ((i & 1) * 64)) + i * 512, on ? src : static_cast<const char*>(a.q), on);
                    src += 4 * a.row_bytes;
                }
                c_block += 2 * U;
            }
            copies_end();
            c_stage = c_stage + 1 == M::kRaw ? 0 : c_stage + 1;
        };
        for (int i = 0; i < M::kRaw - 1; ++i) issue();
        int stage = 0;
        uint32_t before = 0;  // blocks of the items before
        bool ok = true;
        for (int item = first; ok && item < items; item += step, before += nb) {
            int block = (turn - before) & (U - 1);
            const int64_t n = static_cast<int64_t>(item) * 128 + w * 32 + lane;
            const uint8_t* zero_at = a.zeros && n < a.outs ? a.zeros + n * a.groups : nullptr;
            // the zero points of a block's groups, one a byte; loaded a raw stage ahead
            auto zeros_of = [&](int g) {
                uint32_t z = 0x08080808u;
                if (zero_at) {
                    z = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < per && g + i < a.groups) z |= static_cast<uint32_t>(__ldg(zero_at + g + i)) << (8 * i);
                }
                return z;
            };
            uint32_t z_now[2], z_next[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) z_next[h] = zeros_of((b0 + block + U * h) * per);
            for (; ok && block < nb; block += 2 * U) {
                copies_wait<M::kRaw - 2>();
                __syncwarp();
                issue();
                const uint8_t* row = ring_p + stage * kRawStage + lane * 128;
                stage = stage + 1 == M::kRaw ? 0 : stage + 1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    z_now[h] = z_next[h];
                    z_next[h] = zeros_of((b0 + block + 2 * U + U * h) * per);
                }
#pragma unroll 1
                for (int h = 0; h < 2 && block + U * h < nb; ++h) {
                    const uint32_t used = before + block + U * h;
                    const int buf = used % M::kA;
                    uint4 q[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) q[c] = *reinterpret_cast<const uint4*>(row + (((4 * h + c) ^ (lane & 7)) * 16));
                    ok = warp_wait(&bars.a_empty[buf], ((used / M::kA) & 1) ^ 1, &bars.failed);
                    if (!ok) break;
                    fence_after();
                    const uint32_t zs = h ? z_now[1] : z_now[0];
#pragma unroll
                    for (int ci = 0; ci < 4; ++ci) {  // chunks of 32 values
                        uint32_t v[16];
                        {
                            const uint32_t z = (zs >> (8 * (ci * per / 4))) & 0xFFu;
                            const uint32_t z_lo = z | (z << 16), z_hi = z_lo << 4;
                            const uint32_t ws[4] = {q[ci].x, q[ci].y, q[ci].z, q[ci].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t u = ws[i] >> 8;
                                v[4 * i] = sub2(ws[i] & 0x000F000Fu, z_lo);
                                v[4 * i + 1] = sub2(u & 0x000F000Fu, z_lo);
                                v[4 * i + 2] = sub2(ws[i] & 0x00F000F0u, z_hi);
                                v[4 * i + 3] = sub2(u & 0x00F000F0u, z_hi);
                            }
                        }
                        tmem_store16(tmem_a + (static_cast<uint32_t>(w * 32) << 16) + buf * 64 + ci * 16, v);
                    }
                    tmem_wait_store();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&bars.a_full[buf]);
                }
            }
        }
        copies_wait<0>();
    } else if (warp >= kIssue) {
        // one instruction for the four warps that share it
        if constexpr (M::kAdders == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(M::kIssueRegs));
        if (warp == kIssue && elect_one()) {
            // ---- products
            const uint32_t x_at = shared_of(x_ring);
            const bool ok = a.group == 128  ? issue_products<N, H, 128>(bars, x_at, tmem, tmem_a, first, step, items, nb)
                            : a.group == 64 ? issue_products<N, H, 64>(bars, x_at, tmem, tmem_a, first, step, items, nb)
                                            : issue_products<N, H, 32>(bars, x_at, tmem, tmem_a, first, step, items, nb);
            if (!ok) {  // a failed block's products end before its memory goes away
                commit_to(&bars.drained);
                uint32_t quiet = 0;
                bar_wait(&bars.drained, 0, &quiet);
            }
        }
        if (warp == kIssue + 1 && elect_one()) {
            // ---- x
            asm volatile("griddepcontrol.wait;" ::: "memory");
            uint32_t used = 0;
            bool ok = true;
            for (int item = first; ok && item < items; item += step) {
                const uint8_t* src = static_cast<const uint8_t*>(a.x_ready) + static_cast<size_t>(b0) * M::kXHalf;
                for (int b = 0; b < nb; ++b, ++used) {
                    const int xs = used % M::kX;
                    ok = bar_wait(&bars.x_empty[xs], ((used / M::kX) & 1) ^ 1, &bars.failed);
                    if (!ok) break;
                    bar_expect(&bars.x_full[xs], M::kXBytes);
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        asm volatile(
                            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                shared_of(x_ring) + xs * M::kXBytes + h * M::kXHalf),
                            "l"(src + (static_cast<size_t>(h) * a.blocks + b) * M::kXHalf), "r"(M::kXHalf),
                            "r"(shared_of(&bars.x_full[xs]))
                            : "memory");
                }
            }
            // a failed block still waits for its copies in flight before its memory goes away
            if (!ok)
                for (int i = 0; i < M::kX && used > 0; ++i) {
                    const uint32_t u = used - 1 - i;
                    if (u >= used) break;
                    uint32_t quiet = 0;
                    bar_wait(&bars.x_full[u % M::kX], (u / M::kX) & 1, &quiet);
                }
        }
        __syncwarp();
    } else {
        // ---- group sums: a thread for each weight row
        if constexpr (M::kAdders == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(M::kAddRegs));
        constexpr int C = M::kCols;
        const int who = warp >> 2, c0 = who * C, row = tid & 127;  // its columns, its weight row
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // with two products the sums of each are a slot of their own, in turn
        for (int i = tid; i < H * N; i += M::kAdders * 128) bars.back[i] = a.x_back[i];
        asm volatile("bar.sync 1, %0;" ::"n"(M::kAdders * 128) : "memory");
        uint32_t sums = H == 2 ? who : 0;
        bool ok = true;
        for (int item = first; item < items; item += step) {
            const int64_t n = static_cast<int64_t>(item) * 128 + row;
            const uint16_t* scale_at = static_cast<const uint16_t*>(a.scales) + (n < a.outs ? n : 0) * a.groups;
            auto scales_of = [&](int g) {  // eight of them ahead
                uint4 s = make_uint4(0u, 0u, 0u, 0u);
                if (g < a.groups) {
                    if (a.s_vec) {
                        s = __ldg(reinterpret_cast<const uint4*>(scale_at + g));
                    } else {
                        uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (g + i < a.groups) b[i >> 1] |= static_cast<uint32_t>(__ldg(scale_at + g + i)) << (16 * (i & 1));
                        s = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                }
                return s;
            };
            uint64_t y[C / 2];  // pairs of columns
#pragma unroll
            for (int i = 0; i < C / 2; ++i) y[i] = 0;
            int gi = b0 * per;
            uint4 now = scales_of(gi & ~7), next = scales_of((gi & ~7) + 8);
            auto shift = [&]() {
                now.x = __funnelshift_r(now.x, now.y, 16);
                now.y = __funnelshift_r(now.y, now.z, 16);
                now.z = __funnelshift_r(now.z, now.w, 16);
                now.w >>= 16;
            };
            for (int i = 0; i < (gi & 7); ++i) shift();
            const int end = gi + nb * per;
            for (; ok && gi < end; sums += H) {
                const uint32_t bits = now.x & 0xFFFFu;
                const float s = a.x_bf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(bits));
                shift();
                if ((++gi & 7) == 0) {
                    now = next;
                    next = scales_of(gi + 8);
                }
                const int slot = sums % M::kSums;
                ok = warp_wait(&bars.s_full[slot], (sums / M::kSums) & 1, &bars.failed);
                if (!ok) break;
                fence_after();
                // past the last group the weights are copied as zeros and x is zero, whatever the scale
                const float ss = gi - 1 < a.groups ? s : 0.0f;
                const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + slot * N + (H == 2 ? 0 : c0);
                const uint64_t s2 = pack2(ss, ss);
                constexpr int L = C == 128 ? 16 : C == 64 ? 32 : C;  // columns of a load: what the running sums leave registers for
#pragma unroll
                for (int c = 0; c < C; c += L) {
                    uint32_t d[L];
                    if constexpr (L == 32)
                        tmem_load32(at + c, d);
                    else
                        tmem_load16(at + c, d);
                    tmem_wait_load();
                    if (c + L == C) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(&bars.s_empty[slot]);
                    }
#pragma unroll
                    for (int i = 0; i < L / 2; ++i)
                        y[c / 2 + i] = fma2(s2, pack2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), y[c / 2 + i]);
                }
            }
            if (!ok) {
#pragma unroll
                for (int i = 0; i < C / 2; ++i) y[i] = 0x7FC000007FC00000ull;
            }
            const int m0 = c0;
            if (a.cluster == 1) {
                if (n < a.outs) {
                    if (a.y_f32)
                        store_sums<float, C>(a, bars.back, y, m0, n);
                    else if (a.x_bf16)
                        store_sums<__nv_bfloat16, C>(a, bars.back, y, m0, n);
                    else
                        store_sums<__half, C>(a, bars.back, y, m0, n);
                }
            } else {
                // Every copy and product of this block is done: the rings give way to the block's sums. With two
                // products the first group has waited for the last sums of its own alone, and the other's may still
                // be read from x: the groups meet first.
                if constexpr (H == 2) asm volatile("bar.sync 1, %0;" ::"n"(M::kAdders * 128) : "memory");
                float* mine = reinterpret_cast<float*>(dyn);
#pragma unroll
                for (int i = 0; i < C; ++i) mine[(c0 + i) * 128 + row] = half_of(y[i / 2], i & 1);
            }
        }
    }
    __syncthreads();
    if (a.cluster > 1) {
        if (bars.failed) {  // copies that were under way may have landed on the sums: they are NaN again
            for (int i = tid; i < H * N * 128; i += M::kThreads) reinterpret_cast<float*>(dyn)[i] = __uint_as_float(0x7FC00000u);
        }
        // one item a cluster: each block adds up its share of the rows of x
        cluster_sync_all();
        const int item = first;
        for (int i = rank * H * N * 128 / a.cluster + tid; i < (rank + 1) * H * N * 128 / a.cluster; i += M::kThreads) {
            const int m = i / 128;
            const int64_t n = static_cast<int64_t>(item) * 128 + i % 128;
            if (m >= a.rows || n >= a.outs) continue;
            float v = 0.0f;
            for (int c = 0; c < a.cluster; ++c) {
                uint32_t remote;
                float p;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(shared_of(dyn) + i * 4), "r"(c));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(remote));
                v += p;
            }
            v = v * 0x1p24f * bars.back[m];
            const int64_t o = m * a.y_stride + n;
            if (a.y_f32)
                static_cast<float*>(a.y)[o] = v;
            else if (a.x_bf16)
                static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(v);
            else
                static_cast<__half*>(a.y)[o] = __float2half_rn(v);
        }
        __syncwarp();
        cluster_sync_all();  // no block leaves while another reads its memory
    }
    if (warp == kIssue)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(M::kColumns) : "memory");
}

template <int N, int H>
int launch(const ManyArgs& a, int dev, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    static_assert(Many<N, H>::kSmem + sizeof(Bars) <= arc::kSmemPerBlock, "shared memory");
    static_assert(Many<N, H>::kSums * N + Many<N, H>::kA * 64 <= Many<N, H>::kColumns, "tensor memory");
    if (arc::prepare(many_kernel<N, H>, dev, done, 100) != cudaSuccess) return ARC_E_CUDA;
    const unsigned rows = static_cast<unsigned>(a.halves * a.columns);
    if (a.x_bf16)
        many_x_kernel<ARC_BF16><<<rows, 256, 0, st>>>(a);
    else
        many_x_kernel<ARC_F16><<<rows, 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ARC_E_CUDA;
    const int items = a.tiles;
    const int64_t grid = a.cluster > 1 ? int64_t{items} * a.cluster : (items < sms ? items : sms);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(Many<N, H>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Many<N, H>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, many_kernel<N, H>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    return ARC_OK;
}

int columns_of(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

}  // namespace

size_t many_workspace(int64_t ins, int64_t rows) {
    const int64_t columns = columns_of(rows), halves = (rows + columns - 1) / columns;
    const int64_t blocks = (ins + kInner - 1) / kInner;
    return static_cast<size_t>(halves * columns * blocks * kInner * 2 + halves * columns * 4);
}

int launch_many(ManyArgs a, void* workspace, int dev, int sms, cudaStream_t st) {
    a.columns = columns_of(a.rows);
    a.halves = (a.rows + a.columns - 1) / a.columns;
    a.blocks = (a.ins + kInner - 1) / kInner;
    a.groups = a.ins / a.group;
    a.tiles = static_cast<int32_t>((a.outs + 127) / 128);
    a.x_ready = workspace;
    a.x_back = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        static_cast<size_t>(a.halves) * a.columns * a.blocks * kInner * 2);
    a.x_vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride % 8 == 0;
    a.s_vec = reinterpret_cast<uintptr_t>(a.scales) % 16 == 0 && a.groups % 8 == 0;
    // few tiles: split the inner dimension while every block keeps four blocks of it and all run at once (4,096 x
    // 4,096, 16 rows: 9.9 us split in four, 16.2 whole; 128 rows: 15.0 and 20.9)
    a.cluster = 1;
    while (a.cluster < 8 && int64_t{a.tiles} * a.cluster * 2 <= sms && a.blocks >= a.cluster * 8) a.cluster *= 2;
    if (a.columns == 16) return launch<16, 1>(a, dev, sms, st);
    if (a.columns == 32) return launch<32, 1>(a, dev, sms, st);
    if (a.columns == 64) return launch<64, 1>(a, dev, sms, st);
    return a.halves == 1 ? launch<128, 1>(a, dev, sms, st) : launch<128, 2>(a, dev, sms, st);
}

}  // namespace arcs

// arc_norm_join: the norm after a block, its gate, the scaled residual sum and the norm before the next one.
//
// A row's values stay in registers from their one load to their one store: 8 K of them a thread, and a row is a
// warp's (up to 1,024 values) or a block's.  The two sums of squares are added up in fp32: 8 K values in a thread,
// then a tree over the lanes and over the warps, so a sum is off by some 2^-21 of itself whatever the length.
// Many long rows go through rings in shared memory (join_rows_kernel).
//
// Bounds and figures.  HBM: 8,191 rows of 5,120 with a 32-bit stream, gates and a post norm, 587 MB: 105 us, 84% of the
// measured copy rate; 16 bits without gates 55 us, 90%; 60,000 x 512 56 us, 98%.  One row 2.9 us: two sums that wait for
// loads.  Odd rows: 4,000 x 5,003 61 us, 39%, 236 value by value: the weights do not begin as the rows do.
#pragma once

#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "launch_util.cuh"
#include "norm_args.cuh"
#include "serve_util.cuh"
#include "tensor_core.cuh"

namespace {

using namespace arcs;

constexpr int kWarpDim = 1024;   // a warp's row: up to 4 x 8 values a lane
constexpr int kWarpBlock = 128;  // threads of a block whose warps have a row each

template <int DT>
__device__ __forceinline__ float element(const void* p, int64_t i) {
    if constexpr (DT == ARC_F32)
        return static_cast<const float*>(p)[i];
    else
        return Half<DT>::to_float(static_cast<const typename Half<DT>::T*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void put(void* p, int64_t i, float x) {
    if constexpr (DT == ARC_F32)
        static_cast<float*>(p)[i] = x;
    else
        static_cast<typename Half<DT>::T*>(p)[i] = Half<DT>::from_float(x);
}
// Eight consecutive values from element i, a multiple of 8 on a 16-byte boundary.
template <int DT>
__device__ __forceinline__ void load_eight(const void* p, int64_t i, float (&x)[8]) {
    if constexpr (DT == ARC_F32) {
        const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[0];
        const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        load8<DT>(static_cast<const uint16_t*>(p) + i, true, x);
    }
}
template <int DT>
__device__ __forceinline__ void store_eight(void* p, int64_t i, const float (&x)[8]) {
    if constexpr (DT == ARC_F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        store8<DT>(static_cast<uint16_t*>(p) + i, true, x);
    }
}

// The sum over a row's threads; `slot` is another one for each sum of a row.
template <bool WARP>
__device__ __forceinline__ float row_sum(float s, float (*part)[32], int slot) {
#pragma unroll
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    if constexpr (WARP) return s;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[slot][threadIdx.x >> 5] = s;
    __syncthreads();
    s = (threadIdx.x & 31) < warps ? part[slot][threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
    return s;
}

// SD: type of the residual stream, DT of the others.
template <int SD, int DT, int K, bool WARP, Moves MOVES>
__global__ void __launch_bounds__(WARP ? kWarpBlock : K == 8 || (MOVES != kVectors && K > 1) ? 512 : 1024) join_kernel(const __grid_constant__ JoinArgs a) {
    __shared__ float part[4][32];
    const arc_norm_rows& r = a.r;
    const int dim = r.dim;
    const int threads = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int per = WARP ? kWarpBlock / 32 : 1;
    const bool f32w = r.weight_dtype == ARC_F32;
    int lead = 0;  // kShifted: values before the row's first boundary
    auto at = [&](int j, int e) {
        if constexpr (MOVES == kSingly) return (j * 8 + e) * threads + t;
        return (j * threads + t) * 8 + e + (MOVES == kShifted && lead ? lead - 8 : 0);
    };
    auto has = [&](int i) { return i < dim && (MOVES != kShifted || i >= 0); };
    auto whole = [&](int j) {
        if constexpr (MOVES == kShifted) return at(j, 0) >= 0 && at(j, 0) + 8 <= dim;
        return MOVES == kVectors && at(j, 0) < dim;
    };
    // `alike`: the tensor's rows begin as the others do
    auto load = [&](auto type, const void* p, int64_t row, int j, float (&x)[8], bool alike = true) {
        constexpr int D = decltype(type)::value;
        if (MOVES != kSingly && (MOVES == kVectors || alike) && whole(j)) {
            load_eight<D>(p, row + at(j, 0), x);
        } else if (MOVES != kVectors) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (has(at(j, e))) x[e] = element<D>(p, row + at(j, e));
        }
    };
    auto store = [&](auto type, void* p, int64_t row, int j, const float (&x)[8]) {
        constexpr int D = decltype(type)::value;
        if (MOVES != kSingly && whole(j)) {
            store_eight<D>(p, row + at(j, 0), x);
        } else if (MOVES != kVectors) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (has(at(j, e))) put<D>(p, row + at(j, e), x[e]);
        }
    };
    using Stream = std::integral_constant<int, SD>;
    using Other = std::integral_constant<int, DT>;
    using Wide = std::integral_constant<int, ARC_F32>;
    auto weights = [&](const void* p, int j, float (&x)[8]) {
        if (f32w)
            load(Wide{}, p, 0, j, x, false);
        else
            load(Other{}, p, 0, j, x, false);
    };
    // Eight groups: the registers hold one array of them, so the loads of the others stay where they stand.
    constexpr bool kTight = K == 8;
    auto fence = [] {
        if constexpr (kTight) asm volatile("" ::: "memory");
    };
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * per + (WARP ? threadIdx.x >> 5 : 0); row < r.rows;
         row += static_cast<int64_t>(gridDim.x) * per) {
        if constexpr (MOVES == kShifted) lead = static_cast<int>((8 - row * r.x_stride % 8) % 8);
        float u[K][8], x[K][8];
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) u[j][e] = x[j][e] = 0.0f;
        if (r.y) {
#pragma unroll
            for (int j = 0; j < K; ++j) load(Other{}, r.y, row * r.y_stride, j, u[j]);
        }
        if constexpr (!kTight) {
#pragma unroll
            for (int j = 0; j < K; ++j) load(Stream{}, r.x, row * r.x_stride, j, x[j]);
        }
        if (r.post_weight) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(u[j][e], u[j][e], s);
            const float f = rsqrtf(fmaf(row_sum<WARP>(s, part, turn), a.inv_dim, r.eps));
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float w[8] = {};
                fence();
                weights(r.post_weight, j, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[j][e] *= f * (r.offset + w[e]);
            }
        }
        if (r.gate) {
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float g[8] = {};
                fence();
                load(Other{}, r.gate, row * r.gate_stride, j, g, r.gate_stride != 0);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[j][e] *= r.activation == ARC_GATE_SIGMOID ? 1.0f / (1.0f + __expf(-g[e])) : g[e];
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            fence();
            float late[8] = {};
            if constexpr (kTight) load(Stream{}, r.x, row * r.x_stride, j, late);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = kTight ? late[e] : x[j][e];
                u[j][e] = r.y ? fmaf(r.alpha, u[j][e], v) : v;
                s = fmaf(u[j][e], u[j][e], s);
            }
        }
        if (r.n) {
            const float f = rsqrtf(fmaf(row_sum<WARP>(s, part, turn + 1), a.inv_dim, r.eps));
            if (r.h) {
#pragma unroll
                for (int j = 0; j < K; ++j) store(Stream{}, r.h, row * r.h_stride, j, u[j]);
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float w[8] = {};
                fence();
                if (r.weight) weights(r.weight, j, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[j][e] *= r.weight ? f * (r.offset + w[e]) : f;
                store(Other{}, r.n, row * r.n_stride, j, u[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < K; ++j) store(Stream{}, r.h, row * r.h_stride, j, u[j]);
        }
        turn ^= 2;  // the next row's sums go where no warp still reads
    }
}

// Many long rows: blocks that stay, each with a ring of rows in shared memory.  A row's x, y and gate come in by bulk
// copies one or two rows ahead, h and n take the places of x and y and go out the same way, so loads and stores are under way
// whatever the sums wait for.
constexpr int kMostStages = 3;
constexpr int kStreamSmem = 112 * 1024;  // of a block: two an SM

__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
}

template <int SD, int DT, int K>
__global__ void __launch_bounds__(1024) join_rows_kernel(const __grid_constant__ JoinArgs a, int stages) {
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ float part[4][32];
    __shared__ uint64_t full[kMostStages];
    __shared__ uint32_t failed;
    const arc_norm_rows& r = a.r;
    const int dim = r.dim, t = threadIdx.x, threads = blockDim.x;
    constexpr int kSize = SD == ARC_F32 ? 4 : 2;
    const bool gates = r.gate != nullptr && r.gate_stride != 0;
    const bool f32w = r.weight_dtype == ARC_F32;
    const uint32_t x_bytes = dim * kSize, y_bytes = dim * 2, stage = x_bytes + y_bytes * (gates ? 2 : 1);
    if (t == 0) {
        for (int i = 0; i < kMostStages; ++i) bar_init(&full[i], 1);
        failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_operands();
    }
    __syncthreads();
    const int64_t step = gridDim.x;
    auto fetch = [&](int64_t row, int s) {
        if (row >= r.rows) return;
        const uint32_t to = shared_of(dyn) + s * stage;
        bar_expect(&full[s], stage);
        bulk_copy(to, static_cast<const char*>(r.x) + row * r.x_stride * kSize, x_bytes, &full[s]);
        bulk_copy(to + x_bytes, static_cast<const char*>(r.y) + row * r.y_stride * 2, y_bytes, &full[s]);
        if (gates) bulk_copy(to + x_bytes + y_bytes, static_cast<const char*>(r.gate) + row * r.gate_stride * 2, y_bytes, &full[s]);
    };
    if (t == 0)
        for (int i = 0; i < stages - 1; ++i) fetch(blockIdx.x + i * step, i);
    auto weights = [&](const void* p, int at, float (&w)[8]) {
        if (f32w)
            load_eight<ARC_F32>(p, at, w);
        else
            load_eight<DT>(p, at, w);
    };
    int s = 0, turn = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < r.rows; row += step) {
        if (t == 0) {  // the row before has left its place: a later one comes there
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            fetch(row + (stages - 1) * step, s == 0 ? stages - 1 : s - 1);
        }
        const bool ok = bar_wait(&full[s], phase, &failed);
        uint8_t* const xs = dyn + s * stage;
        uint8_t* const ys = xs + x_bytes;
        float u[K][8], x[K][8];
        uint4 gate[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int at = (j * threads + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) u[j][e] = x[j][e] = 0.0f;
            gate[j] = make_uint4(0, 0, 0, 0);
            if (at < dim) {
                load_eight<DT>(ys, at, u[j]);
                load_eight<SD>(xs, at, x[j]);
                if (gates) gate[j] = *reinterpret_cast<const uint4*>(ys + y_bytes + at * 2);
                else if (r.gate) gate[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.gate) + at);
            }
            if (!ok) x[j][0] = __int_as_float(0x7FC00000);
        }
        if (r.post_weight) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(u[j][e], u[j][e], sum);
            const float f = rsqrtf(fmaf(row_sum<false>(sum, part, turn), a.inv_dim, r.eps));
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const int at = (j * threads + t) * 8;
                float w[8] = {};
                if (at < dim) weights(r.post_weight, at, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[j][e] *= f * (r.offset + w[e]);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (r.gate) {
                const uint32_t words[4] = {gate[j].x, gate[j].y, gate[j].z, gate[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 g = Half<DT>::unpack(words[e]);
                    u[j][2 * e] *= r.activation == ARC_GATE_SIGMOID ? 1.0f / (1.0f + __expf(-g.x)) : g.x;
                    u[j][2 * e + 1] *= r.activation == ARC_GATE_SIGMOID ? 1.0f / (1.0f + __expf(-g.y)) : g.y;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[j][e] = fmaf(r.alpha, u[j][e], x[j][e]);
                sum = fmaf(u[j][e], u[j][e], sum);
            }
        }
        const float f = rsqrtf(fmaf(row_sum<false>(sum, part, turn + 1), a.inv_dim, r.eps));
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int at = (j * threads + t) * 8;
            if (at >= dim) continue;
            store_eight<SD>(xs, at, u[j]);
            float w[8] = {};
            if (r.weight) weights(r.weight, at, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[j][e] *= r.weight ? f * (r.offset + w[e]) : f;
            store_eight<DT>(ys, at, u[j]);
        }
        fence_operands();
        __syncthreads();
        if (t == 0) {
            bulk_store(static_cast<char*>(r.h) + row * r.h_stride * kSize, shared_of(xs), x_bytes);
            bulk_store(static_cast<char*>(r.n) + row * r.n_stride * 2, shared_of(ys), y_bytes);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        turn ^= 2;
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    if (t == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int SD, int DT, int K>
int launch_rows(const JoinArgs& a, int threads, int stages, int bytes, int grid, int dev, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (arc::prepare(join_rows_kernel<SD, DT, K>, dev, done, 100) != cudaSuccess) return ARC_E_CUDA;
    join_rows_kernel<SD, DT, K><<<grid, threads, bytes, st>>>(a, stages);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

template <int SD, int DT, Moves MOVES>
int launch(const JoinArgs& a, int dev, int sms, cudaStream_t st) {
    const arc_norm_rows& r = a.r;
    const int groups = (r.dim + 7) / 8 + (MOVES == kShifted ? 1 : 0);
    if (r.dim <= kWarpDim - 8 * (MOVES == kShifted) && r.rows >= sms) {
        const int64_t want = (r.rows + 3) / 4;
        const unsigned grid = static_cast<unsigned>(want < sms * 64 ? want : sms * 64);
        if (MOVES == kVectors && groups <= 32)
            join_kernel<SD, DT, 1, true, kVectors><<<grid, kWarpBlock, 0, st>>>(a);
        else if (MOVES == kVectors && groups <= 64)
            join_kernel<SD, DT, 2, true, kVectors><<<grid, kWarpBlock, 0, st>>>(a);
        else
            join_kernel<SD, DT, 4, true, MOVES><<<grid, kWarpBlock, 0, st>>>(a);
    } else {
        if constexpr (MOVES == kVectors) {
            const int64_t stage = int64_t{r.dim} * ((SD == ARC_F32 ? 4 : 2) + (r.gate && r.gate_stride != 0 ? 4 : 2));
            // With 4 rows an SM and more: 8,191 x 5,120, 32-bit stream, gate and post norm 105 us, 137 by a block a row; 16
            // bits alone 55 and 66; 1,300 x 8,192 13.3 and 15.2; 700 x 2,048 7.3 and 6.7, 16,000 x 2,048 57 and 52: short
            // rows stay with the others, and so do those of which two blocks an SM have no room for two (2,000 x 8,192,
            // gates and a 32-bit stream 53 us, 58 in one block an SM).
            if (r.y && r.h && r.n && groups > 256 && groups <= 2048 && 2 * stage <= kStreamSmem && r.rows >= 4 * sms) {
                const int threads = ((groups + 1) / 2 + 31) / 32 * 32;
                const int stages = 3 * stage <= kStreamSmem ? 3 : 2, bytes = static_cast<int>(stages * stage);
                return launch_rows<SD, DT, 2>(a, threads, stages, bytes, 2 * sms, dev, st);
            }
        }
        const unsigned grid = static_cast<unsigned>(r.rows < sms * 64 ? r.rows : sms * 64);
        // groups of a thread: two while 1,024 threads have registers for them, 512 where rows are not vectors throughout
        // (4,000 x 5,003: 61 us, 85 with four)
        constexpr bool kVec = MOVES == kVectors;
        const int k = groups <= 256 ? 1 : groups <= (kVec ? 2048 : 1024) ? 2 : !kVec && groups <= 2048 ? 4 : 8;
        const int threads = ((groups + k - 1) / k + 31) / 32 * 32;
        if (k == 1)
            join_kernel<SD, DT, 1, false, MOVES><<<grid, threads, 0, st>>>(a);
        else if (k == 2)
            join_kernel<SD, DT, 2, false, MOVES><<<grid, threads, 0, st>>>(a);
        else if (!kVec && k == 4)
            join_kernel<SD, DT, 4, false, kVec ? kSingly : MOVES><<<grid, threads, 0, st>>>(a);
        else
            join_kernel<SD, DT, 8, false, MOVES><<<grid, threads, 0, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

template <int DT>
int launch_join(const JoinArgs& a, Moves moves, int dev, int sms, cudaStream_t st) {
    if (a.r.stream_dtype == ARC_F32)
        return moves == kVectors   ? launch<ARC_F32, DT, kVectors>(a, dev, sms, st)
               : moves == kShifted ? launch<ARC_F32, DT, kShifted>(a, dev, sms, st)
                                   : launch<ARC_F32, DT, kSingly>(a, dev, sms, st);
    return moves == kVectors   ? launch<DT, DT, kVectors>(a, dev, sms, st)
           : moves == kShifted ? launch<DT, DT, kShifted>(a, dev, sms, st)
                               : launch<DT, DT, kSingly>(a, dev, sms, st);
}

}  // namespace

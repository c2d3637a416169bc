// arc_norm_join: the norm after a block, its gate, the scaled residual sum and the norm before the next one.
//
// A row's values stay in registers from their one load to their one store: 8 K of them a thread, and a row is a
// warp's (up to 1,024 values) or a block's.  The two sums of squares are added up in fp32: 8 K values in a thread,
// then a tree over the lanes and over the warps, so a sum is off by some 2^-21 of itself whatever the length.
#include <climits>
#include <cstdint>
#include <type_traits>

#include "serve/arc_norm.h"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kWarpDim = 1024;   // a warp's row: up to 4 x 8 values a lane
constexpr int kWarpBlock = 128;  // threads of a block whose warps have a row each

struct JoinArgs {
    arc_norm_rows r;
    float inv_dim;
};

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

// SD: type of the residual stream, DT of the others.  VEC: a thread has groups of 8 consecutive values and moves
// them 16 bytes at a time; otherwise single values, neighbours in neighbouring threads.
template <int SD, int DT, int K, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? kWarpBlock : K == 8 ? 512 : 1024) join_kernel(const __grid_constant__ JoinArgs a) {
    __shared__ float part[4][32];
    const arc_norm_rows& r = a.r;
    const int dim = r.dim;
    const int threads = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int per = WARP ? kWarpBlock / 32 : 1;
    const bool f32w = r.weight_dtype == ARC_F32;
    auto at = [&](int j, int e) { return VEC ? (j * threads + t) * 8 + e : (j * 8 + e) * threads + t; };
    auto load = [&](auto type, const void* p, int64_t row, int j, float (&x)[8]) {
        constexpr int D = decltype(type)::value;
        if constexpr (VEC) {
            if (at(j, 0) < dim) load_eight<D>(p, row + at(j, 0), x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at(j, e) < dim) x[e] = element<D>(p, row + at(j, e));
        }
    };
    auto store = [&](auto type, void* p, int64_t row, int j, const float (&x)[8]) {
        constexpr int D = decltype(type)::value;
        if constexpr (VEC) {
            if (at(j, 0) < dim) store_eight<D>(p, row + at(j, 0), x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at(j, e) < dim) put<D>(p, row + at(j, e), x[e]);
        }
    };
    using Stream = std::integral_constant<int, SD>;
    using Other = std::integral_constant<int, DT>;
    using Wide = std::integral_constant<int, ARC_F32>;
    auto weights = [&](const void* p, int j, float (&x)[8]) {
        if (f32w)
            load(Wide{}, p, 0, j, x);
        else
            load(Other{}, p, 0, j, x);
    };
    // Eight groups: the registers hold one array of them, so the loads of the others stay where they stand.
    constexpr bool kTight = K == 8;
    auto fence = [] {
        if constexpr (kTight) asm volatile("" ::: "memory");
    };
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * per + (WARP ? threadIdx.x >> 5 : 0); row < r.rows;
         row += static_cast<int64_t>(gridDim.x) * per) {
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
                load(Other{}, r.gate, row * r.gate_stride, j, g);
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

template <int SD, int DT, bool VEC>
int launch(const JoinArgs& a, int sms, cudaStream_t st) {
    const arc_norm_rows& r = a.r;
    const int groups = (r.dim + 7) / 8;
    if (r.dim <= kWarpDim && r.rows >= sms) {
        const int64_t want = (r.rows + 3) / 4;
        const unsigned grid = static_cast<unsigned>(want < sms * 64 ? want : sms * 64);
        if (groups <= 32)
            join_kernel<SD, DT, 1, true, VEC><<<grid, kWarpBlock, 0, st>>>(a);
        else if (groups <= 64)
            join_kernel<SD, DT, 2, true, VEC><<<grid, kWarpBlock, 0, st>>>(a);
        else
            join_kernel<SD, DT, 4, true, VEC><<<grid, kWarpBlock, 0, st>>>(a);
    } else {
        const unsigned grid = static_cast<unsigned>(r.rows < sms * 64 ? r.rows : sms * 64);
        const int k = groups <= 256 ? 1 : groups <= 2048 ? 2 : 8;
        const int threads = ((groups + k - 1) / k + 31) / 32 * 32;
        if (k == 1)
            join_kernel<SD, DT, 1, false, VEC><<<grid, threads, 0, st>>>(a);
        else if (k == 2)
            join_kernel<SD, DT, 2, false, VEC><<<grid, threads, 0, st>>>(a);
        else
            join_kernel<SD, DT, 8, false, VEC><<<grid, threads, 0, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

bool finite(float x) { return x >= -3.4028235e38f && x <= 3.4028235e38f; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

extern "C" int arc_norm_join(const arc_norm_rows* rows, void* stream) {
    if (rows == nullptr) return ARC_E_NULL;
    const arc_norm_rows& r = *rows;
    if (r.x == nullptr || (r.h == nullptr && r.n == nullptr)) return ARC_E_NULL;
    if (r.y == nullptr && (r.gate != nullptr || r.post_weight != nullptr)) return ARC_E_NULL;
    if (r.dtype != ARC_BF16 && r.dtype != ARC_F16) return ARC_E_DTYPE;
    if ((r.stream_dtype != r.dtype && r.stream_dtype != ARC_F32) || (r.weight_dtype != r.dtype && r.weight_dtype != ARC_F32))
        return ARC_E_DTYPE;
    if (r.rows <= 0 || r.rows > INT_MAX || r.dim <= 0 || r.dim > ARC_NORM_MAX_DIM) return ARC_E_SHAPE;
    const bool many = r.rows > 1;
    if (many && (r.x_stride < r.dim || (r.y && r.y_stride < r.dim) || (r.gate && r.gate_stride != 0 && r.gate_stride < r.dim) ||
                 (r.h && r.h_stride < r.dim) || (r.n && r.n_stride < r.dim)))
        return ARC_E_SHAPE;
    if (many && ((r.h == r.x && r.h_stride != r.x_stride) || (r.n && r.n == r.y && r.n_stride != r.y_stride)))
        return ARC_E_OPTION;
    if (r.activation != ARC_GATE_LINEAR && r.activation != ARC_GATE_SIGMOID) return ARC_E_OPTION;
    if (!finite(r.alpha) || !finite(r.offset) || !finite(r.eps) || !(r.eps > 0.0f)) return ARC_E_OPTION;
    const uintptr_t stream_size = r.stream_dtype == ARC_F32 ? 4 : 2, weight_size = r.weight_dtype == ARC_F32 ? 4 : 2;
    if (!aligned(r.x, stream_size) || !aligned(r.h, stream_size) || !aligned(r.y, 2) || !aligned(r.gate, 2) ||
        !aligned(r.n, 2) || !aligned(r.post_weight, weight_size) || !aligned(r.weight, weight_size))
        return ARC_E_ALIGN;
    auto sixteen = [&](const void* p, int64_t stride, uintptr_t size) {
        return p == nullptr || (aligned(p, 16) && (!many || (stride * static_cast<int64_t>(size)) % 16 == 0));
    };
    const bool vec = r.dim % 8 == 0 && sixteen(r.x, r.x_stride, stream_size) && sixteen(r.h, r.h_stride, stream_size) &&
                     sixteen(r.y, r.y_stride, 2) && sixteen(r.gate, r.gate_stride, 2) && sixteen(r.n, r.n_stride, 2) &&
                     aligned(r.post_weight, 16) && aligned(r.weight, 16);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    const JoinArgs a{r, 1.0f / static_cast<float>(r.dim)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = r.stream_dtype == ARC_F32;
    if (r.dtype == ARC_BF16) {
        if (wide) return vec ? launch<ARC_F32, ARC_BF16, true>(a, sms, st) : launch<ARC_F32, ARC_BF16, false>(a, sms, st);
        return vec ? launch<ARC_BF16, ARC_BF16, true>(a, sms, st) : launch<ARC_BF16, ARC_BF16, false>(a, sms, st);
    }
    if (wide) return vec ? launch<ARC_F32, ARC_F16, true>(a, sms, st) : launch<ARC_F32, ARC_F16, false>(a, sms, st);
    return vec ? launch<ARC_F16, ARC_F16, true>(a, sms, st) : launch<ARC_F16, ARC_F16, false>(a, sms, st);
}

// arc_w4_matvec: a few rows times a matrix of 4-bit weights with group scales.
#include <climits>
#include <cstdint>

#include "serve/arc_w4.h"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kThreads = 256;

struct W4Args {
    arc_w4_weight w;
    const void* x;
    void* y;
    int64_t x_stride, y_stride;
    int32_t rows;
    int32_t y_f32;
};

// One warp for each output column, the rows in turn: a lane takes eight
// weights (one 32-bit word) of every 256, whose group is one.
template <int DT>
__global__ void __launch_bounds__(kThreads) w4_kernel(const __grid_constant__ W4Args a) {
    using T = typename Half<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t n = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (n >= a.w.outs) return;
    const int groups = a.w.ins / a.w.group;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const char*>(a.w.q) + n * a.w.row_bytes);
    const T* s = static_cast<const T*>(a.w.scales) + n * groups;
    const uint8_t* z = a.w.zeros ? a.w.zeros + n * groups : nullptr;
    for (int m = 0; m < a.rows; ++m) {
        const T* x = static_cast<const T*>(a.x) + m * a.x_stride;
        float sum = 0.0f;
        for (int k = lane * 8; k < a.w.ins; k += 256) {
            const int g = k / a.w.group;
            const uint32_t w = __ldg(q + (k >> 3));
            const int zero = z ? z[g] : 8;
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part = fmaf(Half<DT>::to_float(x[k + i]), static_cast<float>(static_cast<int>((w >> (4 * i)) & 15) - zero), part);
            sum = fmaf(part, Half<DT>::to_float(s[g]), sum);
        }
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        if (lane == 0) {
            if (a.y_f32)
                static_cast<float*>(a.y)[m * a.y_stride + n] = sum;
            else
                static_cast<T*>(a.y)[m * a.y_stride + n] = Half<DT>::from_float(sum);
        }
    }
}

int check_weight(const arc_w4_weight* w) {
    if (w == nullptr || w->q == nullptr || w->scales == nullptr) return ARC_E_NULL;
    if (w->group != 32 && w->group != 64 && w->group != 128) return ARC_E_UNSUPPORTED;
    if (w->outs <= 0 || w->outs > INT_MAX || w->ins <= 0 || w->ins > ARC_W4_MAX_INS || w->ins % w->group != 0 ||
        w->row_bytes < w->ins / 2)
        return ARC_E_SHAPE;
    if (reinterpret_cast<uintptr_t>(w->q) % 16 != 0 || w->row_bytes % 16 != 0 ||
        reinterpret_cast<uintptr_t>(w->scales) % 2 != 0)
        return ARC_E_ALIGN;
    return ARC_OK;
}

}  // namespace

extern "C" {

size_t arc_w4_workspace_bytes(const arc_w4_weight*, int64_t) { return 0; }

int arc_w4_matvec(const arc_w4_weight* weight, const void* x, int64_t rows, int64_t x_stride, int32_t x_dtype, void* y,
                  int64_t y_stride, int32_t y_dtype, void*, size_t, void* stream) {
    const int rc = check_weight(weight);
    if (rc != ARC_OK) return rc;
    if (x == nullptr || y == nullptr) return ARC_E_NULL;
    if (x_dtype != ARC_BF16 && x_dtype != ARC_F16) return ARC_E_DTYPE;
    if (y_dtype != x_dtype && y_dtype != ARC_F32) return ARC_E_DTYPE;
    if (rows <= 0 || rows > ARC_W4_MAX_ROWS || x_stride < weight->ins || y_stride < weight->outs) return ARC_E_SHAPE;
    if (reinterpret_cast<uintptr_t>(x) % 2 != 0 || reinterpret_cast<uintptr_t>(y) % (y_dtype == ARC_F32 ? 4 : 2) != 0)
        return ARC_E_ALIGN;
    W4Args a{*weight, x, y, x_stride, y_stride, static_cast<int32_t>(rows), y_dtype == ARC_F32};
    const unsigned grid = static_cast<unsigned>((weight->outs * 32 + kThreads - 1) / kThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_dtype == ARC_BF16)
        w4_kernel<ARC_BF16><<<grid, kThreads, 0, st>>>(a);
    else
        w4_kernel<ARC_F16><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

}  // extern "C"

// arc_norm_join: the checks of a call; the kernels are in norm_join.cuh.
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "norm_args.cuh"

namespace {

using namespace arcs;

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
    // rows on 16-byte boundaries; rows that all begin alike, from tensors that do
    const bool based = aligned(r.x, 16) && aligned(r.h, 16) && aligned(r.y, 16) && aligned(r.gate, 16) && aligned(r.n, 16);
    auto strided = [&](const void* p, int64_t stride) { return p == nullptr || !many || stride % 8 == 0; };
    auto alike = [&](const void* p, int64_t stride) { return p == nullptr || !many || (stride - r.x_stride) % 8 == 0; };
    const bool vec = based && r.dim % 8 == 0 && strided(r.x, r.x_stride) && strided(r.h, r.h_stride) &&
                     strided(r.y, r.y_stride) && strided(r.gate, r.gate_stride) && strided(r.n, r.n_stride) &&
                     aligned(r.post_weight, 16) && aligned(r.weight, 16);
    const bool shifted = based && r.dim < ARC_NORM_MAX_DIM - 8 && alike(r.h, r.h_stride) && alike(r.y, r.y_stride) &&
                         (r.gate_stride == 0 || alike(r.gate, r.gate_stride)) && alike(r.n, r.n_stride);
    const Moves moves = vec ? kVectors : shifted ? kShifted : kSingly;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    const JoinArgs a{r, 1.0f / static_cast<float>(r.dim)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return r.dtype == ARC_BF16 ? launch_join_bf16(a, moves, dev, sms, st) : launch_join_f16(a, moves, dev, sms, st);
}

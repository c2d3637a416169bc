// The tensor-core path of arc_w4_matvec (w4_many.cu), for 9 .. 256 rows.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace arcs {

struct ManyArgs {
    const void* q;
    const void* scales;
    const uint8_t* zeros;
    const void* x;
    void* y;
    int64_t row_bytes, outs, x_stride, y_stride;
    int32_t ins, group, rows, y_f32, x_bf16;
    // set by launch_many
    int32_t columns;  // rows of x of a product
    int32_t halves;   // products that cover the rows
    int32_t blocks;   // 128 inner values each
    int32_t groups, tiles, cluster, x_vec, s_vec;
    void* x_ready;
    float* x_back;
};

size_t many_workspace(int64_t ins, int64_t rows);
int launch_many(ManyArgs a, void* workspace, int dev, int sms, cudaStream_t st);

}  // namespace arcs

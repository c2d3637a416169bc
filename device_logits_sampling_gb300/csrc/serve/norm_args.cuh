// What the checks and the kernels of arc_norm_join share.
#pragma once

#include <cuda_runtime.h>

#include "serve/arc_norm.h"

namespace arcs {

struct JoinArgs {
    arc_norm_rows r;
    float inv_dim;
};

// How values are moved.  kVectors: a thread has groups of 8 consecutive values, 16 bytes at a time.  kShifted: the same
// where rows begin anywhere, but all tensors' alike: the groups lie on the 16-byte boundaries, the first and the last are
// short.  kSingly: single values, neighbours in neighbouring threads.
enum Moves { kVectors, kShifted, kSingly };

// norm_bf16.cu, norm_f16.cu
int launch_join_bf16(const JoinArgs& a, Moves moves, int dev, int sms, cudaStream_t st);
int launch_join_f16(const JoinArgs& a, Moves moves, int dev, int sms, cudaStream_t st);

}  // namespace arcs

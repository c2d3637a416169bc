// What the three kernels of arc_kv_attend_shared share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "serve/arc_kv.h"

namespace arcs {

// Where a call's parts lie in its workspace, in bytes.
struct SharedLayout {
    size_t rows, logs;            // the sequences' own tokens: [T][q_heads][head_dim] fp32, and their logarithms
    size_t slots, slot_logs;      // the prefix's partials
    size_t bytes;
    int64_t units, row_groups;    // (cached head, group of rows); groups a head
    int64_t group_rows;           // rows of a group
};
SharedLayout shared_layout(const arc_kv_cache& cache, int64_t T, int64_t q_heads);

// kv_behind.cu: each sequence's tokens behind the prefix, into the workspace.
int launch_behind(const arc_kv_cache& cache, const arc_kv_step& step, const arc_kv_query& query, uint32_t* err_word,
                  void* workspace, const SharedLayout& at, int64_t prefix_tokens, int dev, int sms, cudaStream_t st);

}  // namespace arcs

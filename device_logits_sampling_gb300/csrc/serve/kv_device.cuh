// Device code that arc_kv_append and arc_kv_attend share: which rows a sequence's new tokens are.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "serve/arc_kv.h"

namespace arcs {

// Rows of sequence b: first and count; a pair of offsets that does not ascend within 0 .. T counts as none.
__device__ __forceinline__ bool rows_of(const arc_kv_step& s, int64_t b, int64_t& first, int64_t& n) {
    if (s.row_offsets == nullptr) {
        first = b;
        n = 1;
        return true;
    }
    const int64_t lo = __ldg(s.row_offsets + b), hi = __ldg(s.row_offsets + b + 1);
    first = lo;
    n = hi - lo;
    if (lo < 0 || hi < lo || hi > s.T || (b == 0 && lo != 0) || (b == s.B - 1 && hi != s.T)) {
        n = 0;
        return false;
    }
    return true;
}

// The sequences before the first whose offsets are wrong, as a rule all B; called by a whole block. No two of them
// share a row, and the rows from unclaimed_rows() on belong to none.
__device__ __forceinline__ int64_t sound_sequences(const arc_kv_step& s) {
    __shared__ unsigned long long least;
    int64_t bad = s.B;
    for (int64_t b = threadIdx.x; b < s.B && bad == s.B; b += blockDim.x) {
        int64_t first, n;
        if (!rows_of(s, b, first, n)) bad = b;
    }
    if (!__syncthreads_or(bad < s.B)) return s.B;
    if (threadIdx.x == 0) least = static_cast<unsigned long long>(s.B);
    __syncthreads();
    if (bad < s.B) atomicMin(&least, static_cast<unsigned long long>(bad));
    __syncthreads();
    return static_cast<int64_t>(least);
}

__device__ __forceinline__ int64_t unclaimed_rows(const arc_kv_step& s, int64_t sound) {
    return sound == 0 ? 0 : static_cast<int64_t>(__ldg(s.row_offsets + sound));
}

}  // namespace arcs

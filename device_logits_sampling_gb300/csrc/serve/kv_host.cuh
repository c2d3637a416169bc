// Host-side checks that arc_kv_append and arc_kv_attend share.
#pragma once

#include <climits>
#include <cstdint>

#include "serve/arc_kv.h"

namespace arcs {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int check_cache(const arc_kv_cache* c) {
    if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr)
        return ARC_E_NULL;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ARC_E_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return ARC_E_UNSUPPORTED;
    if (c->pages <= 0 || c->heads <= 0 || c->heads > 4096) return ARC_E_SHAPE;
    if (c->head_stride < int64_t{c->page_size} * c->head_dim || c->page_stride < 0) return ARC_E_SHAPE;
    // heads inside a page or pages inside a head: either order, no overlap
    const bool page_major = c->page_stride >= c->head_stride * (c->heads - 1) + int64_t{c->page_size} * c->head_dim;
    const bool head_major = c->page_stride >= int64_t{c->page_size} * c->head_dim &&
                            c->head_stride >= c->page_stride * (int64_t{c->pages} - 1) + int64_t{c->page_size} * c->head_dim;
    if (c->pages > 1 && c->heads > 1 && !page_major && !head_major) return ARC_E_SHAPE;
    if (c->pages > 1 && c->page_stride < int64_t{c->page_size} * c->head_dim) return ARC_E_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % 16 != 0 || c->head_stride % 16 != 0 ||
        !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return ARC_E_ALIGN;
    return ARC_OK;
}

inline int check_step(const arc_kv_cache* c, const arc_kv_step* s) {
    if (s == nullptr || s->page_table == nullptr || s->positions == nullptr) return ARC_E_NULL;
    if (s->B <= 0 || s->B > (int64_t{1} << 20) || s->T <= 0 || s->T > (int64_t{1} << 24)) return ARC_E_SHAPE;
    if (s->row_offsets == nullptr && s->T != s->B) return ARC_E_SHAPE;
    if (s->max_pages <= 0 || int64_t{s->max_pages} * c->page_size > INT_MAX || s->table_stride < s->max_pages)
        return ARC_E_SHAPE;
    if (s->reserved != 0) return ARC_E_OPTION;
    if (!aligned(s->page_table, 4) || !aligned(s->positions, 4) || !aligned(s->row_offsets, 4)) return ARC_E_ALIGN;
    return ARC_OK;
}

// A strided tensor of 16-bit heads: 0 where 16-byte accesses do not fit it.
inline bool vectors(const void* p, int64_t token_stride, int64_t head_stride) {
    return aligned(p, 16) && token_stride % 8 == 0 && head_stride % 8 == 0;
}

}  // namespace arcs

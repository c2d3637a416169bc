/*
 * arc_norm.h -- the join around a block for GB300 (sm_103a): the norm after the
 * block, its gate, the scaled residual sum and the norm before the next block,
 * in one pass over the rows.
 *
 * Per row, with all sums and products in fp32:
 *     u = y                                   (0 where y is NULL)
 *     u = u * rsqrt(mean(u^2) + eps) * (offset + post_weight)   with post_weight
 *     u = u * gate  or  u * sigmoid(gate)                       with gate
 *     h = x + alpha * u
 *     n = h * rsqrt(mean(h^2) + eps) * (offset + weight)
 * n is computed from h before h is rounded to its type; h and n are rounded
 * once.  The mean of squares has to lie in fp32's range: a row of values near
 * 1e19 and above gives zeros, infinities or NaN in n.  Infinite and NaN values
 * spoil their own row alone.
 *
 * Library: libarcserve.so; conventions as in arc_kv.h.
 */
#ifndef ARC_NORM_H
#define ARC_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "../arc_sample.h" /* ARC_OK, ARC_E_*, ARC_F32, ARC_BF16, ARC_F16 */

#ifdef __cplusplus
extern "C" {
#endif

#define ARC_NORM_MAX_DIM 32768

#define ARC_GATE_LINEAR 0  /* u * gate */
#define ARC_GATE_SIGMOID 1 /* u * 1 / (1 + exp(-gate)) */

/* Host struct.  Strides are elements from one row to the next; the values of a
 * row are contiguous.  Rows on 16-byte boundaries are moved 16 bytes at a time. */
typedef struct arc_norm_rows {
    const void* x;           /* device [rows][dim], stream_dtype: the residual stream */
    const void* y;           /* device [rows][dim], dtype: the block's output; NULL: none */
    const void* gate;        /* device [rows][dim], dtype, or NULL; gate_stride 0: one row for all */
    const void* post_weight; /* device [dim], weight_dtype; NULL: no norm after the block */
    const void* weight;      /* device [dim], weight_dtype; NULL: 1 (whatever the offset) */
    void* h;                 /* device [rows][dim], stream_dtype, or NULL; may be x with its stride */
    void* n;                 /* device [rows][dim], dtype, or NULL; may be y with its stride */
    int64_t x_stride, y_stride, gate_stride, h_stride, n_stride;
    int64_t rows;            /* 1 .. 2^31 - 1 */
    int32_t dim;             /* 1 .. ARC_NORM_MAX_DIM */
    int32_t stream_dtype;    /* dtype or ARC_F32 */
    int32_t dtype;           /* ARC_BF16 or ARC_F16 */
    int32_t weight_dtype;    /* dtype or ARC_F32 */
    int32_t activation;      /* ARC_GATE_* */
    float alpha;             /* finite */
    float offset;            /* finite; 1 for weights stored as their difference from 1 */
    float eps;               /* finite, > 0 */
} arc_norm_rows;

/* gate and post_weight need y; h or n has to be given.  Outputs overlap no
 * input but as said above. */
int arc_norm_join(const arc_norm_rows* rows, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ARC_NORM_H */

/*
 * arc_w4.h -- products of a few rows with a matrix of 4-bit weights and group
 * scales for GB300 (sm_103a): the projections of a decode step, and the last
 * one, whose logits arc_sample_batch (arc_sample.h) reads.
 *
 *     y[m][n] = sum_k x[m][k] * (q[n][k] - z[n][k / group]) * s[n][k / group]
 *
 * q is unsigned, 0 .. 15, two to a byte: byte i of row n holds q[n][2 i] in
 * its low half and q[n][2 i + 1] in its high half.  z is 8 where `zeros` is
 * NULL.  x enters the products as fp16 after a power-of-two scaling of each row
 * (exact but for values below 2^-25 of the row's largest), codes less zero
 * points are exact, and so are products.  Sums are fp32; within a group they are
 * the tensor cores', which cut off where a rounding would be to nearest (one
 * part in 2^23 for 16 products).  y is rounded once.  An infinite or NaN value of
 * x makes its own row infinite or NaN.
 *
 * Library: libarcserve.so; conventions as in arc_kv.h.
 */
#ifndef ARC_W4_H
#define ARC_W4_H

#include <stddef.h>
#include <stdint.h>

#include "../arc_sample.h" /* ARC_OK, ARC_E_*, ARC_F32, ARC_BF16, ARC_F16 */

#ifdef __cplusplus
extern "C" {
#endif

#define ARC_W4_MAX_ROWS 256
#define ARC_W4_MAX_INS 32768

/* Host struct. */
typedef struct arc_w4_weight {
    const void* q;         /* device, [outs][row_bytes], 16-byte aligned */
    const void* scales;    /* device, [outs][ins / group], dtype of x */
    const uint8_t* zeros;  /* device, [outs][ins / group], each 0 .. 15, or NULL */
    int64_t row_bytes;     /* >= ins / 2, a multiple of 16 */
    int64_t outs;          /* 1 .. 2^31 - 1 */
    int32_t ins;           /* a multiple of group, at most ARC_W4_MAX_INS */
    int32_t group;         /* 32, 64 or 128 */
} arc_w4_weight;

/*
 *   x         device [rows][x_stride], ARC_BF16 or ARC_F16
 *   rows      1 .. ARC_W4_MAX_ROWS
 *   y         device [rows][y_stride], dtype of x or ARC_F32
 *   workspace device, 16-byte aligned, arc_w4_workspace_bytes(weight, rows)
 *             bytes (NULL where that is 0); it needs no initial contents.
 *             Calls that share one must be ordered.
 */
int arc_w4_matvec(const arc_w4_weight* weight, const void* x, int64_t rows, int64_t x_stride, int32_t x_dtype,
                  void* y, int64_t y_stride, int32_t y_dtype, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Host only; 0 where no workspace is needed, and for arguments that
 * arc_w4_matvec would refuse. */
size_t arc_w4_workspace_bytes(const arc_w4_weight* weight, int64_t rows);

#ifdef __cplusplus
}
#endif
#endif /* ARC_W4_H */

/*
 * arc_edit.h -- edits of a step's logits before they are sampled for GB300
 * (sm_103a): penalties for the ids of each row's history, biases for some ids,
 * and a bit mask of the ids that a grammar allows, in one pass.
 *
 * Per row r and id i, with z the logit as fp32, in this order:
 *   1. i in the row's history c > 0 times: arc_sample.h's penalties, each an fp32
 *      round-to-nearest operation:  z = z > 0 ? z / rep : z * rep;
 *      z -= fl(c * freq);  z -= pres
 *   2. i has a bias: z += bias.  Where the row lists i more than once, its last
 *      entry counts
 *   3. the mask's bit of i is 0: z = -infinity, whatever it was
 * and z is rounded once to the output's type; ids without an edit keep their
 * value.  A row whose mask allows nothing becomes -infinity throughout, which
 * arc_sample_batch reports as degenerate.
 *
 * Library: libarcserve.so; conventions as in arc_kv.h.
 */
#ifndef ARC_EDIT_H
#define ARC_EDIT_H

#include <stddef.h>
#include <stdint.h>

#include "../arc_sample.h" /* ARC_OK, ARC_E_*, ARC_F32, ARC_BF16, ARC_F16, arc_row_params */

#ifdef __cplusplus
extern "C" {
#endif

/* device-side error bits, ORed into *err_word (never cleared here) */
#define ARC_EDIT_ERR_PARAM 0x1u /* a penalty is out of its range: the row is edited without penalties */
#define ARC_EDIT_ERR_HIST 0x2u  /* a history id outside [0, V) is left out; offsets that do not ascend within
                                   0 .. hist_len: the row is edited without its history */
#define ARC_EDIT_ERR_BIAS 0x4u  /* the same of the biases */
#define ARC_EDIT_ERR_MASK 0x8u  /* allowed_rows names no row of the mask: the row becomes -infinity throughout */

/* Host struct: what is edited.  Each of the three may be left out (all NULL). */
typedef struct arc_logit_edits {
    const arc_row_params* params;  /* device [B]: the three penalties are read; required with a history */
    const int32_t* hist_offsets;   /* device [B + 1]: row r's history is hist_ids[hist_offsets[r] .. hist_offsets[r+1]) */
    const int32_t* hist_ids;       /* device [hist_len]; an id counts as often as it stands there */
    int64_t hist_len;
    const int32_t* bias_offsets;   /* device [B + 1], likewise */
    const int32_t* bias_ids;       /* device [bias_len] */
    const float* bias;             /* device [bias_len] */
    int64_t bias_len;              /* at most 2^31 - 1, as hist_len */
    const uint32_t* allowed;       /* device [allowed_count][allowed_stride]: bit i % 32 of word i / 32 is id i's */
    int64_t allowed_stride;        /* words from one row of the mask to the next, at least V / 32 rounded up */
    int64_t allowed_count;         /* rows of the mask; at least B without allowed_rows */
    const int32_t* allowed_rows;   /* device [B] or NULL: the mask's row of each row (negative: every id is
                                      allowed); NULL: its own */
} arc_logit_edits;

/*
 *   logits    device [B][ld], ARC_F32, ARC_BF16 or ARC_F16
 *   B, V, ld  rows, vocabulary (at most 2^31 - 1), row stride in elements (ld >= V)
 *   out       device [B][out_ld], dtype or ARC_F32; may be logits with its stride
 *             and type, otherwise it must not overlap.  In place, ids are taken in
 *             groups of eight that begin on the 16-byte boundaries of each row: a
 *             group that the mask allows whole and no list names is neither read nor
 *             written, of the others any value may be written back as it was
 */
int arc_edit_logits(const void* logits, int64_t B, int64_t V, int64_t ld, int32_t dtype, void* out, int64_t out_ld,
                    int32_t out_dtype, const arc_logit_edits* edits, uint32_t* err_word, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ARC_EDIT_H */

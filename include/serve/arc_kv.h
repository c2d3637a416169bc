/*
 * arc_kv.h -- a paged key/value cache in 8 bits for GB300 (sm_103a): appending
 * a step's tokens with the position rotation applied on the way, and attention
 * of those tokens over the cache.
 *
 * The two calls are the part of a decode step before the sampler
 * (arc_sample.h): the positions that arc_decode_commit / arc_sample_batch_commit
 * (arc_decode.h) advance in device memory are read here at every launch, so a
 * captured step replays without a host in the middle.
 *
 * Library: libarcserve.so.  Conventions are those of arc_sample.h: plain
 * device pointers, sizes and a stream; the host arguments are checked before
 * any CUDA call and a negative ARC_E_* code means that nothing was enqueued;
 * nothing is allocated and nothing synchronises; what is found wrong on the
 * device becomes sticky bits in *err_word and leaves the other sequences alone
 * (but for offsets: where one is wrong, those after it say nothing either).
 * Calls are safe inside stream capture once the first call of their kind on
 * the device has returned (it sets kernel attributes).
 *
 * The cache.  Pages of `page_size` tokens; each page holds, for each cached
 * head, page_size rows of head_dim e4m3 codes, and one fp32 scale:
 *     value = code * scale[page][head].
 * A sequence's token t lies in page page_table[sequence][t / page_size], slot
 * t % page_size.  Scales written here are powers of two in [2^-32, 2^32], so
 * a value is exact in bf16 and a page whose scale grows is rewritten by
 * shifting exponents; arc_kv_attend takes any scale in that range.
 */
#ifndef ARC_KV_H
#define ARC_KV_H

#include <stddef.h>
#include <stdint.h>

#include "../arc_sample.h" /* ARC_OK, ARC_E_*, ARC_BF16, ARC_F16 */

#ifdef __cplusplus
extern "C" {
#endif

#define ARC_SERVE_ABI_VERSION 1

/* device-side error bits, ORed into *err_word (never cleared here) */
#define ARC_KV_ERR_PAGE 0x1u     /* page id outside [0, pages): tokens not stored; the attention rows of the
                                    sequence that are computed with such a page are NaN */
#define ARC_KV_ERR_POSITION 0x2u /* tokens past max_pages * page_size: not stored; attention rows of the
                                    sequence are NaN */
#define ARC_KV_ERR_NAN 0x4u      /* a rotated key or a value is NaN: stored as 0 */
#define ARC_KV_ERR_OFFSETS 0x8u  /* row_offsets does not ascend from 0 to T: the first sequence where it does not, and
                                    those after it, are left out; their tokens are not stored, and the rows that
                                    no sequence before them has are NaN in q_out and in the attention */
#define ARC_KV_ERR_SCALE 0x10u   /* a page that holds older tokens has a scale outside [2^-32, 2^32]: the new ones
                                    are not stored under that head, and the page stays as it is */

/* Host struct.  k and v have the same layout. */
typedef struct arc_kv_cache {
    void* k;                /* device, e4m3 [pages][heads][page_size][head_dim] */
    void* v;
    float* k_scale;         /* device, [pages][heads] */
    float* v_scale;
    int64_t page_stride;    /* bytes from one page to the next, a multiple of 16 */
    int64_t head_stride;    /* bytes from one head of a page to the next, a multiple of 16 */
    int32_t pages;
    int32_t heads;          /* cached heads */
    int32_t page_size;      /* 16, 32, 64, 128 or 256 tokens */
    int32_t head_dim;       /* 64, 128 or 256 */
} arc_kv_cache;

/* Host struct: the new tokens of one call and where their sequences live. */
typedef struct arc_kv_step {
    const int32_t* page_table;  /* device, [B][table_stride], the first max_pages of each row are read */
    int64_t table_stride;
    const int32_t* positions;   /* device [B]: tokens held before the new ones = position of the first
                                   new token; negative: the sequence is parked (nothing is stored, its
                                   attention rows are 0) */
    const int32_t* row_offsets; /* device [B + 1] or NULL: new tokens of sequence b are rows
                                   row_offsets[b] .. row_offsets[b + 1] - 1; NULL: one each (T == B) */
    int64_t B;                  /* sequences, at most 2^20 */
    int64_t T;                  /* new tokens in all, at most 2^24 */
    int32_t max_pages;          /* per sequence; max_pages * page_size < 2^31 */
    int32_t reserved;           /* 0 */
} arc_kv_step;

#define ARC_ROPE_HALF 0        /* value i of a head pairs with value i + rot_dim / 2 */
#define ARC_ROPE_INTERLEAVED 1 /* value 2 i pairs with value 2 i + 1 */

/*
 * Host struct: the rotation.  Pair i at position p turns by p * turns[i] *
 * 2^-64 of a full turn: 64-bit fixed point, so that the product's low 64 bits
 * are the exact fraction of a turn at any position.  The rotated pair is
 * multiplied by `amplitude` (1 but for contexts stretched with a factor).
 */
typedef struct arc_rope {
    const uint64_t* turns; /* device [rot_dim / 2] */
    float amplitude;       /* finite, > 0 */
    int32_t rot_dim;       /* even, 0 .. head_dim: the first rot_dim values of a head turn */
    int32_t layout;        /* ARC_ROPE_* */
    int32_t reserved;      /* 0 */
} arc_rope;

/*
 * Append T new tokens, one call a layer and step.
 *   q        device [T][q_heads][head_dim] or NULL: rotated into q_out
 *   k, v     device [T][heads][head_dim]: k is rotated; both are rounded once,
 *            to the nearest code (ties to even), from the exact rotated value
 *   *_stride elements from one token / head to the next; the values of a head
 *            are contiguous.  16-byte aligned rows are read 16 bytes at a time
 *   q_out    may be q itself with the same strides; otherwise it must not overlap.
 *            Rows of parked sequences are 0
 *   dtype    ARC_BF16 or ARC_F16, of q, k, v and q_out
 *   rope     NULL: no rotation
 * A page's scale becomes the least 2^e with amax <= 448 * 2^e over its new
 * tokens, e clamped to [-32, 32], or stays where the page already holds tokens
 * and its scale is as large. A scale that stays may be any number of the range
 * (pages that another program filled): the new codes are the nearest ones under
 * it, and the older ones stay. Where it grows, the tokens held are rewritten as
 * e4m3(code * old scale / new scale); a NaN code stays one.  A page whose first token is new starts from
 * nothing: what it held before does not matter.  Infinities and values above
 * 448 * 2^32 saturate.  Pages are written by this call alone: sequences of one
 * call must not share a page that they append to.
 */
typedef struct arc_kv_rows {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t out_token_stride, out_head_stride;
    int32_t q_heads; /* any number; 0 with q NULL */
    int32_t dtype;
} arc_kv_rows;

int arc_kv_append(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_rows* rows,
                  const arc_rope* rope, uint32_t* err_word, void* stream);

/*
 * Attention of the step's T tokens over the cache, which already holds them.
 * Query head h reads cached head h / (q_heads / heads).  The token at position
 * p sees the tokens j <= p of its sequence, and with window > 0 only those
 * with j > p - window:
 *     out = sum_j softmax_j(scale * q . k_j) v_j
 * Scores, the softmax's maximum and sum and the sums over j are fp32; q enters
 * the products as fp16 after a power-of-two scaling of each row (exact but for
 * values below 2^-24 of the row's largest), the weights as fp16 too, relative to
 * the largest of the 16 tokens (32 for heads of 64) they are multiplied with: off
 * by 2^-11 of themselves at most above 2^-28 of that one, 0 below 2^-39.
 *   out        device, dtype; rows of parked sequences are 0
 *   workspace  device, 16-byte aligned, arc_kv_attend_workspace_bytes(cache)
 *              bytes, zero-filled once before its first use; calls leave it
 *              ready for the next.  Calls that share one must be ordered.
 */
typedef struct arc_kv_query {
    const void* q;
    void* out;
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
    int32_t q_heads;  /* a multiple of cache->heads; T * q_heads / heads <= 2^30 */
    int32_t dtype;    /* ARC_BF16 or ARC_F16 */
    float scale;      /* finite */
    int32_t window;   /* 0: off */
} arc_kv_query;

int arc_kv_attend(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_query* query,
                  uint32_t* err_word, void* workspace, size_t workspace_bytes, void* stream);

/* Host only; 0 for a cache that arc_kv_attend would refuse. */
size_t arc_kv_attend_workspace_bytes(const arc_kv_cache* cache);

/* Text for an ARC_E_* code of this library's calls (static storage). */
const char* arc_serve_strerror(int code);

/* ARC_SERVE_ABI_VERSION of the built library. */
int arc_serve_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* ARC_KV_H */

/*
 * cbs_llm.h -- C ABI of libcbs, the operators of a decoder step on low-bit numbers for AMD Instinct MI355X (gfx950):
 * RMS norm with the residual's addition and int8 rows, a linear layer on 4-bit weights, a paged key/value cache that is
 * quantised as it is written, and attention of new tokens over that cache.
 *
 * rne: round to nearest, ties to even.  fp32(.): rounded once to 32 bits.  T(.): rounded once to the tensor's type.
 *
 * RMS norm, per row:
 *   h = T(x + residual) (h = x without one; h goes to residual_out),  y_i = h_i / sqrt(mean_j h_j^2 + eps) * w_i
 *   output of x's type: T(y);  int8: s = fp32(max_i |y_i| / 127), 1 where that is 0,  q_i = clamp(rne(fp32(y_i / s)), -127, 127).
 *   A row that holds a NaN or an infinity has the scale NaN or infinity, and codes without meaning.  The sum of squares is held in
 *   32 bits: one that leaves them (magnitudes of 2^60 and more) gives zeros, and with eps 0 one that vanishes there infinities.
 * 4-bit linear, groups g of `group` consecutive input features:
 *   y[m][n] = x_scale[m] * sum_g scales[g][n] * sum_{k in g} x[m][k] * (code[n][k] - zero[g][n])
 *   x_scale is 1 for floating rows; zero is 8 where none are given.
 *   The sums of x (code - zero) over 128 input features, times 16, are 32-bit floats: an |x| of 2^108 and more may overflow them
 *   (bfloat16 on few rows: not before the formula's own do).
 * Paged cache, of keys and values of `heads` heads:  slot = page * page_size + place;  a token's vector v of one head is kept as
 *   s = fp32(max_i |v_i| / 127), 1 where that is 0,  q_i = clamp(rne(fp32(v_i / s)), -127, 127)   (cache_dtype CBS_I8)
 *   or as it is (cache_dtype CBS_F16 or CBS_BF16), and read back as T(fp32(q_i * s)) or as it is.  A vector that holds a NaN or an
 *   infinity has the step NaN or infinity, and codes without meaning.
 * Attention: new token i (0 <= i < count) of a sequence that has length tokens, its new ones included, is at
 *   place = length - count + i, and sees key j if 0 <= j < length, causal: j <= place, window w > 0: j > place - w.
 *   out_i = sum_j p_j v_j / sum_j p_j over the keys that it sees, p_j = exp(scale * q_i . k_j - max); 0 where it sees none, or
 *   none but of a score of -infinity.
 *   Head h reads the cache's head h / (heads / kv_heads).  What the cache holds where no key is seen, NaN and infinities
 *   among it, does not reach the output.  With 16-bit queries the weights p_j are rounded to 16 bits before they meet the
 *   values.  One that its type does not hold is zero (over a float16 cache below 2^-32 of the row's largest, else below that of
 *   32 bits), and an infinite value that it meets NaN.
 *
 * Layouts (device memory; strides in elements; the innermost axis is dense):
 *   4-bit codes  uint8 [n][round_up(ceil(k / 2), 16)], input feature 2i in the low nibble of byte i, 2i + 1 in the high one;
 *                bits beyond k are not looked at.  From a 16-byte boundary.
 *   scales       [ceil(k / group)][n] of scale_dtype, zero points uint8 [ceil(k / group)][n].
 *   key cache    [pages][heads][page_size][head_dim];  value cache [pages][heads][head_dim][page_size] (a head's values
 *                lie along the tokens, the order in which attention sums them);  both from a 16-byte boundary.
 *   scales       fp32 [pages][heads][page_size], one each for keys and values (CBS_I8 only).
 *   page table   int32 [seqs][columns]: the page of a sequence's tokens page_size * c and on is column c's.
 *
 * Execution, as in cbs.h: a call only enqueues kernels on the given stream (hipStream_t as void*, NULL: the null stream), so
 * it can be captured into a graph; lengths, page tables and slots are device data and may change between replays.
 * Sums, norms and softmax statistics are held in 32 bits.  Results do not depend on the order in which workgroups run.
 *
 * Errors: every entry point returns a cbs_status; cbs_last_error() has a message for the calling thread.  Device data is
 * checked where it is used: a slot outside [0, pages * page_size) is not written and reads as zeros, a page outside
 * [0, pages) in a table hides its keys, lengths are cut at the table's columns.  A cache of no pages and a table of no columns
 * may be NULL.
 */
#ifndef CBS_LLM_H_
#define CBS_LLM_H_

#include "cbs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further element types of these operators (layers of cbs.h do not take them). */
#define CBS_F16 3
#define CBS_BF16 4

/* ---------------------------------------------------------------- RMS norm */

#define CBS_RMS_MAX_DIM 65536

typedef struct cbs_rms_desc {
    int32_t dim;          /* features of a row, 1 to CBS_RMS_MAX_DIM */
    int32_t dtype;        /* of x, residual and residual_out: CBS_F32, CBS_F16 or CBS_BF16 */
    int32_t out_dtype;    /* dtype, or CBS_I8 */
    int32_t weight_dtype; /* CBS_F32, CBS_F16 or CBS_BF16 */
    float eps;            /* >= 0 */
} cbs_rms_desc;

typedef struct cbs_rms_args {
    const void *x;        /* [rows][dim] */
    const void *residual; /* [rows][dim], NULL: none */
    const void *weight;   /* [dim] */
    void *out;            /* [rows][dim] */
    void *residual_out;   /* [rows][dim]: the sum; NULL: not kept */
    float *out_scale;     /* [rows], out_dtype CBS_I8 only */
    int64_t rows;
    int64_t x_stride, residual_stride, out_stride, residual_out_stride; /* between rows; inputs >= 0, outputs >= dim */
    /* Either output may be x or residual, with as many bytes between its rows, and overlaps nothing else. */
} cbs_rms_args;

/* Errors: CBS_EINVAL (NULL or contradictory argument), CBS_EUNSUPPORTED (a size or type that is not offered), CBS_ELAUNCH. */
cbs_status cbs_rms_norm(const cbs_rms_desc *desc, const cbs_rms_args *args, void *stream);

/* ---------------------------------------------------------------- linear layer on 4-bit weights */

typedef struct cbs_w4_desc {
    int32_t k, n;        /* input and output features, >= 1 */
    int32_t group;       /* input features that share a scale: 32, 64 or a multiple of 128 */
    int32_t dtype;       /* of x: CBS_F32, CBS_F16, CBS_BF16, or CBS_I8 with a scale per row */
    int32_t out_dtype;   /* CBS_F32, CBS_F16 or CBS_BF16 */
    int32_t scale_dtype; /* of scales: CBS_F32, CBS_F16 or CBS_BF16 */
} cbs_w4_desc;

typedef struct cbs_w4_args {
    const void *x;        /* [rows][k] */
    const float *x_scale; /* [rows], dtype CBS_I8 only */
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros; /* NULL: 8 everywhere */
    void *out;            /* [rows][n]; overlaps no input */
    int64_t rows;
    int64_t x_stride, out_stride; /* between rows; x_stride >= 0, out_stride >= n */
} cbs_w4_args;

/* Any number of rows is right; it is made for few of them (64 or less), where reading the codes is the cost. */
cbs_status cbs_w4_linear(const cbs_w4_desc *desc, const cbs_w4_args *args, void *stream);

/* ---------------------------------------------------------------- paged key/value cache */

typedef struct cbs_kv_desc {
    int32_t heads;       /* of the cache, >= 1 */
    int32_t head_dim;    /* a multiple of 16 up to 256 */
    int32_t page_size;   /* tokens of a page: a multiple of 16 up to 1024 */
    int32_t dtype;       /* of the vectors written: CBS_F32, CBS_F16 or CBS_BF16 */
    int32_t cache_dtype; /* CBS_I8, or dtype where that has 16 bits */
    int32_t read_dtype;  /* of the vectors read back: CBS_F32, CBS_F16, CBS_BF16; cache_dtype unless that is CBS_I8 */
} cbs_kv_desc;

typedef struct cbs_kv_args {
    void *k, *v;                                                          /* [tokens][heads][head_dim]; read by a write */
    const int64_t *slots;                                                 /* [tokens] */
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;                                             /* CBS_I8 only */
    int64_t tokens, pages;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride; /* of k and v; >= 0, for a read not overlapping */
} cbs_kv_args;

/* Quantise (or copy) the vectors into their slots.  Of two tokens with one slot, one or the other is kept, or parts of both. */
cbs_status cbs_kv_write(const cbs_kv_desc *desc, const cbs_kv_args *args, void *stream);
/* Read the vectors of the slots back. */
cbs_status cbs_kv_read(const cbs_kv_desc *desc, const cbs_kv_args *args, void *stream);

/* ---------------------------------------------------------------- attention over the paged cache */

typedef struct cbs_attn cbs_attn; /* opaque: the operator's workspace on one device */

typedef struct cbs_attn_desc {
    int32_t heads, kv_heads; /* heads a multiple of kv_heads */
    int32_t head_dim;        /* a multiple of 16 up to 256 */
    int32_t page_size;       /* a multiple of 16 up to 1024 */
    int32_t dtype;           /* of q and out: CBS_F32, CBS_F16 or CBS_BF16 */
    int32_t cache_dtype;     /* CBS_I8, or dtype where that has 16 bits */
    int32_t causal;          /* 0 or 1 */
    int32_t window;          /* keys that a token sees at most, its own included; 0: all */
    float scale;             /* of q . k */
    int32_t max_seqs;        /* sequences of one call at most */
} cbs_attn_desc;

typedef struct cbs_attn_args {
    const void *q;          /* [tokens][heads][head_dim] */
    const int32_t *q_start; /* [seqs + 1]: sequence b has the new tokens q_start[b] to q_start[b + 1] - 1 */
    const int32_t *kv_len;  /* [seqs]: tokens of the sequence, its new ones included */
    const int32_t *table;   /* [seqs][columns] */
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale; /* CBS_I8 only */
    void *out;              /* [tokens][heads][head_dim]; rows of no sequence are not written */
    int64_t tokens, pages;
    int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride, table_stride;
    int32_t seqs, columns;
    int32_t max_new, max_kv; /* most new tokens and most tokens of a sequence: they choose how the work of all of them is
                                split, and where a sequence has more, the result is the same */
} cbs_attn_args;

/* The workspace is allocated here; a run allocates nothing.  One handle runs in one stream at a time. */
cbs_status cbs_attn_create(const cbs_attn_desc *desc, cbs_attn **out);
cbs_status cbs_attn_run(const cbs_attn *attn, const cbs_attn_args *args, void *stream);
/* NULL is a no-op.  No enqueued run may be pending. */
void cbs_attn_destroy(cbs_attn *attn);

#ifdef __cplusplus
}
#endif

#endif /* CBS_LLM_H_ */

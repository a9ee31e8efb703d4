/*
 * attention.h -- C ABI of softmax attention in libwkv7, on MI355X (gfx950):
 * the layers that stand between recurrent ones in a hybrid stack.  The norm
 * and rotation of queries and keys, causal attention over a prompt with its
 * gradients, a paged cache of keys and values, and the attention of new tokens
 * over it.
 *
 * Query head h reads key head h / (Hq / Hk).  Over the tokens j <= i of the
 * same sequence:
 *
 *     s_ij = scale q_i . k_j
 *     y_i = sum_j exp(s_ij - lse_i) v_j,   lse_i = log sum_j exp(s_ij)
 *
 * Layouts (row-major, contiguous unless a stride is given, 16-byte aligned):
 *   q, y, dy, dq      [B][T][Hq][D]   dtype
 *   k, v, dk, dv      [B][T][Hk][D]   dtype
 *   lse               [B][T][Hq]      fp32
 *   k_pages, v_pages  [pages][Hk][page][D]   cache_dtype
 *   k_scale, v_scale  [pages][Hk][page]      fp32, with an 8-bit cache
 *   table             [rows][max_pages]      int32: a row's pages, in order
 *   lens              [rows]                 int32: a row's tokens
 * Strides count elements from a token to the next (0: the heads lie end to
 * end), so that q, k and v may be parts of one projection's output: at least
 * heads times D, a multiple of 8, at most 2^22.  Row b starts at token b T.
 *
 * Sequences.  With nseq == 0 the B rows are B sequences of T tokens.  With
 * nseq > 0, B is 1 and sequence s owns the tokens seq_starts[s] ..
 * seq_starts[s + 1] - 1 (int32 device array of nseq + 1 non-decreasing values
 * in [0, T]).  Lengths of zero are allowed.  Rows of outputs outside every
 * sequence are not written, and values of inputs there reach no result.
 * Starts are read on the device: values outside the range are clamped to it
 * (no access leaves the buffers), and starts that decrease give undefined
 * outputs.
 *
 * Numbers.  Products, sums, the softmax's statistics and the angles' products
 * are held in fp32 or more.  With bf16 inputs the weights of v (and, in the
 * gradients, those of k, q and dy) take part in their products rounded to
 * bf16, one rounding of half a step each, as large as that of the outputs;
 * attn_decode carries them in two bf16 parts, over an 8-bit cache in one.  fp32
 * inputs use the fp32 matrix instruction throughout.  Outputs are rounded once.
 * Results are the same bit for bit from run to run: no sum depends on the order
 * in which workgroups run.  What a token does not see reaches none of its
 * outputs, whatever it holds, and none of its gradients what does not see it.
 * Where results are not finite, their tiles are gone over a second time.  A token
 * whose scores are all minus infinity has NaN for y in attn_forward, and minus
 * infinity for lse: there is no weight to divide by (in attn_decode y is 0).
 *
 * Ownership, execution and errors as for wkv7.h: device pointers owned by the
 * caller, work enqueued on `stream`, nothing allocated or synchronised, every
 * argument validated before anything is enqueued (WKV7_* statuses).  No output
 * may overlap an input or another output, but where it says so.
 */
#ifndef ATTENTION_H
#define ATTENTION_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------- a prompt, and training */

typedef struct {
    int64_t B;      /* batch, >= 0; 1 when nseq > 0 */
    int64_t T;      /* tokens of a row, 0 to 2^30 */
    int64_t Hq;     /* query heads: a multiple of Hk, at most 65535 */
    int64_t Hk;     /* key heads, >= 0 */
    int64_t D;      /* head size: 64 or 128 */
    int64_t nseq;   /* packed sequences (at most 65535), or 0 */
    int64_t q_stride, k_stride, v_stride;
    int32_t dtype;  /* wkv7_dtype */
    int32_t flags;  /* 0 */
    float scale;    /* positive, not denormal, at most 2^127 */
} attn_shape;

/* Bytes of the record attn_forward leaves for attn_backward beside lse: what
 * y's rounding to bf16 took away ([B][T][Hq][D] bf16).  0 with fp32 inputs,
 * and when the shape is invalid or empty. */
size_t attn_record_bytes(const attn_shape *shape);
/* Bytes of device workspace attn_backward needs (a table of the tokens'
 * statistics).  0 when the shape is invalid or empty. */
size_t attn_backward_workspace_bytes(const attn_shape *shape);

/* Forward.  y required (with tokens); lse and record: outputs, NULL to skip. */
int attn_forward(const attn_shape *shape, const void *q, const void *k, const void *v,
                 const int32_t *seq_starts, void *y, float *lse, void *record, hipStream_t stream);

/* Backward, from a forward's y, lse and record (NULL: y alone stands for
 * itself, and its rounding enters dq and dk: their errors in bf16 grow from
 * 1.41 to 1.49 times those of one rounding).  y, dy, dq, dk and dv are contiguous
 * whatever the strides of q, k, v, and required.  dk and dv are summed over the query heads
 * that read them.  workspace: 256-byte aligned. */
int attn_backward(const attn_shape *shape, const void *q, const void *k, const void *v,
                  const int32_t *seq_starts, const void *y, const float *lse, const void *record,
                  const void *dy, void *dq, void *dk, void *dv, void *workspace,
                  size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------- the norm and rotation before them */

/* Per token and head, x of q (weight wq) and of k (wk):
 *     n = x / sqrt(mean(x^2) + eps) * w          (w NULL: n = x)
 * and the first R entries in pairs (a, b), pair i turned by the angle
 * positions[token] * theta[i]:
 *     (a cos - b sin, b cos + a sin)              (theta NULL: z = n)
 * Pair i is (n[i], n[i + R / 2]), or with QK_NORM_INTERLEAVED (n[2 i],
 * n[2 i + 1]).  The angle is the product of the two numbers as they are,
 * formed and reduced in fp64: positions may be as far as int32 goes, and
 * below zero.  positions NULL: a token's place in its row, 0 to T - 1. */
enum {
    QK_NORM_INTERLEAVED = 1
};

typedef struct {
    int64_t B, T;   /* >= 0 */
    int64_t Hq, Hk; /* >= 0, at most 65535 */
    int64_t D;      /* 64 or 128 */
    int64_t R;      /* entries that turn: a multiple of 16 up to D; 0 without theta */
    int64_t q_stride, k_stride;
    int32_t dtype;
    int32_t flags;  /* 0 or QK_NORM_INTERLEAVED */
    float eps;      /* > 0, finite */
} qk_norm_shape;

size_t qk_norm_workspace_bytes(const qk_norm_shape *shape);

/* q, k -> qz, kz [B][T][H][D], contiguous; wq and wk come together or are both
 * NULL; wq, wk [D] and theta [R / 2] fp32, positions [B][T] int32.  qz and kz
 * may be q and k themselves where those are contiguous. */
int qk_norm_forward(const qk_norm_shape *shape, const void *q, const void *k, const float *wq,
                    const float *wk, const float *theta, const int32_t *positions, void *qz,
                    void *kz, hipStream_t stream);

/* From dqz, dkz (contiguous) and the forward's inputs: dq, dk, contiguous, and
 * dwq, dwk [D] fp32 (required with wq, wk, NULL without), summed in a fixed
 * order.  dq and dk may be dqz and dkz themselves. */
int qk_norm_backward(const qk_norm_shape *shape, const void *dqz, const void *dkz, const void *q,
                     const void *k, const float *wq, const float *wk, const float *theta,
                     const int32_t *positions, void *dq, void *dk, float *dwq, float *dwk,
                     void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------- the paged cache */

/* What a cache holds: values of the caller's dtype, or e4m3 with a scale for
 * each token and head. */
enum {
    KV_CACHE_SAME = 0,
    KV_CACHE_E4M3 = 1
};

typedef struct {
    int64_t rows;        /* rows of the table: sequences */
    int64_t T;           /* tokens of k and v for each row, or in all (packed) */
    int64_t Hk, D;       /* D: 64 or 128 */
    int64_t packed;      /* 0, or 1: k and v hold the rows' tokens end to end */
    int64_t pages;       /* pages of the pool, at most 2^31 - 1 */
    int64_t page;        /* tokens of a page: a power of two from 16 to 256 */
    int64_t max_pages;   /* entries of a row of the table; times page at most 2^30 */
    int64_t k_stride, v_stride;
    int32_t dtype;       /* of k and v */
    int32_t cache_dtype; /* KV_CACHE_* */
} kv_cache_shape;

/* Writes k and v, the last tokens of each row, into the row's pages: with n
 * tokens of row r (T, or seq_starts[r + 1] - seq_starts[r]), token i goes to
 * position lens[r] - n + i.  lens counts the new tokens.  A token whose
 * position is below 0 or past the table, or whose page is not in [0, pages), is
 * not written.  One place must not be written twice in a call, by two rows that
 * share a page or by one that names a page twice: what it holds is then undefined.
 *
 * 8 bits: scale = max|x| * (1 / 448 rounded to fp32) over the D entries of a
 * token's head, in fp32, stored e4m3(x / scale), the quotient rounded to fp32,
 * then to nearest, ties to even, at most 448 in magnitude; a head of zeros has
 * scale 0.  A head with an infinity or NaN has NaN in its place. */
int kv_write(const kv_cache_shape *shape, const void *k, const void *v, void *k_pages,
             void *v_pages, float *k_scale, float *v_scale, const int32_t *table,
             const int32_t *lens, const int32_t *seq_starts, hipStream_t stream);

/* The reverse: the last tokens of each row, placed as above, out of its pages
 * into k and v (strides 0): e4m3 value times scale, rounded once.  A
 * token that kv_write would not write is zeros. */
int kv_read(const kv_cache_shape *shape, const void *k_pages, const void *v_pages,
            const float *k_scale, const float *v_scale, const int32_t *table,
            const int32_t *lens, const int32_t *seq_starts, void *k, void *v, hipStream_t stream);

/* --------------------------------------------- new tokens over the cache */

/* The T last tokens of each of B rows, whose keys and values the cache holds
 * already: token t of row b sees the positions below lens[b] - (T - 1 - t).
 * Positions past the table or in a page that is not in [0, pages) are seen by
 * nobody, and what lies there, or behind lens in a page, is not used.  What a
 * later one of the new tokens holds does not reach an earlier one, whatever it
 * is.  A token that sees nothing, or nothing but scores of minus infinity, has
 * y = 0.  (In bf16, whose weights have two parts, an infinity in a v that is seen
 * gives an infinity or NaN.)  lens below 0 count as 0. */
typedef struct {
    int64_t B;           /* rows, at most 65535 */
    int64_t T;           /* new tokens of each row, >= 0 */
    int64_t Hq, Hk, D;   /* as attn_shape */
    int64_t pages, page, max_pages;   /* as kv_cache_shape */
    int64_t q_stride;
    int32_t dtype;       /* of q and y */
    int32_t cache_dtype;
    float scale;
} attn_decode_shape;

/* The cache is read in parts at once, which the workspace joins: as many as
 * fill the device, a number that follows from the shape alone.  0 when one
 * part is enough. */
size_t attn_decode_workspace_bytes(const attn_decode_shape *shape);
int attn_decode(const attn_decode_shape *shape, const void *q, const void *k_pages,
                const void *v_pages, const float *k_scale, const float *v_scale,
                const int32_t *table, const int32_t *lens, void *y, void *workspace,
                size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTENTION_H */

/*
 * gdr.h -- C ABI of the gated delta rule in libwkv7, on MI355X (gfx950): its
 * chunked form with gradients (training, prefill), its recurrent form over a
 * pool of states (decode), and the gated head norm after it.
 *
 * The operation.  For every sequence and value head h independently (key head
 * h / (Hv / Hk)), with the state S[i][j] (i = value row, j = key column), the
 * decay a_t = exp(g_t) and the write strength beta_t:
 *
 *     S_t = a_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     y_t = scale S_t q_t
 *
 * The backward returns the exact gradient of
 *     L = sum_t <dy_t, y_t> + <dsT, S_T>
 * with respect to q, k, v, g, beta and the initial state; the gradients of a
 * key head shared by several value heads are summed over them.
 *
 * Layouts (row-major, contiguous, 16-byte aligned):
 *   q, k, dq, dk        [B][T][Hk][K]    dtype per gdr_shape.dtype
 *   v, y, dy, dv        [B][T][Hv][V]    dtype per gdr_shape.dtype
 *   g, beta, dg, dbeta  [B][T][Hv]       fp32
 *   states s0, sT, dsT, ds0  [sequences][Hv][V][K]  fp32
 *   seq_starts, slots   int32 (16-byte aligned too)
 * g is the log decay, at most 0.  Values of g at or below -200, -inf among them,
 * forget the whole state, and their gradient is exactly zero; k should not be longer than
 * sqrt(2 / beta), or the recurrence itself grows.
 *
 * Sequences.  With nseq == 0 the B rows are B sequences of T tokens.  With
 * nseq > 0, B is 1 and the T tokens hold nseq sequences end to end: sequence
 * s owns the tokens seq_starts[s] .. seq_starts[s + 1] - 1 (int32 device
 * array of nseq + 1 non-decreasing values in [0, T]).  Lengths of zero are
 * allowed: their final state is their initial one.  Tokens outside every
 * sequence are neither read nor written, in any output.  The starts are read
 * on the device: values outside the documented range are clamped to it (no
 * access leaves the buffers), and starts that decrease give undefined outputs.
 * A packed sequence runs in one piece, while few, long rows are cut into segments
 * that run at once: a single long document is faster as a row without starts
 * (65536 tokens x 32 heads of 64, bf16: 1.12 ms, packed 2.84).
 *
 * Numbers.  State, sums and the products inside a chunk are fp32 (fp32
 * inputs), or, with bf16 inputs, products of bf16 parts that carry a value's
 * leading 24 bits, with fp32 sums.  y and the gradients of q, k, v are rounded once, to the inputs'
 * type.  Results are the same bit for bit from run to run.  Tokens of a chunk are
 * computed together: an infinity or NaN in one token's inputs may reach every
 * output of its chunk of 64 and of later (in the gradients also earlier) chunks,
 * of its own sequence and head (key head, in the gradients) alone.
 *
 * Sizes.  At most 65535 sequences and value heads, 2^22 chunks of 64 tokens
 * (as gdr_checkpoint_bytes counts them) times value heads, and, in the
 * chunked calls with V above 128, about 3.7 million sequences times value heads,
 * whose launch has 2^32 threads (WKV7_ERR_UNSUPPORTED beyond, before anything
 * is enqueued).
 *
 * Ownership, execution and errors as for wkv7.h: device pointers owned by the
 * caller, work enqueued on `stream`, nothing allocated or synchronised, every
 * argument validated before anything is enqueued (WKV7_* statuses).
 */
#ifndef GDR_H
#define GDR_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of gdr_shape.flags.
 *   GDR_NORM_QK : q and k are normalised first, x / sqrt(x . x + 1e-6) over
 *     a head's K entries, and dq, dk are the gradients of what was passed. */
enum {
    GDR_NORM_QK = 1
};

typedef struct {
    int64_t B;      /* batch, >= 0; 1 when nseq > 0 */
    int64_t T;      /* tokens of a row, >= 0 */
    int64_t Hk;     /* key heads, >= 0 */
    int64_t Hv;     /* value heads: a multiple of Hk, at most 65535 */
    int64_t K;      /* key size: 64 or 128 */
    int64_t V;      /* value size: a multiple of 16, 16 to 256 */
    int64_t nseq;   /* packed sequences, or 0 */
    int32_t dtype;  /* wkv7_dtype of q, k, v, y, dy, dq, dk, dv */
    int32_t flags;  /* 0 or GDR_NORM_QK */
    float scale;    /* a normal number: finite, not zero, not denormal */
} gdr_shape;

/* Bytes of the record that gdr_forward leaves for gdr_backward: for each
 * chunk of 64 tokens and value head, the state before it ([V][K] fp32) and
 * the chunk's 64 correction rows ([64][V] fp32).  The chunks are those of
 * the rows, B ceil(T / 64), or, packed, at most floor(T / 64) + nseq.
 * 0 when the shape is invalid or empty. */
size_t gdr_checkpoint_bytes(const gdr_shape *shape);

/* Bytes of device workspace gdr_forward and gdr_backward need (the chunks'
 * triangular factors where a kernel of their own makes them, decay tables,
 * and for few, long rows the transitions of their segments; for the backward
 * also the chunks' state gradients and, with ckpt_provided 0, the record).
 * 0 when the shape is invalid or empty, or needs none. */
size_t gdr_forward_workspace_bytes(const gdr_shape *shape);
size_t gdr_backward_workspace_bytes(const gdr_shape *shape, int ckpt_provided);

/* Forward.  q, k, v, g, beta required unless there are no tokens; seq_starts
 * required when nseq > 0 and NULL otherwise; s0 NULL = zeros; y, sT, ckpt:
 * outputs, each NULL to skip.  workspace: 256-byte aligned.  No output may
 * overlap an input. */
int gdr_forward(const gdr_shape *shape, const void *q, const void *k, const void *v, const float *g,
                const float *beta, const float *s0, const int32_t *seq_starts, void *y, float *sT,
                float *ckpt, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Backward.  dy required; dsT NULL = zeros; ckpt: the record a gdr_forward
 * with the same inputs wrote, or NULL to recompute it into the workspace (s0
 * is read only then).  dq, dk, dv, dg, dbeta required; ds0 may be NULL.  No
 * output may overlap an input or another output. */
int gdr_backward(const gdr_shape *shape, const void *q, const void *k, const void *v, const float *g,
                 const float *beta, const float *s0, const int32_t *seq_starts, const void *dy,
                 const float *dsT, const float *ckpt, void *dq, void *dk, void *dv, float *dg,
                 float *dbeta, float *ds0, void *workspace, size_t workspace_bytes,
                 hipStream_t stream);

/* The recurrent form: T >= 0 tokens of each of B sequences, one after the
 * other, from and back into a pool of `pool` states [pool][Hv][V][K] fp32.
 * slots [B] int32 device array: the state of each row, or NULL for row b =
 * state b (pool >= B).  A row whose slot is outside [0, pool), or which an
 * earlier row names too, is skipped: its y is not written, and the state it
 * names is written by the earlier row alone.  shape->nseq must be 0.  y may
 * not overlap an input. */
int gdr_decode(const gdr_shape *shape, const void *q, const void *k, const void *v, const float *g,
               const float *beta, float *state, int64_t pool, const int32_t *slots, void *y,
               hipStream_t stream);

/* The epilogue after the scan, per row (a token's head) of N entries:
 *     z = y / sqrt(mean(y^2) + eps) * w * gate / (1 + exp(-gate))
 * y, gate, z, dz, dy, dgate [rows][H][N] of `dtype`, w and dw [Hw][N] fp32
 * with Hw = 1 (one weight for all heads) or H.  N is a power of two from 16
 * to 256.  The backward sums dw in a fixed order through a workspace of
 * gdr_epilogue_workspace_bytes bytes, 256-byte aligned.  No output may overlap
 * an input. */
typedef struct {
    int64_t rows;   /* tokens, >= 0; rows times H at most 2^38 */
    int64_t H;      /* heads, >= 0; at most 65535 with a weight for each */
    int64_t N;      /* entries of a head */
    int64_t Hw;     /* heads of the weight: 1 or H */
    int32_t dtype;  /* wkv7_dtype */
    int32_t flags;  /* 0 */
    float eps;      /* > 0, finite */
} gdr_epilogue_shape;

size_t gdr_epilogue_workspace_bytes(const gdr_epilogue_shape *shape);
int gdr_epilogue_forward(const gdr_epilogue_shape *shape, const void *y, const void *gate,
                         const float *w, void *z, hipStream_t stream);
int gdr_epilogue_backward(const gdr_epilogue_shape *shape, const void *dz, const void *y,
                          const void *gate, const float *w, void *dy, void *dgate, float *dw,
                          void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */

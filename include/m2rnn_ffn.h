/*
 * m2rnn_ffn.h -- C ABI of the feed-forward half of a layer (libm2rnn.so,
 * sm_103a): the residual's addition with the RMS norm behind it, the gated
 * feed-forward products, and their 8-bit form.  Statuses, ownership, streams
 * and the device status word are those of m2rnn.h: device pointers of the
 * caller, 16-byte aligned, on the current device; asynchronous on `stream`;
 * outputs overwritten; no allocation; no pointer kept; argument errors found
 * on the host before anything is launched.
 *
 * Rows.  Operators here act on each token by itself.  The inputs of the norm and of the
 * quantiser are [B,T,D] with the row description of m2rnn_block.h (NULL: contiguous); the
 * products take M tokens whose rows are `x_row` (and so on) elements apart.  Distances are
 * multiples of 16 bytes.  Weights, scales, incoming gradients (dy, dr, dh) and outputs are
 * contiguous.  An
 * output must not overlap an input or another output except where a function
 * says that it may (M2RNN_ERR_INVALID_ARG).
 *
 * 8 bits.  M2RNN_E4M3 codes (1 sign, 4 exponent, 3 mantissa bits; largest 448)
 * with one fp32 scale per row: scale = max|row| / 448, code = the nearest e4m3
 * value of row / scale, ties to even.  A row of zeros has scale 0 and codes 0;
 * a value that is not finite makes its whole row NaN or infinite.
 *
 * Gradients of activations and of weights are summed in fp32 and rounded once to
 * in_dtype (a weight's gradient has the weight's type); that of the norm's weight is
 * fp32.  Every sum runs in a fixed order: the same inputs give the same bits.
 */
#ifndef M2RNN_FFN_H_
#define M2RNN_FFN_H_

#include "m2rnn_block.h" /* m2rnn_rows */

#ifdef __cplusplus
extern "C" {
#endif

/* ---- residual and norm -----------------------------------------------------
 *
 *     r = x + res,   y = w (.) r (mean_d r^2 + eps)^(-1/2)
 *
 * The sum is rounded to in_dtype as it is stored, and y is the norm of what is
 * stored.  res NULL: r = x and the argument `r` must be NULL.
 *   x, res [B,T,D] in_dtype (rows)   w [D] in_dtype or NULL (1)
 *   r, y [B,T,D] in_dtype;  q [B,T,D] e4m3 and scale [B,T] fp32 (the 8-bit form of y, before
 *   y is rounded; the root leaves y / scale = 448 w r / max|w r|, so with bf16 inputs the codes are
 *   the formula's, ties included)
 * D a multiple of 8 up to 16384, B, T >= 0, B*T < 2^31, B*T*D < 2^40; eps >= 0 (with eps = 0
 * a zero row gives NaN, as the formula does).  `r` may be `res` or `x` itself (in
 * place, contiguous). */
typedef struct {
    int B, T, D;
    int in_dtype; /* m2rnn_dtype of x, res, w, r, y, dy, dr, dx */
} m2rnn_norm_shape;

int m2rnn_add_norm_fwd(const m2rnn_norm_shape *s, const void *x, const m2rnn_rows *x_rows,
                       const void *res, const m2rnn_rows *res_rows, const void *w, float eps,
                       void *r, void *y, void *stream);

int m2rnn_add_norm_q8(const m2rnn_norm_shape *s, const void *x, const m2rnn_rows *x_rows,
                      const void *res, const m2rnn_rows *res_rows, const void *w, float eps,
                      void *r, void *q, float *scale, void *stream);

size_t m2rnn_add_norm_bwd_workspace_size(const m2rnn_norm_shape *s);

/* Gradients for dL/dy = dy and dL/dr = dr past the norm (NULL = 0), both [B,T,D] in_dtype:
 * dx [B,T,D] in_dtype, which is the gradient of x and of res alike, and dw [D]
 * fp32 (NULL: not wanted, and no workspace needed).  r (rows) is the norm's input.  dx may
 * be dr or dy itself. */
int m2rnn_add_norm_bwd(const m2rnn_norm_shape *s, const void *r, const m2rnn_rows *r_rows,
                       const void *w, float eps, const void *dy, const void *dr, void *dx,
                       float *dw, void *workspace, size_t ws_bytes, void *stream);

/* Codes and scales of x's rows (an activation, or a weight matrix laid out once): s->D up
 * to 2^20. */
int m2rnn_quant_rows(const m2rnn_norm_shape *s, const void *x, const m2rnn_rows *x_rows, void *q,
                     float *scale, void *stream);

/* ---- gated feed-forward products -------------------------------------------
 *
 *     g = x wg^T,  u = x wu^T,  h = act(g) (.) u
 *
 *   x [M,D] (rows x_row >= D apart), wg, wu [F,D], h, dh [M,F], dx [M,D], dwg, dwu [F,D], all in_dtype
 * act: 0 SiLU g / (1 + e^-g), 1 GELU in its tanh form.  D a multiple of 8 up to 2^16, F
 * of 8 up to 2^20, 0 <= M < 2^31, M*D and M*F < 2^40, D*F < 2^38.  Products are summed in
 * fp32; with fp32 inputs every operand is held whole (three bf16 terms), and where a product
 * meets a value that is not finite the result may be NaN in place of an infinity.  The backward
 * pass forms g and u again.  Between its products their gradients are held in bf16 terms: three
 * with fp32 inputs, two with bf16 ones, so that every gradient of the call is rounded once, at
 * all sizes.
 *
 * act | M2RNN_GLU_ROUND (bf16 only): they are rounded to one bf16 value there, as separate bf16
 * operations would leave them.  The backward pass then takes 50 to 65 % of the time and half of
 * that workspace, and dx, dwg and dwu are off by two roundings (relative 2-norm 2.35e-3, not
 * 1.66e-3).  The other functions take the flag and do nothing else for it. */
#define M2RNN_GLU_ROUND 16
typedef struct {
    long long M;
    int D, F;
    int in_dtype; /* m2rnn_dtype of x, wg, wu, h and the gradients */
    int act;      /* 0 or 1, also with M2RNN_GLU_ROUND */
} m2rnn_glu_shape;

/* Workspace of the forward pass (0 with bf16 inputs). */
size_t m2rnn_glu_fwd_workspace_size(const m2rnn_glu_shape *s);

int m2rnn_glu_fwd(const m2rnn_glu_shape *s, const void *x, long long x_row, const void *wg,
                  const void *wu, void *h, void *workspace, size_t ws_bytes, void *stream);

size_t m2rnn_glu_bwd_workspace_size(const m2rnn_glu_shape *s);

/* Gradients for dL/dh = dh.  dx NULL, or dwg and dwu NULL together: not wanted. */
int m2rnn_glu_bwd(const m2rnn_glu_shape *s, const void *x, long long x_row, const void *wg,
                  const void *wu, const void *dh, void *dx, void *dwg, void *dwu,
                  void *workspace, size_t ws_bytes, void *stream);

/* The forward pass on e4m3 x [M,D] (rows), wg, wu [F,D] with scales xs [M], wgs, wus [F];
 * h in in_dtype, which must be M2RNN_BF16.  D a multiple of 16, F of 8. */
int m2rnn_glu_q8(const m2rnn_glu_shape *s, const void *x, long long x_row, const float *xs,
                 const void *wg, const float *wgs, const void *wu, const float *wus, void *h,
                 void *stream);

/* ---- 8-bit product ------------------------------------------------------------
 *
 *     y[m,f] = xs[m] ws[f] sum_d x[m,d] w[f,d] + res[m,f]
 *
 *   x [M,D] e4m3 (rows), xs [M], w [F,D] e4m3, ws [F], res [M,F] (rows) or NULL (0) and
 *   y [M,F] in in_dtype, which must be M2RNN_BF16.  Sizes as for m2rnn_glu_q8; act has no effect (0).
 * y may be res itself (in place, contiguous). */
int m2rnn_linear_q8(const m2rnn_glu_shape *s, const void *x, long long x_row, const float *xs,
                    const void *w, const float *ws, const void *res, long long res_row, void *y,
                    void *stream);

#ifdef __cplusplus
}
#endif
#endif /* M2RNN_FFN_H_ */

/*
 * m2rnn_block.h -- C ABI of the operators that stand around the M2RNN
 * recurrence in one mixer block (libm2rnn.so, sm_103a): the short causal
 * convolution with SiLU in front of it, the norm of queries and keys for
 * each head with the position rotation, and the selective scan, the linear
 * recurrence with the same state layout that a hybrid model puts beside it.
 * Each has a form for whole sequences, a backward pass and a form for single
 * tokens.  Statuses, ownership, streams and the device status word are those
 * of m2rnn.h: device pointers of the caller, 16-byte aligned, on the current
 * device; asynchronous on `stream`; outputs overwritten; no allocation; no
 * pointer kept; argument errors found on the host before anything is
 * launched.
 *
 * Rows.  An input that is a slice of a wider buffer (q, k and v out of one
 * [B,T,C] projection) is described by an m2rnn_rows: the distance in
 * elements from one batch item to the next and from one token to the next.
 * What follows the token (channels, or heads x features) is packed.  Both
 * are >= 0 and, except for the scan's `a`, multiples of 16 bytes
 * (M2RNN_ERR_MISALIGNED otherwise).  A null m2rnn_rows pointer means a
 * contiguous tensor.  Outputs are always contiguous.  An output must not overlap
 * an input or another output except where a function says that it may.
 *
 * Gradients.  The gradients of activations (dx, dq, dk, dv, da) are summed
 * in fp32 and rounded once to in_dtype, the type the preceding layer takes
 * them in; those of parameters and of fp32 states are fp32.  Every sum runs
 * in a fixed order: the same inputs give the same bits.
 */
#ifndef M2RNN_BLOCK_H_
#define M2RNN_BLOCK_H_

#include "m2rnn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    long long batch; /* elements from batch item b to b + 1 */
    long long token; /* elements from token t to t + 1 */
} m2rnn_rows;

/* ---- short causal convolution --------------------------------------------
 *
 *     z[b,t,c] = bias[c] + sum_{i<W} w[c,i] F[b,t+i,c],
 *     y = z sigmoid(z)  (silu = 1)   or   y = z  (silu = 0)
 *
 * where F = [state; x] along time: the W - 1 inputs before the call, then x.
 * The carried state after the call is F's last W - 1 rows.
 *   x      [B,T,C] in_dtype (rows)          w     [C,W] in_dtype
 *   bias   [C] in_dtype or NULL (0)         state [B,W-1,C] in_dtype or NULL (0)
 *   y      [B,T,C] in_dtype                 state_out [B,W-1,C] in_dtype or NULL
 * C a multiple of 8 up to 2^24, W in {2, 3, 4}, B >= 1, 0 <= T <= 2^30,
 * B*T*C < 2^40.
 * T = 0 copies the state. */
typedef struct {
    int B, T, C, W;
    int in_dtype;   /* m2rnn_dtype of x, w, bias, state, y, dx, dstate */
    int grad_dtype; /* m2rnn_dtype of dy: M2RNN_F32 or in_dtype (backward only) */
    int silu;       /* 1: SiLU after the convolution, 0: none */
} m2rnn_conv_shape;

/* y and state_out must overlap neither x, state nor each other: other tokens' runs
 * still read those (M2RNN_ERR_INVALID_ARG; so for dx and dstate below). */
int m2rnn_conv_fwd(const m2rnn_conv_shape *s, const void *x, const m2rnn_rows *x_rows,
                   const void *w, const void *bias, const void *state, void *y,
                   void *state_out, void *stream);

size_t m2rnn_conv_bwd_workspace_size(const m2rnn_conv_shape *s);

/* Gradients for dL/dy = dy ([B,T,C] grad_dtype) and dL/dstate_out =
 * dstate_out ([B,W-1,C] in_dtype, NULL = 0): dx [B,T,C] in_dtype, dw [C,W]
 * fp32, dbias [C] fp32 or NULL, dstate [B,W-1,C] in_dtype or NULL. */
int m2rnn_conv_bwd(const m2rnn_conv_shape *s, const void *x, const m2rnn_rows *x_rows,
                   const void *w, const void *bias, const void *state, const void *dy,
                   const void *dstate_out, void *dx, float *dw, float *dbias, void *dstate,
                   void *workspace, size_t ws_bytes, void *stream);

/* One token for B sequences (T must be 1): x, y [B,C]; state and state_out
 * are required; state_out may be state itself (in place), otherwise they must
 * not overlap. */
int m2rnn_conv_step(const m2rnn_conv_shape *s, const void *x, const m2rnn_rows *x_rows,
                    const void *w, const void *bias, const void *state, void *y,
                    void *state_out, void *stream);

/* ---- norm of queries and keys, with the position rotation -------------------
 *
 * For each of the Nq + Nk heads of a token, over its K features:
 *     u = w (.) x (mean_k x^2 + eps)^(-1/2)
 * with w = wq for queries and wk for keys (NULL = 1; the L2 norm is w =
 * K^(-1/2)), then the first R features turn by the token's angles: with p =
 * pos[b,t] (or t), c = cos[p,i], n = sin[p,i], i < R/2,
 *     (u1, u2) -> (u1 c - u2 n, u2 c + u1 n)
 * where the pair is features (i, i + R/2), or (2i, 2i+1) if interleaved.
 *   q, qo [B,T,Nq,K], k, ko [B,T,Nk,K] in_dtype (q, k: rows)
 *   wq, wk [K] in_dtype or NULL;  cos, sin [P,R/2] fp32 (NULL if R = 0)
 *   pos [B,T] int32 or NULL (then token t has position t, and T <= P)
 * K a multiple of 8 up to 256; R a multiple of 8, 0 <= R <= K; Nq >= 1,
 * Nk >= 0 (k, ko, wk NULL when 0); eps >= 0 (with eps = 0 a zero row gives
 * NaN, as the formula does).  A position outside [0, P) records
 * M2RNN_ERR_BOUNDS in the device status word (in either build) and gives NaN
 * in the token's rotated features. */
typedef struct {
    int B, T, Nq, Nk, K;
    int R;           /* rotated features per head */
    int P;           /* rows of the cos and sin tables */
    int in_dtype;    /* m2rnn_dtype of q, k, wq, wk, qo, ko, dq, dk */
    int grad_dtype;  /* m2rnn_dtype of dqo, dko: M2RNN_F32 or in_dtype (backward only) */
    int interleaved; /* pairs (2i, 2i+1) instead of (i, i + R/2) */
} m2rnn_qk_shape;

int m2rnn_qk_norm_fwd(const m2rnn_qk_shape *s, const void *q, const m2rnn_rows *q_rows,
                      const void *k, const m2rnn_rows *k_rows, const void *wq, const void *wk,
                      float eps, const float *cos, const float *sin, const int *pos, void *qo,
                      void *ko, void *stream);

size_t m2rnn_qk_norm_bwd_workspace_size(const m2rnn_qk_shape *s);

/* Gradients for dL/dqo = dqo, dL/dko = dko (grad_dtype, contiguous):
 * dq, dk in_dtype; dwq, dwk [K] fp32 (each NULL if not wanted). */
int m2rnn_qk_norm_bwd(const m2rnn_qk_shape *s, const void *q, const m2rnn_rows *q_rows,
                      const void *k, const m2rnn_rows *k_rows, const void *wq, const void *wk,
                      float eps, const float *cos, const float *sin, const int *pos,
                      const void *dqo, const void *dko, void *dq, void *dk, float *dwq,
                      float *dwk, void *workspace, size_t ws_bytes, void *stream);

/* ---- selective scan ----------------------------------------------------------
 *
 * The linear recurrence with the state of the M2RNN layer, per (b, n):
 *     dt_t = softplus(a_t + beta_n),   f_t = exp(-alpha_n dt_t)
 *     H_t  = f_t H_{t-1} + dt_t k_t v_t^T,     y_t = H_t^T q_t + w_r (.) v_t
 * Shapes, layouts and the sharing of q and k by groups of heads are those of
 * m2rnn_shape (K in {16,32,64,128}, V in {16,32}; ckpt_every is ignored), for
 * whole sequences with T <= 2^30 and N <= 2^20:
 *   q, k [B,T,Nq,K], v [B,T,N,V], a [B,T,N] in_dtype (rows)
 *   alpha, beta [N] in_dtype; w_r [N,V] in_dtype or NULL (0)
 *   H0, H_T [B,N,K,V] fp32 or NULL;   y [B,T,N,V] in_dtype
 * alpha < 0 is not rejected (the formula is evaluated as given).  a = -inf
 * gives dt = 0: the token leaves the state as it is (padding; its k and v have to
 * be finite).  y_t depends on no later token, whatever that holds; of its own and
 * earlier tokens an infinity may come out as NaN.  In gradients a value that is not
 * finite spreads over its neighbours. */
typedef struct {
    m2rnn_rows q, k, v, a;
} m2rnn_scan_rows;

/* Bytes of `saved`: what the forward pass can keep for the backward pass (the
 * state before every 64th token and the gate's sums).  0 when T = 0. */
size_t m2rnn_scan_saved_size(const m2rnn_shape *s);

/* Least bytes of workspace of m2rnn_scan_fwd; saved_given = 1 when `saved` is
 * passed (0 then).  With fewer than m2rnn_scan_saved_size bytes, which bf16
 * inputs allow (room for the fp32 states of half of the sequences), the call runs
 * the sequences in two parts, one after the other, with the same results;
 * m2rnn_scan_saved_size bytes let it run them at once. */
size_t m2rnn_scan_fwd_workspace_size(const m2rnn_shape *s, int saved_given);

/* saved: m2rnn_scan_saved_size(s) bytes, or NULL. */
int m2rnn_scan_fwd(const m2rnn_shape *s, const m2rnn_scan_rows *rows, const void *q,
                   const void *k, const void *v, const void *a, const void *alpha,
                   const void *beta, const void *w_r, const float *H0, void *y, float *H_T,
                   void *saved, void *workspace, size_t ws_bytes, void *stream);

size_t m2rnn_scan_bwd_workspace_size(const m2rnn_shape *s, int saved_given);

/* Gradients for dL/dy = dy ([B,T,N,V] in_dtype) and dL/dH_T = dH_T (NULL = 0).
 *   saved : from m2rnn_scan_fwd with the same inputs, or NULL (recomputed
 *           into the workspace)
 *   dq, dk [B,T,Nq,K] (summed over each group's heads), dv [B,T,N,V],
 *   da [B,T,N] : in_dtype;  dalpha, dbeta [N], dw_r [N,V] : fp32 (dw_r NULL
 *   exactly when w_r is);  dH0 [B,N,K,V] fp32 or NULL. */
int m2rnn_scan_bwd(const m2rnn_shape *s, const m2rnn_scan_rows *rows, const void *q,
                   const void *k, const void *v, const void *a, const void *alpha,
                   const void *beta, const void *w_r, const float *H0, const void *saved,
                   const void *dy, const float *dH_T, void *dq, void *dk, void *dv, void *da,
                   float *dalpha, float *dbeta, float *dw_r, float *dH0, void *workspace,
                   size_t ws_bytes, void *stream);

/* One token for B sequences (s->T must be 1): q, k [B,Nq,K], v, y [B,N,V],
 * a [B,N]; of the rows only the batch distances are read.  H_out may be H_in
 * itself (in place), otherwise the two must not overlap. */
int m2rnn_scan_step(const m2rnn_shape *s, const m2rnn_scan_rows *rows, const void *q,
                    const void *k, const void *v, const void *a, const void *alpha,
                    const void *beta, const void *w_r, const float *H_in, float *H_out, void *y,
                    void *stream);

#ifdef __cplusplus
}
#endif
#endif /* M2RNN_BLOCK_H_ */

// m2rnn_block.h (internal) -- launch parameters of the block operators
// (convolution, q/k norm, selective scan) and the host checks that the API
// layer shares with m2rnn_api.cu.  Not part of the public ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/m2rnn_block.h"
#include "m2rnn_internal.h"

namespace m2rnn {

// m2rnn_api.cu: the current device with its status word and SM count, and the
// test that every tensor pointer passes.
int host_device_info(int* dev, int** status, int* sms);
int host_check_ptr(const void* p, int dev, bool required);
// The same for a required tensor that is read element by element (aligned to
// `unit` bytes only).
int host_check_elem_ptr(const void* p, int dev, size_t unit);

// Location codes of the block operators' index checks.
enum BlockCheckSite : int {
  CHK_CONV_IN = 501,     // x, state, dy, dstate_out loads
  CHK_CONV_OUT = 502,    // y, dx, dstate, state_out stores
  CHK_CONV_PARAM = 503,  // w, bias loads, dw, dbias partials and sums
  CHK_QK_IN = 601,       // q, k, dqo, dko loads
  CHK_QK_OUT = 602,      // qo, ko, dq, dk stores
  CHK_QK_PARAM = 603,    // wq, wk loads, dw partials and sums
  CHK_QK_POS = 604,      // a position outside the table (reported in every build)
  CHK_SCAN_IN = 701,     // q, k, v, a, dy loads
  CHK_SCAN_OUT = 702,    // y, dq, dk, dv, da stores
  CHK_SCAN_STATE = 703,  // H0, H_T, dH_T, dH0
  CHK_SCAN_WS = 704,     // saved and workspace
  CHK_SCAN_PARAM = 705,  // alpha, beta, w_r loads, parameter gradients
};

struct ConvParams {
  const void *x, *w, *bias, *state, *dy, *dstate_out;
  void *y, *state_out, *dx, *dstate;
  float *dw, *dbias;   // [C,W], [C]
  float* part;         // backward: [nparts][C][W+1] sums of dw, dbias
  long long xb, xt;    // x rows
  int B, T, C, W;
  int TT;              // tokens per thread
  int nT;              // chunks of TT tokens
  int nparts;
  int* status;
};
cudaError_t launch_conv_fwd(const ConvParams& p, bool f32, bool silu, cudaStream_t st);
cudaError_t launch_conv_step(const ConvParams& p, bool f32, bool silu, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvParams& p, bool f32, bool grad_f32, bool silu,
                            cudaStream_t st);
int conv_fwd_tokens(const m2rnn_conv_shape* s, int sms);
void conv_bwd_plan(const m2rnn_conv_shape* s, int* TT, int* nT, int* nparts);

struct QkParams {
  const void *q, *k, *wq, *wk, *dqo, *dko;
  const float *cs, *sn;
  const int* pos;
  void *qo, *ko, *dq, *dk;
  float *dwq, *dwk;
  float* part;         // backward: [nparts][2][K]
  long long qb, qt, kb, kt;
  long long tokens;    // B * T
  int T, Nq, Nk, K, R, P;
  int interleaved;
  int split;           // lane groups per token
  int nparts;
  float eps;
  int* status;
};
cudaError_t launch_qk_fwd(const QkParams& p, bool f32, cudaStream_t st);
cudaError_t launch_qk_bwd(const QkParams& p, bool f32, bool grad_f32, cudaStream_t st);
int qk_split(const m2rnn_qk_shape* s);
int qk_bwd_parts(const m2rnn_qk_shape* s);

struct ScanStepParams {
  const void *q, *k, *v, *a, *alpha, *beta, *w_r;
  const float* H_in;
  float* H_out;
  void* y;
  long long qb, kb, vb, ab;
  int B, N, Nq, K;
  int* status;
};
cudaError_t launch_scan_step(const ScanStepParams& p, int V, bool f32, cudaStream_t st);

// Selective scan over whole sequences (m2rnn_scan_*.cu).
constexpr int kChunk = 64;    // tokens per chunk
constexpr int kCols = 64;     // value columns per head block: 64 / V heads
constexpr int kGate = 4 * kChunk;  // gate values of a chunk and head

struct ScanParams {
  const void *q, *k, *v, *a, *alpha, *beta, *w_r;
  const float* H0;
  void* y;
  float* HT;
  const void* dy;
  const float* dHT;
  void *dq, *dk, *dv, *da;
  float *dalpha, *dbeta, *dw_r, *dH0;
  long long qb, qt, kb, kt, vb, vt, ab, at;  // rows
  int B, T, N, Nq, K, V;
  int nc;         // chunks
  int hpg, nhb;   // heads per group, head blocks per group
  int nseg, cps;  // segments of a sequence in the state kernels, chunks in each
  int hsplit;     // CTAs that share a chunk's head blocks
  // The gate's values of a chunk, [B][N][nc][4][64]: sums of log2 decay from the
  // token's 16-block's start (loc); dt; the token's weight at its block's end,
  // dt 2^(block's sum - loc); what loc's rounding leaves of its sum.
  float* gate;
  float* cdec;    // [B][N][nc]: log2 decay from the segment's start to the chunk
  float* Hl;      // [B][Nq * nhb][nc][64 x K]: states before each chunk, without what
                  // came before their segment
  float* Hseg;    // [B][Nq * nhb][nseg][64 x K]: states at the segments' ends
  float* rdec;    // cdec, Hl and Hseg of the reverse states
  float* Rl;
  float* Rseg;
  float* dqk;     // hsplit > 1: [hsplit][2][B][T][Nq][K] shares of dq, dk
  float* part;    // [B * nc][N * (2 + V)] shares of dalpha, dbeta, dw_r
  int* status;
};
cudaError_t launch_scan_states(const ScanParams& p, bool f32, bool reverse, cudaStream_t st);
cudaError_t launch_scan_out(const ScanParams& p, bool f32, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanParams& p, bool f32, cudaStream_t st);

}  // namespace m2rnn

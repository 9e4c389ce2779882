// m2rnn_block_api.cu -- the extern "C" entry points declared in
// include/m2rnn_block.h: argument validation and launch planning of the
// convolution, the q/k norm and the selective scan.
#include <cuda_runtime.h>

#include <cstdint>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"

namespace {

using m2rnn::host_check_ptr;
using m2rnn::host_device_info;
using m2rnn::overlap_spans;
using m2rnn::read_rows;
using m2rnn::rows_overlap;

int status_from_cuda(cudaError_t e) { return e == cudaSuccess ? M2RNN_OK : M2RNN_ERR_CUDA; }

bool is_dtype(int d) { return d == M2RNN_F32 || d == M2RNN_BF16; }
size_t esize(int dtype) { return dtype == M2RNN_F32 ? 4 : 2; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

bool overlap(const void* a, const void* b, size_t bytes) { return overlap_spans(a, bytes, b, bytes); }

int check_all(const void* const* ptrs, int n, int dev, bool required) {
  for (int i = 0; i < n; ++i) {
    const int rc = host_check_ptr(ptrs[i], dev, required);
    if (rc != M2RNN_OK) return rc;
  }
  return M2RNN_OK;
}
template <int N>
int require(const void* const (&ptrs)[N], int dev) {
  return check_all(ptrs, N, dev, true);
}
template <int N>
int allow(const void* const (&ptrs)[N], int dev) {
  return check_all(ptrs, N, dev, false);
}

// ---- convolution ---------------------------------------------------------------

int check_conv(const m2rnn_conv_shape* s, bool backward) {
  if (s == nullptr) return M2RNN_ERR_INVALID_ARG;
  if (s->B < 1 || s->T < 0 || s->C < 1) return M2RNN_ERR_INVALID_ARG;
  if (!is_dtype(s->in_dtype) || (s->silu != 0 && s->silu != 1)) return M2RNN_ERR_INVALID_ARG;
  if (backward && s->grad_dtype != M2RNN_F32 && s->grad_dtype != s->in_dtype)
    return M2RNN_ERR_INVALID_ARG;
  if (s->C % 8 != 0 || s->W < 2 || s->W > 4) return M2RNN_ERR_UNSUPPORTED_SHAPE;
  if (s->C > (1 << 24) || s->T > (1 << 30)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<double>(s->B) * (static_cast<double>(s->T) + s->W) * s->C >= 1099511627776.0)
    return M2RNN_ERR_UNSUPPORTED_SHAPE;  // 2^40
  return M2RNN_OK;
}

size_t conv_state_bytes(const m2rnn_conv_shape* s) {
  return static_cast<size_t>(s->B) * (s->W - 1) * s->C * esize(s->in_dtype);
}

// The outputs of a whole sequence's convolution (`y`, like x in size, and `so`, like
// the state) over what neighbouring runs still read: x's rows and the others of `in`
// (of the type's or, dy, of ge bytes).
bool conv_outputs_overlap(const m2rnn_conv_shape* s, const m2rnn_rows& xr, const void* x, const void* dy,
                          size_t ge, const void* state, const void* state2, const void* y, const void* so) {
  const size_t e = esize(s->in_dtype), sb = conv_state_bytes(s);
  const size_t n = static_cast<size_t>(s->B) * s->T * s->C;
  const struct { const void* p; size_t bytes; } outs[] = {{y, n * e}, {so, sb}};
  for (const auto& o : outs) {
    if (o.p == nullptr || o.bytes == 0) continue;
    if (rows_overlap(x, xr, s->B, s->T, s->C, e, o.p, o.bytes)) return true;
    if (dy != nullptr && n > 0 && overlap_spans(dy, n * ge, o.p, o.bytes)) return true;
    for (const void* st : {state, state2})
      if (st != nullptr && overlap_spans(st, sb, o.p, o.bytes)) return true;
  }
  return y != nullptr && so != nullptr && overlap_spans(y, n * e, so, sb) && n > 0;
}

m2rnn::ConvParams conv_params(const m2rnn_conv_shape* s, const m2rnn_rows& xr, const void* x,
                              const void* w, const void* bias, const void* state, int* status) {
  m2rnn::ConvParams p{};
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.state = state;
  p.xb = xr.batch;
  p.xt = xr.token;
  p.B = s->B;
  p.T = s->T;
  p.C = s->C;
  p.W = s->W;
  p.status = status;
  return p;
}

// ---- q/k norm -----------------------------------------------------------------

int check_qk(const m2rnn_qk_shape* s, bool backward) {
  if (s == nullptr) return M2RNN_ERR_INVALID_ARG;
  if (s->B < 1 || s->T < 0 || s->Nq < 1 || s->Nk < 0 || s->K < 1 || s->R < 0 || s->P < 0)
    return M2RNN_ERR_INVALID_ARG;
  if (!is_dtype(s->in_dtype) || (s->interleaved != 0 && s->interleaved != 1))
    return M2RNN_ERR_INVALID_ARG;
  if (backward && s->grad_dtype != M2RNN_F32 && s->grad_dtype != s->in_dtype)
    return M2RNN_ERR_INVALID_ARG;
  if (s->K % 8 != 0 || s->K > 256 || s->R > s->K || s->R % 8 != 0)
    return M2RNN_ERR_UNSUPPORTED_SHAPE;
  if (s->Nq >= (1 << 20) || s->Nk >= (1 << 20)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
  const double tokens = static_cast<double>(s->B) * s->T;
  if (tokens >= 2147483648.0 ||
      tokens * (static_cast<double>(s->Nq) + s->Nk) * s->K >= 1099511627776.0)
    return M2RNN_ERR_UNSUPPORTED_SHAPE;  // 2^31 tokens, 2^40 elements
  return M2RNN_OK;
}

// The arguments that both passes share.
int qk_common(const m2rnn_qk_shape* s, const void* q, const m2rnn_rows* q_rows, const void* k,
              const m2rnn_rows* k_rows, const void* wq, const void* wk, float eps,
              const float* cs, const float* sn, const int* pos, bool backward,
              m2rnn::QkParams* p, int* sms) {
  int rc = check_qk(s, backward);
  if (rc != M2RNN_OK) return rc;
  if (!(eps >= 0.f)) return M2RNN_ERR_INVALID_ARG;  // also rejects NaN
  m2rnn_rows qr, kr;
  rc = read_rows(q_rows, s->T, static_cast<long long>(s->Nq) * s->K, s->in_dtype, 16, &qr);
  if (rc != M2RNN_OK) return rc;
  rc = read_rows(k_rows, s->T, static_cast<long long>(s->Nk) * s->K, s->in_dtype, 16, &kr);
  if (rc != M2RNN_OK) return rc;
  if (s->Nk == 0 && (k != nullptr || wk != nullptr)) return M2RNN_ERR_INVALID_ARG;
  if (s->R > 0 && (cs == nullptr || sn == nullptr || s->P < 1)) return M2RNN_ERR_INVALID_ARG;
  if (s->R > 0 && pos == nullptr && s->T > s->P) return M2RNN_ERR_INVALID_ARG;
  int dev, *status;
  rc = host_device_info(&dev, &status, sms);
  if (rc != M2RNN_OK) return rc;
  const void* opt[] = {wq, wk, cs, sn};
  if ((rc = allow(opt, dev)) != M2RNN_OK) return rc;
  if (s->T > 0) {
    const void* req[] = {q};
    if ((rc = require(req, dev)) != M2RNN_OK) return rc;
    if ((rc = host_check_ptr(k, dev, s->Nk > 0)) != M2RNN_OK) return rc;
    if ((rc = host_check_ptr(pos, dev, false)) != M2RNN_OK) return rc;
  }
  *p = m2rnn::QkParams{};
  p->q = q;
  p->k = k;
  p->wq = wq;
  p->wk = wk;
  p->cs = cs;
  p->sn = sn;
  p->pos = pos;
  p->qb = qr.batch;
  p->qt = qr.token;
  p->kb = kr.batch;
  p->kt = kr.token;
  p->tokens = static_cast<long long>(s->B) * s->T;
  p->T = s->T;
  p->Nq = s->Nq;
  p->Nk = s->Nk;
  p->K = s->K;
  p->R = s->R;
  p->P = s->P;
  p->interleaved = s->interleaved;
  p->split = m2rnn::qk_split(s);
  p->eps = eps;
  p->status = status;
  return M2RNN_OK;
}

// ---- selective scan -------------------------------------------------------------

struct ScanPlan {
  int nc, hpg, nhb, nseg, cps;
  size_t gate, dec, states, ends;  // bytes, for B sequences (sized_for)
  size_t saved() const { return gate + one_way(); }
  size_t one_way() const { return dec + states + ends; }
};

// Segments of the state kernel: a sequence's chunks form a chain, so it is cut
// where there are fewer (sequence, head block) pairs than 608 CTAs (the four that
// are resident on each of 152 SMs), into runs of two chunks at least.  With 912 the
// kernel took 115 us instead of 99 and the join 9.5 instead of 7.7 (B=1 T=65536 N=64).
ScanPlan sized_for(ScanPlan q, const m2rnn_shape* s, int B);
ScanPlan scan_plan(const m2rnn_shape* s) {
  ScanPlan q;
  const int Nq = s->Nq == 0 ? 1 : s->Nq;
  q.nc = (s->T + m2rnn::kChunk - 1) / m2rnn::kChunk;
  q.hpg = s->N / Nq;
  q.nhb = (q.hpg * s->V + m2rnn::kCols - 1) / m2rnn::kCols;
  const long long pairs = static_cast<long long>(s->B) * Nq * q.nhb;
  long long seg = 608 / pairs;
  if (seg > q.nc / 2) seg = q.nc / 2;
  if (seg < 1) seg = 1;
  q.cps = static_cast<int>((q.nc + seg - 1) / seg);
  if (q.cps < 1) q.cps = 1;
  q.nseg = (q.nc + q.cps - 1) / q.cps;
  return sized_for(q, s, s->B);
}

// The plan's buffers for `B` of the sequences.
ScanPlan sized_for(ScanPlan q, const m2rnn_shape* s, int B) {
  const size_t tile = static_cast<size_t>(m2rnn::kCols) * s->K * sizeof(float);
  const size_t heads = static_cast<size_t>(B) * s->N;
  const size_t pairs = static_cast<size_t>(B) * (s->Nq == 0 ? 1 : s->Nq) * q.nhb;
  q.gate = align256(heads * q.nc * m2rnn::kGate * sizeof(float));
  q.dec = align256(heads * (q.nc + q.nseg) * sizeof(float));
  q.states = align256(pairs * q.nc * tile);
  q.ends = q.nseg > 1 ? align256(pairs * q.nseg * tile) : 0;
  return q;
}

// CTAs that share a chunk's head blocks.  Outputs: about 1,216 (twice what is
// resident), so that they even out over the SMs; a CTA's own cost, its q and k tiles
// and their product, is about 0.4 of a head block.  B=8 T=2048 N=32 (256 chunks, 8
// head blocks): the call takes 64 us, with one CTA per chunk 100, with 3,648 67.
int scan_out_split(const m2rnn_shape* s, const ScanPlan& q) {
  const long long chunks = static_cast<long long>(s->B) * (s->Nq == 0 ? 1 : s->Nq) * q.nc;
  long long want = (1216 + chunks - 1) / chunks;
  if (want > q.nhb) want = q.nhb;
  const int per = static_cast<int>((q.nhb + want - 1) / want);
  return (q.nhb + per - 1) / per;
}
// Gradients: more than one costs shares of dq and dk in fp32, so only as many as
// it takes to give each SM its two resident CTAs.  A training step at B=1 T=8192
// N=32 (128 chunks) takes 134 us so, 139 with 608 CTAs (and, when it took 139, 181
// with one CTA per chunk).
int scan_bwd_split(const m2rnn_shape* s, const ScanPlan& q) {
  const long long chunks = static_cast<long long>(s->B) * (s->Nq == 0 ? 1 : s->Nq) * q.nc;
  long long want = 304 / chunks;
  if (want > q.nhb) want = q.nhb;
  if (want < 1) want = 1;
  const int per = static_cast<int>((q.nhb + want - 1) / want);
  return (q.nhb + per - 1) / per;
}

// Workspace of the backward pass: fp32 shares of dq, dk where several CTAs add
// to them, and the chunks' shares of the parameters' gradients.
size_t scan_share_bytes(const m2rnn_shape* s, const ScanPlan& q) {
  const int split = scan_bwd_split(s, q);
  if (split == 1) return 0;
  return align256(static_cast<size_t>(split) * 2 * s->B * s->T * (s->Nq == 0 ? 1 : s->Nq) * s->K *
                  sizeof(float));
}
size_t scan_part_bytes(const m2rnn_shape* s, const ScanPlan& q) {
  return align256(static_cast<size_t>(s->B) * q.nc * s->N * (2 + s->V) * sizeof(float));
}

int check_scan(const m2rnn_shape* s) {
  const int rc = m2rnn::validate_shape(s);
  if (rc != M2RNN_OK) return rc;
  if (s->T > (1 << 30) || s->N > (1 << 20)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
  const ScanPlan q = scan_plan(s);
  const double ctas = static_cast<double>(s->B) * q.nhb * (s->Nq == 0 ? 1 : s->Nq) * q.nc;
  return ctas < 1073741824.0 ? M2RNN_OK : M2RNN_ERR_UNSUPPORTED_SHAPE;  // 2^30
}

// The arguments that both directions share, with rows and plan.
int scan_common(const m2rnn_shape* s, const m2rnn_scan_rows* rows, const void* q, const void* k,
                const void* v, const void* a, const void* alpha, const void* beta,
                const void* w_r, const float* H0, m2rnn::ScanParams* p, ScanPlan* plan, int* dev) {
  int rc = check_scan(s);
  if (rc != M2RNN_OK) return rc;
  const int Nq = s->Nq == 0 ? 1 : s->Nq;
  const long long qw = static_cast<long long>(Nq) * s->K, vw = static_cast<long long>(s->N) * s->V;
  const long long e = static_cast<long long>(esize(s->in_dtype));
  m2rnn_rows qr, kr, vr, ar;
  if ((rc = read_rows(rows ? &rows->q : nullptr, s->T, qw, s->in_dtype, 16, &qr)) != M2RNN_OK ||
      (rc = read_rows(rows ? &rows->k : nullptr, s->T, qw, s->in_dtype, 16, &kr)) != M2RNN_OK ||
      (rc = read_rows(rows ? &rows->v : nullptr, s->T, vw, s->in_dtype, 16, &vr)) != M2RNN_OK ||
      (rc = read_rows(rows ? &rows->a : nullptr, s->T, s->N, s->in_dtype, e, &ar)) != M2RNN_OK)
    return rc;
  int sms, *status;
  if ((rc = host_device_info(dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* req[] = {alpha, beta};
  const void* opt[] = {w_r, H0};
  if ((rc = require(req, *dev)) != M2RNN_OK || (rc = allow(opt, *dev)) != M2RNN_OK) return rc;
  if (s->T > 0) {
    const void* req2[] = {q, k, v};
    if ((rc = require(req2, *dev)) != M2RNN_OK) return rc;
    if ((rc = m2rnn::host_check_elem_ptr(a, *dev, static_cast<size_t>(e))) != M2RNN_OK) return rc;
  }
  *plan = scan_plan(s);
  *p = m2rnn::ScanParams{};
  p->q = q;
  p->k = k;
  p->v = v;
  p->a = a;
  p->alpha = alpha;
  p->beta = beta;
  p->w_r = w_r;
  p->H0 = H0;
  p->qb = qr.batch;
  p->qt = qr.token;
  p->kb = kr.batch;
  p->kt = kr.token;
  p->vb = vr.batch;
  p->vt = vr.token;
  p->ab = ar.batch;
  p->at = ar.token;
  p->B = s->B;
  p->T = s->T;
  p->N = s->N;
  p->Nq = Nq;
  p->K = s->K;
  p->V = s->V;
  p->nc = plan->nc;
  p->hpg = plan->hpg;
  p->nhb = plan->nhb;
  p->nseg = plan->nseg;
  p->cps = plan->cps;
  p->status = status;
  return M2RNN_OK;
}

// The parameters of `count` sequences from b0 on.
m2rnn::ScanParams items_from(m2rnn::ScanParams p, int b0, int count, size_t e) {
  const auto in = [&](const void* x, long long elems) {
    return static_cast<const char*>(x) + b0 * elems * static_cast<long long>(e);
  };
  const long long state = static_cast<long long>(b0) * p.N * p.K * p.V;
  p.q = in(p.q, p.qb);
  p.k = in(p.k, p.kb);
  p.v = in(p.v, p.vb);
  p.a = in(p.a, p.ab);
  p.y = const_cast<char*>(in(p.y, static_cast<long long>(p.T) * p.N * p.V));
  if (p.H0 != nullptr) p.H0 += state;
  if (p.HT != nullptr) p.HT += state;
  p.B = count;
  return p;
}

// Hands out pieces of the workspace.
struct Carve {
  char* at;
  float* take(size_t bytes) {
    float* r = bytes ? reinterpret_cast<float*>(at) : nullptr;
    at += bytes;
    return r;
  }
};

int scan_fwd_part(m2rnn::ScanParams p, const m2rnn_shape* s, const ScanPlan& plan, void* buffer,
                  bool f32, cudaStream_t st) {
  Carve keep{static_cast<char*>(buffer)};
  p.gate = keep.take(plan.gate);
  p.cdec = keep.take(plan.dec);
  p.Hl = keep.take(plan.states);
  p.Hseg = keep.take(plan.ends);
  p.hsplit = scan_out_split(s, plan);
  if (m2rnn::launch_scan_states(p, f32, false, st) != cudaSuccess) return M2RNN_ERR_CUDA;
  return status_from_cuda(m2rnn::launch_scan_out(p, f32, st));
}

}  // namespace

extern "C" {

int m2rnn_conv_fwd(const m2rnn_conv_shape* s, const void* x, const m2rnn_rows* x_rows,
                   const void* w, const void* bias, const void* state, void* y, void* state_out,
                   void* stream) {
  int rc = check_conv(s, false);
  if (rc != M2RNN_OK) return rc;
  m2rnn_rows xr;
  if ((rc = read_rows(x_rows, s->T, s->C, s->in_dtype, 16, &xr)) != M2RNN_OK) return rc;
  if (conv_outputs_overlap(s, xr, x, nullptr, 0, state, nullptr, y, state_out)) return M2RNN_ERR_INVALID_ARG;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* req[] = {w};
  const void* opt[] = {bias, state, state_out};
  if ((rc = require(req, dev)) != M2RNN_OK || (rc = allow(opt, dev)) != M2RNN_OK) return rc;
  const size_t sb = conv_state_bytes(s);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->T == 0) {
    if (state_out == nullptr) return M2RNN_OK;
    return status_from_cuda(state ? cudaMemcpyAsync(state_out, state, sb, cudaMemcpyDeviceToDevice, st)
                                  : cudaMemsetAsync(state_out, 0, sb, st));
  }
  const void* req2[] = {x, y};
  if ((rc = require(req2, dev)) != M2RNN_OK) return rc;
  m2rnn::ConvParams p = conv_params(s, xr, x, w, bias, state, status);
  p.y = y;
  p.state_out = state_out;
  p.TT = m2rnn::conv_fwd_tokens(s, sms);
  p.nT = (s->T + p.TT - 1) / p.TT;
  return status_from_cuda(m2rnn::launch_conv_fwd(p, s->in_dtype == M2RNN_F32, s->silu != 0, st));
}

size_t m2rnn_conv_bwd_workspace_size(const m2rnn_conv_shape* s) {
  if (check_conv(s, true) != M2RNN_OK || s->T == 0) return 0;
  int TT, nT, nparts;
  m2rnn::conv_bwd_plan(s, &TT, &nT, &nparts);
  return align256(static_cast<size_t>(nparts) * s->C * (s->W + 1) * sizeof(float));
}

int m2rnn_conv_bwd(const m2rnn_conv_shape* s, const void* x, const m2rnn_rows* x_rows,
                   const void* w, const void* bias, const void* state, const void* dy,
                   const void* dstate_out, void* dx, float* dw, float* dbias, void* dstate,
                   void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_conv(s, true);
  if (rc != M2RNN_OK) return rc;
  m2rnn_rows xr;
  if ((rc = read_rows(x_rows, s->T, s->C, s->in_dtype, 16, &xr)) != M2RNN_OK) return rc;
  if (conv_outputs_overlap(s, xr, x, dy, esize(s->grad_dtype), state, dstate_out, dx, dstate))
    return M2RNN_ERR_INVALID_ARG;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* req[] = {w, dw};
  const void* opt[] = {bias, state, dstate_out, dbias, dstate};
  if ((rc = require(req, dev)) != M2RNN_OK || (rc = allow(opt, dev)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->T == 0) {  // no tokens: the state passes through
    if (cudaMemsetAsync(dw, 0, static_cast<size_t>(s->C) * s->W * sizeof(float), st) != cudaSuccess)
      return M2RNN_ERR_CUDA;
    if (dbias != nullptr && cudaMemsetAsync(dbias, 0, s->C * sizeof(float), st) != cudaSuccess)
      return M2RNN_ERR_CUDA;
    if (dstate == nullptr) return M2RNN_OK;
    const size_t sb = conv_state_bytes(s);
    return status_from_cuda(dstate_out
                                ? cudaMemcpyAsync(dstate, dstate_out, sb, cudaMemcpyDeviceToDevice, st)
                                : cudaMemsetAsync(dstate, 0, sb, st));
  }
  const void* req2[] = {x, dy, dx};
  if ((rc = require(req2, dev)) != M2RNN_OK) return rc;
  if (workspace == nullptr || ws_bytes < m2rnn_conv_bwd_workspace_size(s)) return M2RNN_ERR_WORKSPACE;
  const void* ws[] = {workspace};
  if ((rc = require(ws, dev)) != M2RNN_OK) return rc;
  m2rnn::ConvParams p = conv_params(s, xr, x, w, bias, state, status);
  p.dy = dy;
  p.dstate_out = dstate_out;
  p.dx = dx;
  p.dstate = dstate;
  p.dw = dw;
  p.dbias = dbias;
  p.part = static_cast<float*>(workspace);
  m2rnn::conv_bwd_plan(s, &p.TT, &p.nT, &p.nparts);
  return status_from_cuda(m2rnn::launch_conv_bwd(p, s->in_dtype == M2RNN_F32,
                                                 s->grad_dtype == M2RNN_F32, s->silu != 0, st));
}

int m2rnn_conv_step(const m2rnn_conv_shape* s, const void* x, const m2rnn_rows* x_rows,
                    const void* w, const void* bias, const void* state, void* y, void* state_out,
                    void* stream) {
  int rc = check_conv(s, false);
  if (rc != M2RNN_OK) return rc;
  if (s->T != 1) return M2RNN_ERR_INVALID_ARG;
  m2rnn_rows xr;
  if ((rc = read_rows(x_rows, 1, s->C, s->in_dtype, 16, &xr)) != M2RNN_OK) return rc;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* req[] = {x, w, state, y, state_out};
  const void* opt[] = {bias};
  if ((rc = require(req, dev)) != M2RNN_OK || (rc = allow(opt, dev)) != M2RNN_OK) return rc;
  if (state != state_out && overlap(state, state_out, conv_state_bytes(s)))
    return M2RNN_ERR_INVALID_ARG;
  m2rnn::ConvParams p = conv_params(s, xr, x, w, bias, state, status);
  p.y = y;
  p.state_out = state_out;
  return status_from_cuda(m2rnn::launch_conv_step(p, s->in_dtype == M2RNN_F32, s->silu != 0,
                                                  static_cast<cudaStream_t>(stream)));
}

int m2rnn_qk_norm_fwd(const m2rnn_qk_shape* s, const void* q, const m2rnn_rows* q_rows,
                      const void* k, const m2rnn_rows* k_rows, const void* wq, const void* wk,
                      float eps, const float* cos, const float* sin, const int* pos, void* qo,
                      void* ko, void* stream) {
  m2rnn::QkParams p;
  int sms;
  int rc = qk_common(s, q, q_rows, k, k_rows, wq, wk, eps, cos, sin, pos, false, &p, &sms);
  if (rc != M2RNN_OK || s->T == 0) return rc;
  int dev, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  if ((rc = host_check_ptr(qo, dev, true)) != M2RNN_OK) return rc;
  if ((rc = host_check_ptr(ko, dev, s->Nk > 0)) != M2RNN_OK) return rc;
  p.qo = qo;
  p.ko = ko;
  return status_from_cuda(m2rnn::launch_qk_fwd(p, s->in_dtype == M2RNN_F32,
                                               static_cast<cudaStream_t>(stream)));
}

size_t m2rnn_qk_norm_bwd_workspace_size(const m2rnn_qk_shape* s) {
  if (check_qk(s, true) != M2RNN_OK || s->T == 0) return 0;
  return align256(static_cast<size_t>(m2rnn::qk_bwd_parts(s)) * 2 * s->K * sizeof(float));
}

int m2rnn_qk_norm_bwd(const m2rnn_qk_shape* s, const void* q, const m2rnn_rows* q_rows,
                      const void* k, const m2rnn_rows* k_rows, const void* wq, const void* wk,
                      float eps, const float* cos, const float* sin, const int* pos,
                      const void* dqo, const void* dko, void* dq, void* dk, float* dwq,
                      float* dwk, void* workspace, size_t ws_bytes, void* stream) {
  m2rnn::QkParams p;
  int sms;
  int rc = qk_common(s, q, q_rows, k, k_rows, wq, wk, eps, cos, sin, pos, true, &p, &sms);
  if (rc != M2RNN_OK) return rc;
  int dev, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* opt[] = {dwq, dwk};
  if ((rc = allow(opt, dev)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->T == 0) {
    for (float* d : {dwq, dwk})
      if (d != nullptr && cudaMemsetAsync(d, 0, s->K * sizeof(float), st) != cudaSuccess)
        return M2RNN_ERR_CUDA;
    return M2RNN_OK;
  }
  const void* req[] = {dqo, dq};
  if ((rc = require(req, dev)) != M2RNN_OK) return rc;
  for (const void* x : {dko, static_cast<const void*>(dk)})
    if ((rc = host_check_ptr(x, dev, s->Nk > 0)) != M2RNN_OK) return rc;
  if (workspace == nullptr || ws_bytes < m2rnn_qk_norm_bwd_workspace_size(s))
    return M2RNN_ERR_WORKSPACE;
  if ((rc = host_check_ptr(workspace, dev, true)) != M2RNN_OK) return rc;
  p.dqo = dqo;
  p.dko = dko;
  p.dq = dq;
  p.dk = dk;
  p.dwq = dwq;
  p.dwk = dwk;
  p.part = static_cast<float*>(workspace);
  p.nparts = m2rnn::qk_bwd_parts(s);
  return status_from_cuda(m2rnn::launch_qk_bwd(p, s->in_dtype == M2RNN_F32,
                                               s->grad_dtype == M2RNN_F32, st));
}

size_t m2rnn_scan_saved_size(const m2rnn_shape* s) {
  if (check_scan(s) != M2RNN_OK || s->T == 0) return 0;
  const ScanPlan q = scan_plan(s);
  return q.saved();
}

size_t m2rnn_scan_fwd_workspace_size(const m2rnn_shape* s, int saved_given) {
  if (check_scan(s) != M2RNN_OK || s->T == 0) return 0;
  const ScanPlan q = scan_plan(s);
  if (saved_given) return 0;
  // with the states of half of the sequences the call runs in two parts
  return s->in_dtype == M2RNN_F32 ? q.saved() : q.saved() - sized_for(q, s, s->B / 2).states;
}

int m2rnn_scan_fwd(const m2rnn_shape* s, const m2rnn_scan_rows* rows, const void* q,
                   const void* k, const void* v, const void* a, const void* alpha,
                   const void* beta, const void* w_r, const float* H0, void* y, float* H_T,
                   void* saved, void* workspace, size_t ws_bytes, void* stream) {
  m2rnn::ScanParams p;
  ScanPlan plan;
  int dev;
  int rc = scan_common(s, rows, q, k, v, a, alpha, beta, w_r, H0, &p, &plan, &dev);
  if (rc != M2RNN_OK) return rc;
  const void* opt[] = {H_T, saved};
  if ((rc = allow(opt, dev)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->T == 0) {
    if (H_T == nullptr) return M2RNN_OK;
    const size_t bytes = static_cast<size_t>(s->B) * s->N * s->K * s->V * sizeof(float);
    return status_from_cuda(H0 ? cudaMemcpyAsync(H_T, H0, bytes, cudaMemcpyDeviceToDevice, st)
                               : cudaMemsetAsync(H_T, 0, bytes, st));
  }
  if ((rc = host_check_ptr(y, dev, true)) != M2RNN_OK) return rc;
  const size_t need = m2rnn_scan_fwd_workspace_size(s, saved != nullptr);
  if (need > 0) {
    if (workspace == nullptr || ws_bytes < need) return M2RNN_ERR_WORKSPACE;
    if ((rc = host_check_ptr(workspace, dev, true)) != M2RNN_OK) return rc;
  }
  p.y = y;
  p.HT = H_T;
  const bool f32 = s->in_dtype == M2RNN_F32;
  // All sequences at once, or in two parts where the workspace has the states of the
  // larger one only; the segments are the same, and so are the results' bits.
  const int most = saved != nullptr || ws_bytes >= plan.saved() ? s->B : s->B - s->B / 2;
  for (int b0 = 0; b0 < s->B; b0 += most) {
    m2rnn_shape part = *s;
    part.B = s->B - b0 < most ? s->B - b0 : most;
    const ScanPlan size = sized_for(plan, s, part.B);
    const m2rnn::ScanParams x = items_from(p, b0, part.B, esize(s->in_dtype));
    if ((rc = scan_fwd_part(x, &part, size, saved ? saved : workspace, f32, st)) != M2RNN_OK) return rc;
  }
  return M2RNN_OK;
}

size_t m2rnn_scan_bwd_workspace_size(const m2rnn_shape* s, int saved_given) {
  if (check_scan(s) != M2RNN_OK || s->T == 0) return 0;
  const ScanPlan q = scan_plan(s);
  return (saved_given ? 0 : q.saved()) + q.one_way() + scan_share_bytes(s, q) + scan_part_bytes(s, q);
}

int m2rnn_scan_bwd(const m2rnn_shape* s, const m2rnn_scan_rows* rows, const void* q,
                   const void* k, const void* v, const void* a, const void* alpha,
                   const void* beta, const void* w_r, const float* H0, const void* saved,
                   const void* dy, const float* dH_T, void* dq, void* dk, void* dv, void* da,
                   float* dalpha, float* dbeta, float* dw_r, float* dH0, void* workspace,
                   size_t ws_bytes, void* stream) {
  m2rnn::ScanParams p;
  ScanPlan plan;
  int dev;
  int rc = scan_common(s, rows, q, k, v, a, alpha, beta, w_r, H0, &p, &plan, &dev);
  if (rc != M2RNN_OK) return rc;
  if ((w_r == nullptr) != (dw_r == nullptr)) return M2RNN_ERR_INVALID_ARG;
  const void* req[] = {dalpha, dbeta};
  const void* opt[] = {saved, dH_T, dw_r, dH0};
  if ((rc = require(req, dev)) != M2RNN_OK || (rc = allow(opt, dev)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->T == 0) {  // no tokens: dH0 = dH_T
    const size_t n = s->N * sizeof(float);
    const size_t bytes = static_cast<size_t>(s->B) * s->N * s->K * s->V * sizeof(float);
    if (cudaMemsetAsync(dalpha, 0, n, st) != cudaSuccess ||
        cudaMemsetAsync(dbeta, 0, n, st) != cudaSuccess ||
        (dw_r != nullptr && cudaMemsetAsync(dw_r, 0, n * s->V, st) != cudaSuccess))
      return M2RNN_ERR_CUDA;
    if (dH0 == nullptr) return M2RNN_OK;
    return status_from_cuda(dH_T ? cudaMemcpyAsync(dH0, dH_T, bytes, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(dH0, 0, bytes, st));
  }
  const void* req2[] = {dy, dq, dk, dv, da};
  if ((rc = require(req2, dev)) != M2RNN_OK) return rc;
  if (workspace == nullptr || ws_bytes < m2rnn_scan_bwd_workspace_size(s, saved != nullptr))
    return M2RNN_ERR_WORKSPACE;
  if ((rc = host_check_ptr(workspace, dev, true)) != M2RNN_OK) return rc;
  Carve ws{static_cast<char*>(workspace)};
  Carve keep{static_cast<char*>(const_cast<void*>(saved))};  // read only
  Carve& fwd = saved ? keep : ws;
  p.gate = fwd.take(plan.gate);
  p.cdec = fwd.take(plan.dec);
  p.Hl = fwd.take(plan.states);
  p.Hseg = fwd.take(plan.ends);
  p.dy = dy;
  p.dHT = dH_T;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.da = da;
  p.dalpha = dalpha;
  p.dbeta = dbeta;
  p.dw_r = dw_r;
  p.dH0 = dH0;
  p.rdec = ws.take(plan.dec);
  p.Rl = ws.take(plan.states);
  p.Rseg = ws.take(plan.ends);
  p.dqk = ws.take(scan_share_bytes(s, plan));
  p.part = ws.take(scan_part_bytes(s, plan));
  p.hsplit = scan_bwd_split(s, plan);
  const bool f32 = s->in_dtype == M2RNN_F32;
  if (saved == nullptr && m2rnn::launch_scan_states(p, f32, false, st) != cudaSuccess)
    return M2RNN_ERR_CUDA;
  if (m2rnn::launch_scan_states(p, f32, true, st) != cudaSuccess) return M2RNN_ERR_CUDA;
  return status_from_cuda(m2rnn::launch_scan_bwd(p, f32, st));
}

int m2rnn_scan_step(const m2rnn_shape* s, const m2rnn_scan_rows* rows, const void* q,
                    const void* k, const void* v, const void* a, const void* alpha,
                    const void* beta, const void* w_r, const float* H_in, float* H_out, void* y,
                    void* stream) {
  int rc = m2rnn::validate_shape(s);
  if (rc != M2RNN_OK) return rc;
  if (s->T != 1) return M2RNN_ERR_INVALID_ARG;
  const int Nq = s->Nq == 0 ? 1 : s->Nq;
  m2rnn_rows qr, kr, vr, ar;
  const long long qw = static_cast<long long>(Nq) * s->K, vw = static_cast<long long>(s->N) * s->V;
  const long long e = static_cast<long long>(esize(s->in_dtype));
  if ((rc = read_rows(rows ? &rows->q : nullptr, 1, qw, s->in_dtype, 16, &qr)) != M2RNN_OK ||
      (rc = read_rows(rows ? &rows->k : nullptr, 1, qw, s->in_dtype, 16, &kr)) != M2RNN_OK ||
      (rc = read_rows(rows ? &rows->v : nullptr, 1, vw, s->in_dtype, 16, &vr)) != M2RNN_OK ||
      (rc = read_rows(rows ? &rows->a : nullptr, 1, s->N, s->in_dtype, e, &ar)) != M2RNN_OK)
    return rc;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* req[] = {q, k, v, alpha, beta, H_in, H_out, y};
  const void* opt[] = {w_r};
  if ((rc = require(req, dev)) != M2RNN_OK || (rc = allow(opt, dev)) != M2RNN_OK) return rc;
  if ((rc = m2rnn::host_check_elem_ptr(a, dev, static_cast<size_t>(e))) != M2RNN_OK) return rc;
  if (H_out != H_in &&
      overlap(H_in, H_out, static_cast<size_t>(s->B) * s->N * s->K * s->V * sizeof(float)))
    return M2RNN_ERR_INVALID_ARG;
  m2rnn::ScanStepParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.a = a;
  p.alpha = alpha;
  p.beta = beta;
  p.w_r = w_r;
  p.H_in = H_in;
  p.H_out = H_out;
  p.y = y;
  p.qb = qr.batch;
  p.kb = kr.batch;
  p.vb = vr.batch;
  p.ab = ar.batch;
  p.B = s->B;
  p.N = s->N;
  p.Nq = Nq;
  p.K = s->K;
  p.status = status;
  return status_from_cuda(m2rnn::launch_scan_step(p, s->V, s->in_dtype == M2RNN_F32,
                                                  static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

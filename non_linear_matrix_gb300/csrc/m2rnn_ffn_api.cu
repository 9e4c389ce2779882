// m2rnn_ffn_api.cu -- the extern "C" entry points declared in
// include/m2rnn_ffn.h: argument validation, tensor maps and launch planning of the
// residual and norm, the gated products and the 8-bit product.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "m2rnn_ffn.h"

namespace {

using m2rnn::host_check_ptr;
using m2rnn::host_device_info;

int status_from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return M2RNN_OK;
  cudaGetLastError();  // (not left for the next call to find)
  return M2RNN_ERR_CUDA;
}
bool is_dtype(int d) { return d == M2RNN_F32 || d == M2RNN_BF16; }
size_t esize(int dtype) { return dtype == M2RNN_F32 ? 4 : 2; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
constexpr double kMostElems = 1099511627776.0;  // 2^40

template <int N>
int check(const void* const (&ptrs)[N], int dev, bool required) {
  for (const void* p : ptrs) {
    const int rc = host_check_ptr(p, dev, required);
    if (rc != M2RNN_OK) return rc;
  }
  return M2RNN_OK;
}

// A row distance (in elements of e bytes) keeps rows on 16-byte boundaries and is below 2^40
// bytes (a tensor map's limit), and M rows stay below 2^40 elements.
int check_row(long long row, size_t e, long long M, long long least) {
  if (row < 0 || row < least) return M2RNN_ERR_INVALID_ARG;
  if ((row * static_cast<long long>(e)) % 16 != 0) return M2RNN_ERR_MISALIGNED;
  if (static_cast<double>(row) * (M > 0 ? M : 1) >= kMostElems || static_cast<double>(row) * e >= kMostElems)
    return M2RNN_ERR_UNSUPPORTED_SHAPE;
  return M2RNN_OK;
}

// ---- residual and norm ---------------------------------------------------------

int check_norm(const m2rnn_norm_shape* s, int most_d) {
  if (s == nullptr) return M2RNN_ERR_INVALID_ARG;
  if (s->B < 0 || s->T < 0 || s->D < 1 || !is_dtype(s->in_dtype)) return M2RNN_ERR_INVALID_ARG;
  const double rows = static_cast<double>(s->B) * s->T;
  if (s->D % 8 != 0 || s->D > most_d || rows >= 2147483648.0 || rows * s->D >= kMostElems)
    return M2RNN_ERR_UNSUPPORTED_SHAPE;
  return M2RNN_OK;
}
constexpr int kNormMostD = 16384, kMostD = 1 << 20, kMostSum = 1 << 16;
long long rows_of(const m2rnn_norm_shape* s) { return static_cast<long long>(s->B) * s->T; }

// Rows of x, whose distances keep every offset below 2^40 elements.
int norm_rows(const m2rnn_norm_shape* s, const m2rnn_rows* rows, m2rnn_rows* out) {
  const int rc = m2rnn::read_rows(rows, s->T, s->D, s->in_dtype, 16, out);
  if (rc != M2RNN_OK) return rc;
  const double span = static_cast<double>(out->batch) * s->B + static_cast<double>(out->token) * s->T;
  return span >= 2.0 * kMostElems ? M2RNN_ERR_UNSUPPORTED_SHAPE : M2RNN_OK;
}
bool contiguous(const m2rnn_norm_shape* s, const m2rnn_rows& r) {
  return (s->T <= 1 || r.token == s->D) && (s->B <= 1 || r.batch == static_cast<long long>(s->T) * s->D);
}
bool norm_overlap(const m2rnn_norm_shape* s, const void* x, const m2rnn_rows& r, const void* y, size_t bytes) {
  return s->B > 0 && m2rnn::rows_overlap(x, r, s->B, s->T, s->D, esize(s->in_dtype), y, bytes);
}

bool spans_overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  return a != nullptr && b != nullptr && a_bytes > 0 && b_bytes > 0 && m2rnn::overlap_spans(a, a_bytes, b, b_bytes);
}
// The same for M rows of the products' inputs.
bool row_overlap(const void* x, long long row, long long M, long long D, size_t e, const void* y, size_t bytes) {
  const m2rnn_rows r = {0, row};
  return M > 0 && m2rnn::rows_overlap(x, r, 1, M, D, e, y, bytes);
}

// Rows that are evenly spaced over all items need no division in the kernels.
void set_rows(const m2rnn_norm_shape* s, const m2rnn_rows& x, const m2rnn_rows* res, m2rnn::Norm2Params* p) {
  const auto even = [&](const m2rnn_rows& r) { return r.batch == r.token * s->T; };
  p->M = rows_of(s);
  p->T = s->B == 1 || (even(x) && (res == nullptr || even(*res))) ? static_cast<int>(p->M) : s->T;
  p->xb = x.batch;
  p->xt = x.token;
  if (res != nullptr) {
    p->rb = res->batch;
    p->rt = res->token;
  }
  if (s->T == 1 && s->B > 1) {  // items are the rows
    p->T = static_cast<int>(p->M);
    p->xt = x.batch;
    if (res != nullptr) p->rt = res->batch;
  }
  p->D = s->D;
}

int add_norm(const m2rnn_norm_shape* s, const void* x, const m2rnn_rows* x_rows, const void* res,
             const m2rnn_rows* res_rows, const void* w, float eps, void* r, void* y, void* q, float* scale, bool q8,
             void* stream) {
  int rc = check_norm(s, kNormMostD);
  if (rc != M2RNN_OK) return rc;
  if (!(eps >= 0.f)) return M2RNN_ERR_INVALID_ARG;  // also rejects NaN
  const size_t e = esize(s->in_dtype), M = static_cast<size_t>(rows_of(s));
  m2rnn_rows xr, rr;
  if ((rc = norm_rows(s, x_rows, &xr)) != M2RNN_OK || (rc = norm_rows(s, res_rows, &rr)) != M2RNN_OK) return rc;
  if ((res == nullptr) != (r == nullptr) && M > 0) return M2RNN_ERR_INVALID_ARG;
  // outputs apart from inputs and each other; r may be x or res itself
  const struct { const void* p; size_t bytes; } outs[] = {
      {r, M * s->D * e}, {y, M * s->D * e}, {q, M * s->D}, {scale, M * 4}};
  for (int i = 0; i < 4; ++i) {
    const bool here_x = i == 0 && r == x && contiguous(s, xr), here_res = i == 0 && r == res && contiguous(s, rr);
    if (!here_x && norm_overlap(s, x, xr, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
    if (!here_res && norm_overlap(s, res, rr, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
    if (spans_overlap(w, static_cast<size_t>(s->D) * e, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (spans_overlap(outs[j].p, outs[j].bytes, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
  }
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  if (M == 0) return M2RNN_OK;
  const void* opt[] = {res, w, r};
  if ((rc = check(opt, dev, false)) != M2RNN_OK) return rc;
  const void* req[] = {x, q8 ? q : y};
  if ((rc = check(req, dev, true)) != M2RNN_OK || (rc = host_check_ptr(scale, dev, q8)) != M2RNN_OK) return rc;
  m2rnn::Norm2Params p{};
  p.x = x;
  p.res = res;
  p.w = w;
  p.r = r;
  p.y = y;
  p.q = static_cast<uint8_t*>(q);
  p.scale = scale;
  set_rows(s, xr, res == nullptr ? nullptr : &rr, &p);
  p.eps = eps;
  p.status = status;
  return status_from_cuda(
      m2rnn::launch_add_norm(p, s->in_dtype == M2RNN_F32, sms, static_cast<cudaStream_t>(stream)));
}

// ---- products --------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, looked up once.
EncodeFn encoder() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load();
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    fn.store(f);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// [planes][outer][inner] elements of e bytes (1: e4m3, 2: bf16), rows `row` elements and
// planes `plane` elements apart, read in boxes of 128 bytes by `box` rows.
bool make_map(CUtensorMap* m, const void* base, size_t e, long long inner, long long outer, long long planes,
              long long row, long long plane, int box) {
  const EncodeFn f = encoder();
  if (f == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row) * e, static_cast<cuuint64_t>(plane) * e};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(128 / e), static_cast<cuuint32_t>(box), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  return f(m, e == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
           dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int act_of(const m2rnn_glu_shape* s) { return s->act & ~M2RNN_GLU_ROUND; }
int check_glu(const m2rnn_glu_shape* s, bool q8) {
  if (s == nullptr) return M2RNN_ERR_INVALID_ARG;
  if (s->M < 0 || s->D < 1 || s->F < 1 || !is_dtype(s->in_dtype)) return M2RNN_ERR_INVALID_ARG;
  if (act_of(s) != 0 && act_of(s) != 1) return M2RNN_ERR_INVALID_ARG;
  if (act_of(s) != s->act && s->in_dtype != M2RNN_BF16) return M2RNN_ERR_INVALID_ARG;
  if (q8 && s->in_dtype != M2RNN_BF16) return M2RNN_ERR_INVALID_ARG;
  if (s->D % (q8 ? 16 : 8) != 0 || s->F % 8 != 0 || s->D > kMostSum || s->F > kMostD || s->M >= (1LL << 31))
    return M2RNN_ERR_UNSUPPORTED_SHAPE;
  const double M = static_cast<double>(s->M);
  if (M * s->D >= kMostElems || M * s->F >= kMostElems || static_cast<double>(s->D) * s->F >= kMostElems / 4)
    return M2RNN_ERR_UNSUPPORTED_SHAPE;
  return M2RNN_OK;
}

// fp32: K tiles whose products one chain of sums takes, over all segments (256 k, 16 steps
// of the tensor core, each of which cuts its sum off: 3.1 2^-24 of it where all terms have one
// sign, measured).  Relative 2-norm, terms of both signs and of one: h 4.7e-7, 8.1e-7, gradients at most
// 5.6e-7, 7.9e-7; with 128 k 2.6e-7, 3.7e-7, for 5 to 14 % of the time (M=4096 D=2048, M=8192
// D=512).  The formula in plain fp32: 7e-7 to 9e-7.
constexpr int kChunkTiles = 4;

// Rows of what lies in the workspace start on 128 bytes: a copied row of 128 bytes then is one
// line of L2 (rows of 1,040 and 2,800 bytes took twice the time).
int pitch_of(int n) { return (n + 63) / 64 * 64; }

m2rnn::GemmParams gemm_params(const m2rnn::GemmPlan& q, long long M, int N, int nseg, int kt, bool f32, int* status) {
  m2rnn::GemmParams p{};
  p.M = M;
  p.N = N;
  p.kt = kt;
  p.kc = !f32 ? kt : nseg < kChunkTiles ? kChunkTiles / nseg : 1;
  p.nseg = nseg;
  p.aterms = 1;
  p.mt = q.mt;
  p.nt = q.nt;
  p.nbatch = q.nbatch;
  p.whole = q.whole;
  p.split = q.split;
  p.nparts = q.nparts;
  p.status = status;
  p.limit_ns = m2rnn::host_wait_limit_ns();
  p.inject_stall = m2rnn::host_fault_injection() == 1;
  return p;
}
int k_tiles(long long K, size_t e) { return static_cast<int>((K * static_cast<long long>(e) + 127) / 128); }

// Hands out pieces of the workspace.
struct Pieces {
  char* at;
  __nv_bfloat16* take(size_t elems) {
    __nv_bfloat16* r = reinterpret_cast<__nv_bfloat16*>(at);
    at += align256(elems * 2);
    return r;
  }
};
size_t terms_bytes(const m2rnn_glu_shape* s) {  // of x, wg and wu
  if (s->in_dtype != M2RNN_F32) return 0;
  const size_t pitch = pitch_of(s->D);
  return align256(6 * s->M * pitch) + 2 * align256(6 * s->F * pitch);
}
// bf16 terms that hold each gradient of g and u between the products: 3 with fp32 inputs, 2 with
// bf16 ones.  With 1 (the caller's choice) its rounding (2^-9 of each of many terms of a sum) adds as
// much error to dx, dwg and dwu as their own rounding does: relative 2-norm 2.35e-3 instead of
// 1.66e-3.  With 2 the products that take them are twice as long: backward pass 556 against 331 us at
// M=16384 D=1024 F=2816 (kernel of the gradients 139 against 111, dx 203 against 106, dwg and dwu
// 211 against 114).
int grad_terms(const m2rnn_glu_shape* s) {
  if (s->in_dtype == M2RNN_F32) return 3;
  return act_of(s) != s->act ? 1 : 2;
}
size_t dgu_bytes(const m2rnn_glu_shape* s) {  // the gradients of g and u
  return align256(static_cast<size_t>(s->M) * pitch_of(s->F) * (4 * grad_terms(s)));
}
// Segments of dx's products; of each weight's gradient half as many.
int dx_segments(const m2rnn_glu_shape* s) { return s->in_dtype == M2RNN_F32 ? 2 : 2 * grad_terms(s); }
m2rnn::GemmPlan pair_plan(const m2rnn_glu_shape* s, int epi) {
  return m2rnn::gemm_plan(epi, s->in_dtype == M2RNN_F32, s->M, s->F, 1, 1, k_tiles(s->D, 2));
}
m2rnn::GemmPlan dx_plan(const m2rnn_glu_shape* s) {
  return m2rnn::gemm_plan(m2rnn::EPI_STORE, s->in_dtype == M2RNN_F32, s->M, s->D, 1, dx_segments(s), k_tiles(s->F, 2));
}
m2rnn::GemmPlan dw_plan(const m2rnn_glu_shape* s) {
  return m2rnn::gemm_plan(m2rnn::EPI_STORE, s->in_dtype == M2RNN_F32, s->F, s->D, 2, dx_segments(s) / 2,
                          k_tiles(s->M, 2));
}

// What the products read: the caller's bf16 matrices, or their terms.
struct Operands {
  const void *x, *wg, *wu;
  long long x_row, w_row;
  int terms;
};
int make_operands(const m2rnn_glu_shape* s, const void* x, long long x_row, const void* wg, const void* wu,
                  Pieces* ws, int* status, cudaStream_t st, Operands* o) {
  if (s->in_dtype == M2RNN_BF16) {
    *o = {x, wg, wu, x_row, s->D, 1};
    return M2RNN_OK;
  }
  m2rnn::SplitParams q{};
  const void* src[3] = {x, wg, wu};
  for (int i = 0; i < 3; ++i) {
    q.src[i] = static_cast<const float*>(src[i]);
    q.row[i] = i == 0 ? x_row : s->D;
    q.M[i] = i == 0 ? s->M : s->F;
    q.dst[i] = ws->take(static_cast<size_t>(3 * q.M[i]) * pitch_of(s->D));
  }
  q.D = s->D;
  q.pitch = pitch_of(s->D);
  q.n = 3;
  q.status = status;
  *o = {q.dst[0], q.dst[1], q.dst[2], q.pitch, q.pitch, 3};
  return status_from_cuda(m2rnn::launch_split(q, st));
}

// g and u of every token (EPI_GLU: h; EPI_DGLU: their gradients).
int run_pair(const m2rnn_glu_shape* s, const Operands& o, int epi, const void* dh, void* out, float* parts,
             int* status, int sms, cudaStream_t st) {
  const bool f32 = o.terms == 3;
  const m2rnn::GemmPlan q = pair_plan(s, epi);
  m2rnn::GemmParams p = gemm_params(q, s->M, s->F, 1, k_tiles(s->D, 2), f32, status);
  p.parts = parts;
  const long long x_plane = s->M * o.x_row, w_plane = s->F * o.w_row;
  if (!make_map(&p.a, o.x, 2, s->D, s->M, o.terms, o.x_row, f32 ? x_plane : o.x_row, 128) ||
      !make_map(&p.b0, o.wg, 2, s->D, s->F, o.terms, o.w_row, f32 ? w_plane : o.w_row, q.bn / 2) ||
      !make_map(&p.b1, o.wu, 2, s->D, s->F, o.terms, o.w_row, f32 ? w_plane : o.w_row, q.bn / 2))
    return M2RNN_ERR_CUDA;
  p.out[0] = out;
  p.pitch = epi == m2rnn::EPI_DGLU ? pitch_of(s->F) : s->F;
  p.aterms = grad_terms(s);
  p.in = dh;
  p.act = act_of(s);
  return status_from_cuda(m2rnn::launch_gemm(p, {epi, f32, false, q.bn, q.rows}, sms, st));
}

}  // namespace

extern "C" {

int m2rnn_add_norm_fwd(const m2rnn_norm_shape* s, const void* x, const m2rnn_rows* x_rows, const void* res,
                       const m2rnn_rows* res_rows, const void* w, float eps, void* r, void* y, void* stream) {
  return add_norm(s, x, x_rows, res, res_rows, w, eps, r, y, nullptr, nullptr, false, stream);
}

int m2rnn_add_norm_q8(const m2rnn_norm_shape* s, const void* x, const m2rnn_rows* x_rows, const void* res,
                      const m2rnn_rows* res_rows, const void* w, float eps, void* r, void* q, float* scale,
                      void* stream) {
  return add_norm(s, x, x_rows, res, res_rows, w, eps, r, nullptr, q, scale, true, stream);
}

size_t m2rnn_add_norm_bwd_workspace_size(const m2rnn_norm_shape* s) {
  if (check_norm(s, kNormMostD) != M2RNN_OK || rows_of(s) == 0) return 0;
  return align256(static_cast<size_t>(m2rnn::add_norm_bwd_parts(s)) * s->D * sizeof(float));
}

int m2rnn_add_norm_bwd(const m2rnn_norm_shape* s, const void* r, const m2rnn_rows* r_rows, const void* w, float eps,
                       const void* dy, const void* dr, void* dx, float* dw, void* workspace, size_t ws_bytes,
                       void* stream) {
  int rc = check_norm(s, kNormMostD);
  if (rc != M2RNN_OK) return rc;
  if (!(eps >= 0.f)) return M2RNN_ERR_INVALID_ARG;
  m2rnn_rows rr;
  if ((rc = norm_rows(s, r_rows, &rr)) != M2RNN_OK) return rc;
  const size_t e = esize(s->in_dtype), M = static_cast<size_t>(rows_of(s));
  const size_t n = M * s->D * e, db = static_cast<size_t>(s->D) * 4, wb = static_cast<size_t>(s->D) * e;
  if (norm_overlap(s, r, rr, dx, n) || spans_overlap(w, wb, dx, n) || (dx != dy && spans_overlap(dy, n, dx, n)) ||
      (dx != dr && spans_overlap(dr, n, dx, n)) || spans_overlap(dw, db, dx, n) || norm_overlap(s, r, rr, dw, db) ||
      spans_overlap(dw, db, dy, n) || spans_overlap(dw, db, dr, n) || spans_overlap(dw, db, w, wb))
    return M2RNN_ERR_INVALID_ARG;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* opt[] = {w, dr, dw};
  if ((rc = check(opt, dev, false)) != M2RNN_OK) return rc;
  if (M == 0) return dw == nullptr ? M2RNN_OK : status_from_cuda(cudaMemsetAsync(dw, 0, db, st));
  const void* req[] = {r, dy, dx};
  if ((rc = check(req, dev, true)) != M2RNN_OK) return rc;
  if (dw != nullptr) {
    if (workspace == nullptr || ws_bytes < m2rnn_add_norm_bwd_workspace_size(s)) return M2RNN_ERR_WORKSPACE;
    if ((rc = host_check_ptr(workspace, dev, true)) != M2RNN_OK) return rc;
  }
  m2rnn::Norm2Params p{};
  p.x = r;
  set_rows(s, rr, nullptr, &p);
  p.w = w;
  p.dy = dy;
  p.dr = dr;
  p.dx = dx;
  p.dw = dw;
  p.part = dw == nullptr ? nullptr : static_cast<float*>(workspace);
  p.nparts = m2rnn::add_norm_bwd_parts(s);
  p.eps = eps;
  p.status = status;
  return status_from_cuda(m2rnn::launch_add_norm_bwd(p, s->in_dtype == M2RNN_F32, st));
}

int m2rnn_quant_rows(const m2rnn_norm_shape* s, const void* x, const m2rnn_rows* x_rows, void* q, float* scale,
                     void* stream) {
  int rc = check_norm(s, kMostD);
  if (rc != M2RNN_OK) return rc;
  m2rnn_rows xr;
  if ((rc = norm_rows(s, x_rows, &xr)) != M2RNN_OK) return rc;
  const size_t M = static_cast<size_t>(rows_of(s)), qb = M * s->D, sb = M * 4;
  if (norm_overlap(s, x, xr, q, qb) || norm_overlap(s, x, xr, scale, sb) || spans_overlap(q, qb, scale, sb))
    return M2RNN_ERR_INVALID_ARG;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  if (M == 0) return M2RNN_OK;
  const void* req[] = {x, q, scale};
  if ((rc = check(req, dev, true)) != M2RNN_OK) return rc;
  m2rnn::Norm2Params p{};
  p.x = x;
  set_rows(s, xr, nullptr, &p);
  p.q = static_cast<uint8_t*>(q);
  p.scale = scale;
  p.status = status;
  return status_from_cuda(
      m2rnn::launch_quant_rows(p, s->in_dtype == M2RNN_F32, static_cast<cudaStream_t>(stream)));
}

size_t m2rnn_glu_fwd_workspace_size(const m2rnn_glu_shape* s) {
  if (check_glu(s, false) != M2RNN_OK || s->M <= m2rnn::few_most(s->in_dtype == M2RNN_F32)) return 0;
  return terms_bytes(s) + align256(pair_plan(s, m2rnn::EPI_GLU).parts_bytes);
}

int m2rnn_glu_fwd(const m2rnn_glu_shape* s, const void* x, long long x_row, const void* wg, const void* wu, void* h,
                  void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_glu(s, false);
  if (rc != M2RNN_OK) return rc;
  const size_t e = esize(s->in_dtype);
  if ((rc = check_row(x_row, e, s->M, s->D)) != M2RNN_OK) return rc;
  const size_t hb = static_cast<size_t>(s->M) * s->F * e, wb = static_cast<size_t>(s->F) * s->D * e;
  if (row_overlap(x, x_row, s->M, s->D, e, h, hb) || spans_overlap(wg, wb, h, hb) ||
      spans_overlap(wu, wb, h, hb))
    return M2RNN_ERR_INVALID_ARG;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  if (s->M == 0) return M2RNN_OK;
  const void* req[] = {x, wg, wu, h};
  if ((rc = check(req, dev, true)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->M <= m2rnn::few_most(s->in_dtype == M2RNN_F32)) {
    m2rnn::FewParams p{};
    p.x = x;
    p.x_row = x_row;
    p.w0 = wg;
    p.w1 = wu;
    p.out = h;
    p.M = static_cast<int>(s->M);
    p.D = s->D;
    p.F = s->F;
    p.act = act_of(s);
    p.status = status;
    return status_from_cuda(m2rnn::launch_few(p, m2rnn::EPI_GLU, false, s->in_dtype == M2RNN_F32, st));
  }
  const size_t need = m2rnn_glu_fwd_workspace_size(s);
  if (need > 0) {
    if (workspace == nullptr || ws_bytes < need) return M2RNN_ERR_WORKSPACE;
    if ((rc = host_check_ptr(workspace, dev, true)) != M2RNN_OK) return rc;
  }
  Pieces ws{static_cast<char*>(workspace)};
  Operands o;
  if ((rc = make_operands(s, x, x_row, wg, wu, &ws, status, st, &o)) != M2RNN_OK) return rc;
  return run_pair(s, o, m2rnn::EPI_GLU, nullptr, h, reinterpret_cast<float*>(ws.at), status, sms, st);
}

size_t m2rnn_glu_bwd_workspace_size(const m2rnn_glu_shape* s) {
  if (check_glu(s, false) != M2RNN_OK || s->M == 0) return 0;
  size_t parts = pair_plan(s, m2rnn::EPI_DGLU).parts_bytes;  // (one after the other in the same place)
  for (size_t more : {dx_plan(s).parts_bytes, dw_plan(s).parts_bytes}) parts = more > parts ? more : parts;
  return terms_bytes(s) + dgu_bytes(s) + align256(parts);
}

int m2rnn_glu_bwd(const m2rnn_glu_shape* s, const void* x, long long x_row, const void* wg, const void* wu,
                  const void* dh, void* dx, void* dwg, void* dwu, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_glu(s, false);
  if (rc != M2RNN_OK) return rc;
  const size_t e = esize(s->in_dtype);
  if ((rc = check_row(x_row, e, s->M, s->D)) != M2RNN_OK) return rc;
  if ((dwg == nullptr) != (dwu == nullptr)) return M2RNN_ERR_INVALID_ARG;
  const size_t xb = static_cast<size_t>(s->M) * s->D * e, wb = static_cast<size_t>(s->F) * s->D * e;
  const size_t hb = static_cast<size_t>(s->M) * s->F * e;
  const struct { const void* p; size_t bytes; } outs[] = {{dx, xb}, {dwg, wb}, {dwu, wb}},
                                                ins[] = {{wg, wb}, {wu, wb}, {dh, hb}};
  for (int i = 0; i < 3; ++i) {
    if (row_overlap(x, x_row, s->M, s->D, e, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
    for (const auto& in : ins)
      if (spans_overlap(in.p, in.bytes, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (spans_overlap(outs[j].p, outs[j].bytes, outs[i].p, outs[i].bytes)) return M2RNN_ERR_INVALID_ARG;
  }
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  const void* opt[] = {dx, dwg, dwu};
  if ((rc = check(opt, dev, false)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dx == nullptr && dwg == nullptr) return M2RNN_OK;
  if (s->M == 0) {
    if (dwg == nullptr) return M2RNN_OK;
    const cudaError_t a = cudaMemsetAsync(dwg, 0, wb, st);
    return status_from_cuda(a != cudaSuccess ? a : cudaMemsetAsync(dwu, 0, wb, st));
  }
  const void* req[] = {x, wg, wu, dh};
  if ((rc = check(req, dev, true)) != M2RNN_OK) return rc;
  if (workspace == nullptr || ws_bytes < m2rnn_glu_bwd_workspace_size(s)) return M2RNN_ERR_WORKSPACE;
  if ((rc = host_check_ptr(workspace, dev, true)) != M2RNN_OK) return rc;
  Pieces ws{static_cast<char*>(workspace)};
  Operands o;
  if ((rc = make_operands(s, x, x_row, wg, wu, &ws, status, st, &o)) != M2RNN_OK) return rc;
  const bool f32 = o.terms == 3;
  const int hrow = pitch_of(s->F), gt = grad_terms(s), segs = dx_segments(s);
  const long long hp = s->M * hrow;
  __nv_bfloat16* dgu = ws.take(static_cast<size_t>(2 * gt) * hp);
  float* parts = reinterpret_cast<float*>(ws.at);
  if ((rc = run_pair(s, o, m2rnn::EPI_DGLU, dh, dgu, parts, status, sms, st)) != M2RNN_OK) return rc;
  const long long xp = s->M * o.x_row, wp = s->F * o.w_row;
  if (dx != nullptr) {  // dg wg + du wu
    const m2rnn::GemmPlan q = dx_plan(s);
    m2rnn::GemmParams p = gemm_params(q, s->M, s->D, segs, k_tiles(s->F, 2), f32, status);
    p.aterms = gt;
    if (!make_map(&p.a, dgu, 2, s->F, s->M, 2 * gt, hrow, hp, 128) ||
        !make_map(&p.b0, o.wg, 2, s->D, s->F, o.terms, o.w_row, f32 ? wp : o.w_row, 64) ||
        !make_map(&p.b1, o.wu, 2, s->D, s->F, o.terms, o.w_row, f32 ? wp : o.w_row, 64))
      return M2RNN_ERR_CUDA;
    p.out[0] = dx;
    p.parts = parts;
    rc = status_from_cuda(m2rnn::launch_gemm(p, {m2rnn::EPI_STORE, f32, false, q.bn, q.rows}, sms, st));
    if (rc != M2RNN_OK) return rc;
  }
  if (dwg != nullptr) {  // dg^T x and du^T x, which share x
    const m2rnn::GemmPlan q = dw_plan(s);
    m2rnn::GemmParams p = gemm_params(q, s->F, s->D, segs / 2, k_tiles(s->M, 2), f32, status);
    p.aterms = gt;
    if (!make_map(&p.a, dgu, 2, s->F, s->M, 2 * gt, hrow, hp, 64) ||
        !make_map(&p.b0, o.x, 2, s->D, s->M, o.terms, o.x_row, f32 ? xp : o.x_row, 64))
      return M2RNN_ERR_CUDA;
    p.b1 = p.b0;
    p.out[0] = dwg;
    p.out[1] = dwu;
    p.parts = parts;
    return status_from_cuda(m2rnn::launch_gemm(p, {m2rnn::EPI_STORE, f32, true, q.bn, q.rows}, sms, st));
  }
  return M2RNN_OK;
}

}  // extern "C"

namespace {

// Both 8-bit products: the arguments, then few tokens or tiles.
int product_q8(const m2rnn_glu_shape* s, const void* x, long long x_row, const float* xs, const void* w0,
               const float* s0, const void* w1, const float* s1, const void* res, long long res_row, void* out,
               bool pair, void* stream) {
  int rc = check_glu(s, true);
  if (rc != M2RNN_OK) return rc;
  if ((rc = check_row(x_row, 1, s->M, s->D)) != M2RNN_OK) return rc;
  if (res != nullptr && (rc = check_row(res_row, 2, s->M, 0)) != M2RNN_OK) return rc;
  const size_t ob = static_cast<size_t>(s->M) * s->F * 2, wb = static_cast<size_t>(s->F) * s->D;
  const size_t fb = static_cast<size_t>(s->F) * 4;
  const bool in_place = res == out && res_row == s->F;
  if (row_overlap(x, x_row, s->M, s->D, 1, out, ob) || spans_overlap(w0, wb, out, ob) ||
      spans_overlap(w1, wb, out, ob) || spans_overlap(xs, static_cast<size_t>(s->M) * 4, out, ob) ||
      spans_overlap(s0, fb, out, ob) || spans_overlap(s1, fb, out, ob) ||
      (!in_place && row_overlap(res, res_row, s->M, s->F, 2, out, ob)))
    return M2RNN_ERR_INVALID_ARG;
  int dev, sms, *status;
  if ((rc = host_device_info(&dev, &status, &sms)) != M2RNN_OK) return rc;
  if (s->M == 0) return M2RNN_OK;
  const void* req[] = {x, xs, w0, s0, out};
  if ((rc = check(req, dev, true)) != M2RNN_OK) return rc;
  const void* more[] = {w1, s1};
  if ((rc = check(more, dev, pair)) != M2RNN_OK) return rc;
  if ((rc = host_check_ptr(res, dev, false)) != M2RNN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int epi = pair ? m2rnn::EPI_GLU8 : m2rnn::EPI_LIN8;
  if (s->M <= m2rnn::few_most(false)) {
    m2rnn::FewParams p{};
    p.x = x;
    p.x_row = x_row;
    p.w0 = w0;
    p.w1 = w1;
    p.res = res;
    p.res_row = res_row;
    p.sa = xs;
    p.sb0 = s0;
    p.sb1 = s1;
    p.out = out;
    p.M = static_cast<int>(s->M);
    p.D = s->D;
    p.F = s->F;
    p.act = act_of(s);
    p.status = status;
    return status_from_cuda(m2rnn::launch_few(p, epi, true, false, st));
  }
  const int kt = k_tiles(s->D, 1);
  const m2rnn::GemmPlan q = m2rnn::gemm_plan(epi, false, s->M, s->F, 1, 1, kt);
  m2rnn::GemmParams p = gemm_params(q, s->M, s->F, 1, kt, false, status);
  const int box = pair ? q.bn / 2 : 128;
  if (!make_map(&p.a, x, 1, s->D, s->M, 1, x_row, x_row, 128) ||
      !make_map(&p.b0, w0, 1, s->D, s->F, 1, s->D, s->D, box))
    return M2RNN_ERR_CUDA;
  if (!pair)
    p.b1 = p.b0;
  else if (!make_map(&p.b1, w1, 1, s->D, s->F, 1, s->D, s->D, box))
    return M2RNN_ERR_CUDA;
  p.out[0] = out;
  p.in = res;
  p.in_row = res_row;
  p.sa = xs;
  p.sb0 = s0;
  p.sb1 = s1;
  p.act = act_of(s);
  return status_from_cuda(m2rnn::launch_gemm(p, {epi, false, false, q.bn, q.rows}, sms, st));
}

}  // namespace

extern "C" {

int m2rnn_glu_q8(const m2rnn_glu_shape* s, const void* x, long long x_row, const float* xs, const void* wg,
                 const float* wgs, const void* wu, const float* wus, void* h, void* stream) {
  return product_q8(s, x, x_row, xs, wg, wgs, wu, wus, nullptr, 0, h, true, stream);
}

int m2rnn_linear_q8(const m2rnn_glu_shape* s, const void* x, long long x_row, const float* xs, const void* w,
                    const float* ws, const void* res, long long res_row, void* y, void* stream) {
  return product_q8(s, x, x_row, xs, w, ws, nullptr, nullptr, res, res_row, y, false, stream);
}

}  // extern "C"

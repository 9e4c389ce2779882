// m2rnn_ffn.h (internal) -- launch parameters of the feed-forward operators
// (residual and norm, gated products, 8-bit product).  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/m2rnn_ffn.h"
#include "m2rnn_block.h"

namespace m2rnn {

// m2rnn_api.cu: the time limit of waits inside kernels.
unsigned long long host_wait_limit_ns();
int host_fault_injection();  // 1: kernels start no input transfers (a test hook)

// Location codes of the index checks and of waits that gave up.
enum FfnCheckSite : int {
  CHK_NORM2_IN = 801,     // x, res, r, dy, dr loads
  CHK_NORM2_OUT = 802,    // r, y, q, scale, dx stores
  CHK_NORM2_PARAM = 803,  // w loads, dw partials and sums
  CHK_GLU_IN = 901,       // x, weights, scales, dh, res loads
  CHK_GLU_OUT = 902,      // h, y, dx, dwg, dwu stores
  CHK_GLU_WS = 903,       // bf16 terms and the gradients of g and u
  SITE_GEMM_COPY = 951,   // waits of the product kernel
  SITE_GEMM_MMA = 952,
  SITE_GEMM_OUT = 953,
  SITE_GEMM_DRAIN = 954,
};

struct Norm2Params {
  const void *x, *res, *w, *dy, *dr;
  void *r, *y, *dx;
  uint8_t* q;
  float* scale;
  float* part;  // backward: [nparts][D]
  float* dw;
  long long xb, xt, rb, rt;  // rows of x (r in the backward pass) and res
  long long M;               // B * T rows of D elements
  int T, D;                  // T per item (M where the rows are evenly spaced)
  int nparts;
  float eps;
  int* status;
};
cudaError_t launch_add_norm(const Norm2Params& p, bool f32, int sms, cudaStream_t st);
cudaError_t launch_add_norm_bwd(const Norm2Params& p, bool f32, cudaStream_t st);
int add_norm_bwd_parts(const m2rnn_norm_shape* s);
cudaError_t launch_quant_rows(const Norm2Params& p, bool f32, cudaStream_t st);

// Products on the 5th-generation tensor core: out[m][n] = sum over segments and k of
// A[z][m][k] B[z][n][k], A and B as tensor maps of three dimensions.
enum GemmEpi : int {
  EPI_GLU,    // act(g) (.) u of a pair of products
  EPI_DGLU,   // gradients of g and u, as bf16 terms (1 or 2, fp32 3)
  EPI_STORE,  // the product itself
  EPI_GLU8,   // act(g) (.) u with scales
  EPI_LIN8,   // the product with scales, plus res
};
struct GemmParams {
  CUtensorMap a, b0, b1;  // b1: of a pair, or of the second segment
  int nseg;               // products that are added up: A's planes one after the other
  int aterms;             // bf16: planes of A that belong to one of B (b0, then b1)
  int kt;                 // K tiles of a segment
  int kc;                 // K tiles of a chunk (fp32: what one chain of sums takes)
  int mt, nt, nbatch;     // tiles; products that share B, of A's planes one after the other
  int whole;              // tiles that one unit of work takes each
  int split, nparts;      // parts of each other tile, and of all of them
  float* parts;           // their sums
  long long M;            // rows and columns of out
  int N;
  int pitch;              // EPI_DGLU: elements from a row of out to the next
  void* out[2];           // one for each of nbatch
  const void* in;         // dh, res
  long long in_row;
  const float *sa, *sb0, *sb1;
  int act;
  int* status;
  unsigned long long limit_ns;
  int inject_stall;       // test hook: no copies are issued
};
// Which instance: fp32 operands as terms; A with M fastest in memory (the weights' gradients); the
// tile's accumulator columns and rows (128 or 256).
struct GemmKind {
  int epi;
  bool f32, a_mn;
  int bn, rows;
};
cudaError_t launch_gemm(const GemmParams& p, const GemmKind& k, int sms, cudaStream_t st);
struct GemmPlan {
  int bn, rows;  // accumulator columns and rows of a tile
  int mt, nt, nbatch, whole, split, nparts;
  size_t parts_bytes;
};
GemmPlan gemm_plan(int epi, bool f32, long long m, int n, int nbatch, int nseg, int kt);

// Few tokens: the weights stream through registers (mma.sync).
struct FewParams {
  const void *x, *w0, *w1, *res;
  long long x_row, res_row;
  const float *sa, *sb0, *sb1;
  void* out;
  int M, D, F, act;
  int* status;
};
// Up to 16 tokens (fp32: 64) go this way.  us in a CUDA graph over 450 MB of weights, so from HBM,
// 16 tokens this way | 17 by the tiles:
//   D, F             gated bf16    gated e4m3    8-bit product (F to D)
//   1024, 2816       6.3 |  7.3    5.4 |  5.8    6.8 |  9.0
//   2048, 5632      12.7 | 18.0   10.9 | 11.4    7.2 | 13.5
//   4096, 11008     43.6 | 47.8   28.1 | 28.8   16.5 | 23.0
// fp32, 64 | 65 tokens: D=512 F=1408 12.0 | 17.4, D=1024 F=2816 38.1 | 27.7 (32 tokens 26.5).
// At D=2048 the tiles take 17.4 to 18.5 for 17 to 31 bf16 tokens and 12.3 from 32 on, for e4m3 10.6 to 11.5
// below 64 and 8.6 from there: the products are the same; why is not known.
inline int few_most(bool f32) { return f32 ? 64 : 16; }
cudaError_t launch_few(const FewParams& p, int epi, bool e4m3, bool f32, cudaStream_t st);

// fp32 matrices into three bf16 terms [3][M][pitch] each.
struct SplitParams {
  const float* src[3];
  long long row[3], M[3];
  __nv_bfloat16* dst[3];
  int D, pitch, n;
  int* status;
};
cudaError_t launch_split(const SplitParams& p, cudaStream_t st);

}  // namespace m2rnn

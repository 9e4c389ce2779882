// m2rnn_conv.cu -- the short causal convolution of a mixer block (a filter of
// W = 2..4 taps for each channel along time, then SiLU), its gradient and its
// single-token form:
//
//     z[t,c] = bias[c] + sum_{i<W} w[c,i] F[t+i,c],   y = z sigmoid(z),
//     dz = dy sigmoid(z) (1 + z (1 - sigmoid(z))),    dF[m,c] = sum_i w[c,i] dz[m-i,c],
//     dw[c,i] = sum_t dz[t,c] F[t+i,c],               dbias[c] = sum_t dz[t,c]
//
// with F = [state; x] along time (F[0..W-2] the carried inputs).
//
// All three kernels are bound by HBM traffic (2 W + 5 operations for each
// value read and written).  A thread owns a few neighbouring channels
// and walks along time with the last W rows of F (backward: and of dz) in
// registers, so each value is loaded once apart from the W - 1 rows
// before a thread's run, which its neighbour has just pulled into L2.
// Neighbouring lanes own neighbouring channels: every row is read in whole
// 128-byte lines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"
#include "m2rnn_vec.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

// sigmoid(z) from e = exp(-z): e = inf gives 0.
template <bool F32>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (F32)
    return 1.f / (1.f + expf(-z));
  else  // the fast forms' error (about 2^-21) is far below the output's rounding (2^-9)
    return __fdividef(1.f, 1.f + __expf(-z));
}

// Row m of F for channels c0.. of batch item b (m in [0, T + W - 1)).
template <bool F32, int VEC, int W>
__device__ __forceinline__ Raw<F32, VEC> row_of(const ConvParams& p, int b, long long m, int c0) {
  using E = typename Elem<F32>::T;
  if (m >= W - 1) {
    const long long t = m - (W - 1);
    if (!in_range(p.status, static_cast<size_t>(t), 1, p.T, CHK_CONV_IN) ||
        !in_range(p.status, c0, VEC, p.C, CHK_CONV_IN))
      return raw_zero<F32, VEC>();
    return raw_load<F32, VEC>(static_cast<const E*>(p.x) + b * p.xb + t * p.xt + c0);
  }
  if (p.state == nullptr) return raw_zero<F32, VEC>();
  const size_t at = (static_cast<size_t>(b) * (W - 1) + m) * p.C + c0;
  if (!in_range(p.status, at, VEC, static_cast<size_t>(p.B) * (W - 1) * p.C, CHK_CONV_IN))
    return raw_zero<F32, VEC>();
  return raw_load<F32, VEC>(static_cast<const E*>(p.state) + at);
}

// The taps of VEC channels, w[c][i], and their bias.
template <bool F32, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvParams& p, int c0, float (&w)[VEC][W],
                                          float (&bias)[VEC]) {
  using E = typename Elem<F32>::T;
#pragma unroll
  for (int j = 0; j < VEC; ++j) bias[j] = 0.f;
  if (!in_range(p.status, c0, VEC, p.C, CHK_CONV_PARAM)) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) w[j][i] = 0.f;
    return;
  }
  const E* src = static_cast<const E*>(p.w) + static_cast<size_t>(c0) * W;
#pragma unroll
  for (int g = 0; g < W; ++g) {  // VEC * W values, VEC at a time
    float t[VEC];
    load_vec<F32, VEC>(src + g * VEC, t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[(g * VEC + e) / W][(g * VEC + e) % W] = t[e];
  }
  if (p.bias != nullptr) load_vec<F32, VEC>(static_cast<const E*>(p.bias) + c0, bias);
}

template <bool F32, int VEC, int W, bool SILU>
__device__ __forceinline__ void apply(const float (&f)[W][VEC], const float (&w)[VEC][W],
                                      const float (&bias)[VEC], float (&y)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    float z = bias[j];
#pragma unroll
    for (int i = 0; i < W; ++i) z = fmaf(w[j][i], f[i][j], z);
    y[j] = SILU ? z * sigmoid<F32>(z) : z;
  }
}

// One thread: VEC channels x TT tokens.
template <bool F32, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const ConvParams p) {
  using E = typename Elem<F32>::T;
  constexpr int U = 4;  // rows in flight per thread
  const int cv = p.C / VEC;
  const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (item >= static_cast<long long>(p.B) * p.nT * cv) return;
  const int c0 = static_cast<int>(item % cv) * VEC;
  const int chunk = static_cast<int>((item / cv) % p.nT);
  const int b = static_cast<int>(item / cv / p.nT);
  const int t0 = chunk * p.TT, t1 = min(p.T, t0 + p.TT);
  float w[VEC][W], bias[VEC], f[W][VEC];
  Raw<F32, VEC> last[W - 1];  // F[t .. t+W-2] as they lie in memory
#pragma unroll
  for (int i = 0; i < W - 1; ++i) last[i] = row_of<F32, VEC, W>(p, b, t0 + i, c0);
  load_taps<F32, VEC, W>(p, c0, w, bias);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) raw_unpack<F32, VEC>(last[i], f[i]);
  E* y = static_cast<E*>(p.y);
  for (int t = t0; t < t1; t += U) {
    Raw<F32, VEC> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      r[u] = t + u < t1 ? row_of<F32, VEC, W>(p, b, t + u + W - 1, c0) : raw_zero<F32, VEC>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u >= t1) break;
      raw_unpack<F32, VEC>(r[u], f[W - 1]);
      float o[VEC];
      apply<F32, VEC, W, SILU>(f, w, bias, o);
      const size_t at = (static_cast<size_t>(b) * p.T + t + u) * p.C + c0;
      if (in_range(p.status, at, VEC, static_cast<size_t>(p.B) * p.T * p.C, CHK_CONV_OUT))
        store_vec<F32, VEC>(y + at, o);
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[i][j] = f[i + 1][j];
    }
  }
  if (t1 == p.T && p.state_out != nullptr) {  // f now holds F's last W - 1 rows
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const size_t at = (static_cast<size_t>(b) * (W - 1) + i) * p.C + c0;
      if (in_range(p.status, at, VEC, static_cast<size_t>(p.B) * (W - 1) * p.C, CHK_CONV_OUT))
        store_vec<F32, VEC>(static_cast<E*>(p.state_out) + at, f[i]);
    }
  }
}

// One thread: 4 channels of one sequence; the state may be updated in place.
template <bool F32, int W, bool SILU>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p) {
  using E = typename Elem<F32>::T;
  constexpr int VEC = 4;
  const int cv = p.C / VEC;
  const long long item = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  if (item >= static_cast<long long>(p.B) * cv) return;
  const int c0 = static_cast<int>(item % cv) * VEC, b = static_cast<int>(item / cv);
  Raw<F32, VEC> r[W];
  float f[W][VEC], w[VEC][W], bias[VEC], o[VEC];
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = row_of<F32, VEC, W>(p, b, i, c0);
  load_taps<F32, VEC, W>(p, c0, w, bias);
#pragma unroll
  for (int i = 0; i < W; ++i) raw_unpack<F32, VEC>(r[i], f[i]);
  apply<F32, VEC, W, SILU>(f, w, bias, o);
  const size_t yat = static_cast<size_t>(b) * p.C + c0;
  if (in_range(p.status, yat, VEC, static_cast<size_t>(p.B) * p.C, CHK_CONV_OUT))
    store_vec<F32, VEC>(static_cast<E*>(p.y) + yat, o);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const size_t at = (static_cast<size_t>(b) * (W - 1) + i) * p.C + c0;
    if (in_range(p.status, at, VEC, static_cast<size_t>(p.B) * (W - 1) * p.C, CHK_CONV_OUT))
      raw_store<F32, VEC>(static_cast<E*>(p.state_out) + at, r[i + 1]);
  }
}

// A warp takes 128 channels (4 per lane: more would not leave the registers
// for the taps, the two windows and the sums) and runs of TT rows of F; a run
// [m0, m0 + TT) writes dF there and adds dz's products for tokens in it.  The
// eight warps' sums are added in warp order, the CTAs' by sum_parts_kernel.
template <bool F32, bool G32, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvParams p) {
  using E = typename Elem<F32>::T;
  using G = typename Elem<G32>::T;
  constexpr int VEC = 4, kWarps = kThreads / 32, U = 2;
  __shared__ float sums[kWarps][32 * VEC * (W + 1)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (blockIdx.x * 32 + lane) * VEC;
  const bool active = c0 < p.C;
  const long long rows = static_cast<long long>(p.T) + W - 1;
  const size_t xn = static_cast<size_t>(p.B) * p.T * p.C;
  const size_t sn = static_cast<size_t>(p.B) * (W - 1) * p.C;
  float dw[VEC][W], db[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    db[j] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) dw[j][i] = 0.f;
  }
  if (active) {
    float w[VEC][W], bias[VEC];
    load_taps<F32, VEC, W>(p, c0, w, bias);
    const long long runs = static_cast<long long>(p.B) * p.nT;
    for (long long g = static_cast<long long>(blockIdx.y) * kWarps + warp; g < runs;
         g += static_cast<long long>(gridDim.y) * kWarps) {
      const int b = static_cast<int>(g / p.nT);
      const long long m0 = (g % p.nT) * p.TT;
      const long long m1 = m0 + p.TT < rows ? m0 + p.TT : rows;
      const long long first = m0 - (W - 1) > 0 ? m0 - (W - 1) : 0;
      float f[W][VEC], dz[W][VEC];  // dz[i]: of token t - (W-1) + i
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[i][j] = dz[i][j] = 0.f;
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
        if (first + i < rows) raw_unpack<F32, VEC>(row_of<F32, VEC, W>(p, b, first + i, c0), f[i]);
      for (long long t = first; t < m1; t += U) {
        Raw<F32, VEC> rx[U];
        Raw<G32, VEC> rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = raw_zero<F32, VEC>();
          rg[u] = raw_zero<G32, VEC>();
          if (t + u < p.T && t + u < m1) {
            rx[u] = row_of<F32, VEC, W>(p, b, t + u + W - 1, c0);
            const size_t at = (static_cast<size_t>(b) * p.T + t + u) * p.C + c0;
            if (in_range(p.status, at, VEC, xn, CHK_CONV_IN))
              rg[u] = raw_load<G32, VEC>(static_cast<const G*>(p.dy) + at);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long m = t + u;
          if (m >= m1) break;
          float gy[VEC];
          raw_unpack<F32, VEC>(rx[u], f[W - 1]);
          raw_unpack<G32, VEC>(rg[u], gy);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float d = gy[j];
            if (SILU) {
              float z = bias[j];
#pragma unroll
              for (int i = 0; i < W; ++i) z = fmaf(w[j][i], f[i][j], z);
              const float s = sigmoid<F32>(z);
              d *= s * fmaf(z, 1.f - s, 1.f);
            }
            dz[W - 1][j] = m < p.T ? d : 0.f;
          }
          if (m >= m0) {
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              o[j] = 0.f;
#pragma unroll
              for (int i = 0; i < W; ++i) {
                o[j] = fmaf(w[j][i], dz[W - 1 - i][j], o[j]);
                dw[j][i] = fmaf(dz[W - 1][j], f[i][j], dw[j][i]);
              }
              db[j] += dz[W - 1][j];
            }
            if (m >= p.T && p.dstate_out != nullptr) {
              const size_t at = (static_cast<size_t>(b) * (W - 1) + (m - p.T)) * p.C + c0;
              float ds[VEC];
              if (in_range(p.status, at, VEC, sn, CHK_CONV_IN)) {
                load_vec<F32, VEC>(static_cast<const E*>(p.dstate_out) + at, ds);
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[j] += ds[j];
              }
            }
            if (m >= W - 1) {
              const size_t at = (static_cast<size_t>(b) * p.T + (m - (W - 1))) * p.C + c0;
              if (in_range(p.status, at, VEC, xn, CHK_CONV_OUT))
                store_vec<F32, VEC>(static_cast<E*>(p.dx) + at, o);
            } else if (p.dstate != nullptr) {
              const size_t at = (static_cast<size_t>(b) * (W - 1) + m) * p.C + c0;
              if (in_range(p.status, at, VEC, sn, CHK_CONV_OUT))
                store_vec<F32, VEC>(static_cast<E*>(p.dstate) + at, o);
            }
          }
#pragma unroll
          for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              f[i][j] = f[i + 1][j];
              dz[i][j] = dz[i + 1][j];
            }
        }
      }
    }
  }
  // the part's layout: dw [C][W], then dbias [C]
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
#pragma unroll
    for (int i = 0; i < W; ++i) sums[warp][(lane * VEC + j) * W + i] = dw[j][i];
    sums[warp][32 * VEC * W + lane * VEC + j] = db[j];
  }
  __syncthreads();
  const int cols = min(32 * VEC, p.C - static_cast<int>(blockIdx.x) * 32 * VEC);
  float* part = p.part + static_cast<size_t>(blockIdx.y) * p.C * (W + 1);
  for (int e = threadIdx.x; e < 32 * VEC * (W + 1); e += kThreads) {
    const bool is_w = e < 32 * VEC * W;
    const int c = is_w ? e / W : e - 32 * VEC * W;
    if (c >= cols) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) s += sums[k][e];
    const size_t at = is_w ? static_cast<size_t>(blockIdx.x) * 32 * VEC * W + e
                           : static_cast<size_t>(p.C) * W + blockIdx.x * 32 * VEC + c;
    if (in_range(p.status, at, 1, static_cast<size_t>(p.C) * (W + 1), CHK_CONV_PARAM)) part[at] = s;
  }
}

template <bool F32, int W, bool SILU>
cudaError_t fwd_w(const ConvParams& p, cudaStream_t st) {
  // 16-byte loads in both types: 8 channels of bf16, 4 of fp32
  constexpr int VEC = F32 ? 4 : 8;
  const long long items = static_cast<long long>(p.B) * p.nT * (p.C / VEC);
  const long long grid = (items + kThreads - 1) / kThreads;
  conv_fwd_kernel<F32, VEC, W, SILU><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool F32, int W, bool SILU>
cudaError_t step_w(const ConvParams& p, cudaStream_t st) {
  const long long items = static_cast<long long>(p.B) * (p.C / 4);
  conv_step_kernel<F32, W, SILU>
      <<<static_cast<unsigned>((items + 127) / 128), 128, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool F32, int W, bool SILU>
cudaError_t bwd_w(const ConvParams& p, bool grad_f32, cudaStream_t st) {
  const dim3 grid((p.C + 127) / 128, p.nparts);
  if (F32 || grad_f32)
    conv_bwd_kernel<F32, true, W, SILU><<<grid, kThreads, 0, st>>>(p);
  else
    conv_bwd_kernel<F32, F32, W, SILU><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// f<F32, W, SILU>(args...) for the call's type, taps and activation.
#define M2RNN_CONV_DISPATCH(fn, ...)                                                       \
  do {                                                                                     \
    if (f32) {                                                                             \
      if (p.W == 2) return silu ? fn<true, 2, true>(__VA_ARGS__) : fn<true, 2, false>(__VA_ARGS__);   \
      if (p.W == 3) return silu ? fn<true, 3, true>(__VA_ARGS__) : fn<true, 3, false>(__VA_ARGS__);   \
      return silu ? fn<true, 4, true>(__VA_ARGS__) : fn<true, 4, false>(__VA_ARGS__);      \
    }                                                                                      \
    if (p.W == 2) return silu ? fn<false, 2, true>(__VA_ARGS__) : fn<false, 2, false>(__VA_ARGS__);   \
    if (p.W == 3) return silu ? fn<false, 3, true>(__VA_ARGS__) : fn<false, 3, false>(__VA_ARGS__);   \
    return silu ? fn<false, 4, true>(__VA_ARGS__) : fn<false, 4, false>(__VA_ARGS__);      \
  } while (0)

}  // namespace

// Tokens per thread: long runs re-read fewer rows at their start (W - 1 of
// TT), short ones give more threads; the longest run that still leaves
// 2,048 threads for each SM, 4 tokens at least.
int conv_fwd_tokens(const m2rnn_conv_shape* s, int sms) {
  const int vec = s->in_dtype == M2RNN_F32 ? 4 : 8;
  const long long per_token = static_cast<long long>(s->B) * (s->C / vec);
  int tt = 32;
  while (tt > 4 && per_token * ((s->T + tt - 1) / tt) < 2048LL * sms) tt /= 2;
  return tt;
}

// Runs of 32 rows, 16 or 8 where the sequences are short; at most 1,216 CTAs
// (8 for each of 152 SMs), so that the parts stay a small share of the bytes.
void conv_bwd_plan(const m2rnn_conv_shape* s, int* TT, int* nT, int* nparts) {
  const long long rows = static_cast<long long>(s->T) + s->W - 1;
  const int groups = (s->C + 127) / 128;
  int tt = 32;
  while (tt > 8 && s->B * ((rows + tt - 1) / tt) * groups < 8LL * 1216) tt /= 2;
  *TT = tt;
  *nT = static_cast<int>((rows + tt - 1) / tt);
  const long long need = (static_cast<long long>(s->B) * *nT + 7) / 8;
  const long long most = 1216 / groups > 1 ? 1216 / groups : 1;
  *nparts = static_cast<int>(need < most ? need : most);
}

cudaError_t launch_conv_fwd(const ConvParams& p, bool f32, bool silu, cudaStream_t st) {
  M2RNN_CONV_DISPATCH(fwd_w, p, st);
}

cudaError_t launch_conv_step(const ConvParams& p, bool f32, bool silu, cudaStream_t st) {
  M2RNN_CONV_DISPATCH(step_w, p, st);
}

static cudaError_t conv_bwd_main(const ConvParams& p, bool f32, bool grad_f32, bool silu,
                                 cudaStream_t st) {
  M2RNN_CONV_DISPATCH(bwd_w, p, grad_f32, st);
}

cudaError_t launch_conv_bwd(const ConvParams& p, bool f32, bool grad_f32, bool silu,
                            cudaStream_t st) {
  const cudaError_t e = conv_bwd_main(p, f32, grad_f32, silu, st);
  if (e != cudaSuccess) return e;
  const SumOut o{{p.dw, p.dbias, nullptr}, {p.C * p.W, p.C, 0}};
  return launch_sum_parts(p.part, p.nparts, o, p.status, CHK_CONV_PARAM, st);
}

}  // namespace m2rnn

// m2rnn_qknorm.cu -- RMS norm of every query and key head with the position
// rotation in the same pass, and its gradient:
//
//     r = (mean_k x^2 + eps)^(-1/2),   xh = x r,   u = w (.) xh,   out = Rot(u),
//     du = Rot^T(dout),  g = w (.) du,  dx = r (g - xh mean_k(g xh)),
//     dw = sum over rows of du (.) xh
//
// where Rot turns the pairs of the first R features by the token's angles.
//
// Bound by HBM traffic: every row is read once and written once.  K / 8 lanes
// hold a head's row, 8 features each (one 16-byte load of bf16); the row's
// sums are shuffles among them.  The rotation's partner feature is in the
// same lane (interleaved pairs) or in the lane R / 16 further on (one
// shuffle).  A lane group takes several heads of one token, so that the
// token's cosines and sines are loaded once for all of them: per head they
// would be 8 R bytes next to 2 K bytes of row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"
#include "m2rnn_vec.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

// Sum over the LPR lanes of a row, in every lane.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m >= 1; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// A lane's share of one token's rotation.
struct Angles {
  float c[8], n[8];  // cosine and signed sine of each of the lane's features
  int src;           // lane (of the row's) that holds the partner features
};

// The partner of feature j (0..7) of the lane, given the lane's own values.
__device__ __forceinline__ void partners(const QkParams& p, const Angles& a, const float (&u)[8],
                                         float (&o)[8], int lpr) {
  if (p.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = u[j ^ 1];
  } else if (p.R == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = u[j ^ 4];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, u[j], a.src, lpr);
  }
}

// Angles of token `token` for row lane l.  The sine carries the sign with
// which the partner enters: first of a pair -, second +.
__device__ __forceinline__ void load_angles(const QkParams& p, long long token, int l, bool valid,
                                            Angles& a) {
  a.src = l;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a.c[j] = 1.f;
    a.n[j] = 0.f;
  }
  if (p.R == 0) return;
  const int half = p.R / 2;
  if (!p.interleaved && p.R >= 16 && 8 * l < p.R) a.src = 8 * l < half ? l + half / 8 : l - half / 8;
  if (!valid || 8 * l >= p.R) return;
  int pos = static_cast<int>(token % p.T);
  if (p.pos != nullptr) pos = __ldg(p.pos + token);
  if (pos < 0 || pos >= p.P) {
    if (atomicCAS(&p.status[0], 0, kStatusBounds) == 0) atomicExch(&p.status[1], CHK_QK_POS);
#pragma unroll
    for (int j = 0; j < 8; ++j) a.c[j] = a.n[j] = __int_as_float(0x7fffffff);
    return;
  }
  const float* cs = p.cs + static_cast<size_t>(pos) * half;
  const float* sn = p.sn + static_cast<size_t>(pos) * half;
  if (p.interleaved || p.R == 8) {  // four angles for the lane's eight features
    const int i0 = p.interleaved ? 4 * l : 0;
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i0));
    const float4 n = __ldg(reinterpret_cast<const float4*>(sn + i0));
    const float cc[4] = {c.x, c.y, c.z, c.w}, nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ci = p.interleaved ? j / 2 : j % 4;
      const bool second = p.interleaved ? (j & 1) : j >= 4;
      a.c[j] = ci == 0 ? cc[0] : ci == 1 ? cc[1] : ci == 2 ? cc[2] : cc[3];
      const float s = ci == 0 ? nn[0] : ci == 1 ? nn[1] : ci == 2 ? nn[2] : nn[3];
      a.n[j] = second ? s : -s;
    }
    return;
  }
  const bool second = 8 * l >= half;
  const int i0 = second ? 8 * l - half : 8 * l;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i0) + g);
    const float4 n = __ldg(reinterpret_cast<const float4*>(sn + i0) + g);
    a.c[4 * g] = c.x; a.c[4 * g + 1] = c.y; a.c[4 * g + 2] = c.z; a.c[4 * g + 3] = c.w;
    a.n[4 * g] = second ? n.x : -n.x;
    a.n[4 * g + 1] = second ? n.y : -n.y;
    a.n[4 * g + 2] = second ? n.z : -n.z;
    a.n[4 * g + 3] = second ? n.w : -n.w;
  }
}

// o = Rot(u) for sign = 1, Rot^T(u) for sign = -1.
__device__ __forceinline__ void rotate(const QkParams& p, const Angles& a, float sign, int lpr,
                                       const float (&u)[8], float (&o)[8]) {
  if (p.R == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = u[j];
    return;
  }
  float v[8];
  partners(p, a, u, v, lpr);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = fmaf(u[j], a.c[j], sign * a.n[j] * v[j]);
}

template <bool F32>
__device__ __forceinline__ void load_weight(const QkParams& p, const void* w, int l, float (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = 1.f;
  if (w != nullptr && in_range(p.status, 8 * l, 8, p.K, CHK_QK_PARAM))
    load_vec<F32, 8>(static_cast<const typename Elem<F32>::T*>(w) + 8 * l, o);
}

// Input row of head h (queries first, then keys) of a token.
template <bool F32>
__device__ __forceinline__ Raw<F32, 8> load_row(const QkParams& p, int b, int t, int h, int l) {
  using E = typename Elem<F32>::T;
  const bool isq = h < p.Nq;
  const int hh = isq ? h : h - p.Nq;
  if (!in_range(p.status, static_cast<size_t>(hh) * p.K + 8 * l, 8,
                static_cast<size_t>(isq ? p.Nq : p.Nk) * p.K, CHK_QK_IN) ||
      !in_range(p.status, t, 1, p.T, CHK_QK_IN))
    return raw_zero<F32, 8>();
  const E* base = isq ? static_cast<const E*>(p.q) + b * p.qb + t * p.qt
                      : static_cast<const E*>(p.k) + b * p.kb + t * p.kt;
  return raw_load<F32, 8>(base + hh * p.K + 8 * l);
}

// Offset of head h's row of a token in a contiguous [tokens][Nq or Nk][K].
__device__ __forceinline__ size_t out_at(const QkParams& p, long long token, int h, int l) {
  return h < p.Nq ? (static_cast<size_t>(token) * p.Nq + h) * p.K + 8 * l
                  : (static_cast<size_t>(token) * p.Nk + (h - p.Nq)) * p.K + 8 * l;
}
__device__ __forceinline__ size_t out_extent(const QkParams& p, int h) {
  return static_cast<size_t>(p.tokens) * (h < p.Nq ? p.Nq : p.Nk) * p.K;
}

// A lane group takes heads g, g + split, ... of one token, U at a time.
template <bool F32, int LPR>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const QkParams p) {
  using E = typename Elem<F32>::T;
  constexpr int U = F32 ? 2 : 4;  // rows in flight
  const long long gid = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  const long long token = gid / p.split;
  const int g = static_cast<int>(gid % p.split);
  const int heads = p.Nq + p.Nk;
  const bool valid = token < p.tokens && 8 * l < p.K;
  const int b = static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
  Angles a;
  load_angles(p, token, l, valid, a);
  float wq[8], wk[8];
  load_weight<F32>(p, 8 * l < p.K ? p.wq : nullptr, l, wq);
  load_weight<F32>(p, 8 * l < p.K ? p.wk : nullptr, l, wk);
  const float inv_k = 1.f / static_cast<float>(p.K);
  const int steps = (heads + p.split - 1) / p.split;  // the same for every lane: shuffles below
  for (int s0 = 0; s0 < steps; s0 += U) {
    Raw<F32, 8> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = g + (s0 + u) * p.split;
      r[u] = valid && h < heads ? load_row<F32>(p, b, t, h, l) : raw_zero<F32, 8>();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u >= steps) break;
      const int h = g + (s0 + u) * p.split;
      float x[8], o[8], ss = 0.f;
      raw_unpack<F32, 8>(r[u], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
      const float rs = rsqrtf(row_sum<LPR>(ss) * inv_k + p.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= rs * (h < p.Nq ? wq[j] : wk[j]);
      rotate(p, a, 1.f, LPR, x, o);
      if (valid && h < heads) {
        const size_t at = out_at(p, token, h, l);
        if (in_range(p.status, at, 8, out_extent(p, h), CHK_QK_OUT))
          store_vec<F32, 8>(static_cast<E*>(h < p.Nq ? p.qo : p.ko) + at, o);
      }
    }
  }
}

// As the forward kernel, with the groups walking over the tokens: a lane
// keeps its features' shares of dwq and dwk in registers throughout.
template <bool F32, bool G32, int LPR>
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const QkParams p) {
  using E = typename Elem<F32>::T;
  using G = typename Elem<G32>::T;
  constexpr int U = 2, kGroups = kThreads / LPR;
  __shared__ float sums[2][kGroups][8 * LPR + 1];
  const int l = threadIdx.x % LPR;
  const int heads = p.Nq + p.Nk;
  const float inv_k = 1.f / static_cast<float>(p.K);
  const bool lane_on = 8 * l < p.K;
  float wq[8], wk[8], dwq[8], dwk[8];
  load_weight<F32>(p, lane_on ? p.wq : nullptr, l, wq);
  load_weight<F32>(p, lane_on ? p.wk : nullptr, l, wk);
#pragma unroll
  for (int j = 0; j < 8; ++j) dwq[j] = dwk[j] = 0.f;
  const long long items = p.tokens * p.split;
  const int steps = (heads + p.split - 1) / p.split;
  // i0: the CTA's first group, the same for all of its warps
  for (long long i0 = static_cast<long long>(blockIdx.x) * kGroups; i0 < items;
       i0 += static_cast<long long>(gridDim.x) * kGroups) {
    const long long item = i0 + threadIdx.x / LPR;
    const long long token = item / p.split;
    const int g = static_cast<int>(item % p.split);
    const bool valid = item < items && lane_on;
    const int b = static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
    Angles a;
    load_angles(p, token, l, valid, a);
    for (int s0 = 0; s0 < steps; s0 += U) {
      Raw<F32, 8> rx[U];
      Raw<G32, 8> ry[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = g + (s0 + u) * p.split;
        rx[u] = raw_zero<F32, 8>();
        ry[u] = raw_zero<G32, 8>();
        if (valid && h < heads) {
          rx[u] = load_row<F32>(p, b, t, h, l);
          const size_t at = out_at(p, token, h, l);
          if (in_range(p.status, at, 8, out_extent(p, h), CHK_QK_IN))
            ry[u] = raw_load<G32, 8>(static_cast<const G*>(h < p.Nq ? p.dqo : p.dko) + at);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s0 + u >= steps) break;
        const int h = g + (s0 + u) * p.split;
        const bool on = valid && h < heads, isq = h < p.Nq;
        float x[8], y[8], du[8], ss = 0.f;
        raw_unpack<F32, 8>(rx[u], x);
        raw_unpack<G32, 8>(ry[u], y);
        rotate(p, a, -1.f, LPR, y, du);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        const float rs = rsqrtf(row_sum<LPR>(ss) * inv_k + p.eps);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] *= rs;  // xh
          if (on) {    // a head that is not there has x = 0 and, for eps = 0, xh = NaN
            if (isq)
              dwq[j] = fmaf(du[j], x[j], dwq[j]);
            else
              dwk[j] = fmaf(du[j], x[j], dwk[j]);
          }
          du[j] *= isq ? wq[j] : wk[j];  // g
          dot = fmaf(du[j], x[j], dot);
        }
        // Lanes past the row's end hold zeros, or NaN times zero when eps = 0:
        // they must not enter the row's sum.
        dot = row_sum<LPR>(lane_on ? dot : 0.f) * inv_k;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = rs * fmaf(-x[j], dot, du[j]);
        if (on) {
          const size_t at = out_at(p, token, h, l);
          if (in_range(p.status, at, 8, out_extent(p, h), CHK_QK_OUT))
            store_vec<F32, 8>(static_cast<E*>(isq ? p.dq : p.dk) + at, y);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sums[0][threadIdx.x / LPR][8 * l + j] = dwq[j];
    sums[1][threadIdx.x / LPR][8 * l + j] = dwk[j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * p.K; e += kThreads) {
    float s = 0.f;
    for (int i = 0; i < kGroups; ++i) s += sums[e / p.K][i][e % p.K];
    const size_t at = static_cast<size_t>(blockIdx.x) * 2 * p.K + e;
    if (in_range(p.status, at, 1, static_cast<size_t>(p.nparts) * 2 * p.K, CHK_QK_PARAM))
      p.part[at] = s;
  }
}

int lanes_per_row(int K) {
  int n = 1;
  while (8 * n < K) n *= 2;
  return n;
}

template <bool F32, int LPR>
cudaError_t fwd_l(const QkParams& p, cudaStream_t st) {
  const long long threads = p.tokens * p.split * LPR;
  const long long grid = (threads + kThreads - 1) / kThreads;
  qk_fwd_kernel<F32, LPR><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool F32, int LPR>
cudaError_t bwd_l(const QkParams& p, bool grad_f32, cudaStream_t st) {
  if (F32 || grad_f32)
    qk_bwd_kernel<F32, true, LPR><<<p.nparts, kThreads, 0, st>>>(p);
  else
    qk_bwd_kernel<F32, F32, LPR><<<p.nparts, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

#define M2RNN_QK_DISPATCH(fn, F32, ...)             \
  switch (lanes_per_row(p.K)) {                     \
    case 1: return fn<F32, 1>(__VA_ARGS__);         \
    case 2: return fn<F32, 2>(__VA_ARGS__);         \
    case 4: return fn<F32, 4>(__VA_ARGS__);         \
    case 8: return fn<F32, 8>(__VA_ARGS__);         \
    case 16: return fn<F32, 16>(__VA_ARGS__);       \
    default: return fn<F32, 32>(__VA_ARGS__);       \
  }

cudaError_t bwd_main(const QkParams& p, bool f32, bool grad_f32, cudaStream_t st) {
  if (f32) {
    M2RNN_QK_DISPATCH(bwd_l, true, p, grad_f32, st)
  }
  M2RNN_QK_DISPATCH(bwd_l, false, p, grad_f32, st)
}

}  // namespace

// Lane groups per token: one, so that a token's angles are loaded once,
// unless that leaves fewer than 1,024 threads for each of 152 SMs.
int qk_split(const m2rnn_qk_shape* s) {
  const long long tokens = static_cast<long long>(s->B) * s->T;
  const int heads = s->Nq + s->Nk, lpr = lanes_per_row(s->K);
  if (tokens <= 0) return 1;
  const long long want = (152LL * 1024 / lpr + tokens - 1) / tokens;
  return static_cast<int>(want < 1 ? 1 : want > heads ? heads : want);
}

int qk_bwd_parts(const m2rnn_qk_shape* s) {
  const long long groups = static_cast<long long>(s->B) * s->T * qk_split(s);
  const long long per_cta = kThreads / lanes_per_row(s->K);
  const long long need = (groups + per_cta - 1) / per_cta;
  return static_cast<int>(need < 152 * 4 ? need : 152 * 4);
}

cudaError_t launch_qk_fwd(const QkParams& p, bool f32, int sms, cudaStream_t st) {
  (void)sms;
  if (f32) {
    M2RNN_QK_DISPATCH(fwd_l, true, p, st)
  }
  M2RNN_QK_DISPATCH(fwd_l, false, p, st)
}

cudaError_t launch_qk_bwd(const QkParams& p, bool f32, bool grad_f32, cudaStream_t st) {
  const cudaError_t e = bwd_main(p, f32, grad_f32, st);
  if (e != cudaSuccess) return e;
  const SumOut o{{p.dwq, p.dwk, nullptr}, {p.K, p.K, 0}};
  return launch_sum_parts(p.part, p.nparts, o, p.status, CHK_QK_PARAM, st);
}

}  // namespace m2rnn

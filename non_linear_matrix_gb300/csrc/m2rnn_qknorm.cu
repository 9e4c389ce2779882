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
// hold a head's row as two quads of features each; the row's sums are
// shuffles among them.  A lane's quads are chosen so that both features of a
// rotated pair are its own (quads i and i + R/2 for pairs at that distance), so
// that the rotation needs no exchange: with eight neighbouring features per
// lane it took eight shuffles a row, and the forward kernel 77 us instead of 44
// (B=8 T=2048, 64 heads of 64, 269 MB: 6.1 TB/s; the backward one takes 51 us at
// B=8 T=4096, 10 heads of 128, 252 MB: 4.9 TB/s).  A lane group takes several heads of one token,
// so that the token's cosines and sines are loaded once for all of them: per head
// they would be 4 R bytes next to 2 K bytes of row.
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

// A lane's place in a row: the first features of its two quads, whether they
// rotate, and the token's angles for them.
struct Lane {
  int o[2];
  bool on, turns;
  float2 c[2], n[2];  // cosine, sine of angles i .. i + 3
};

template <int LPR>
__device__ __forceinline__ Lane lane_of(const QkParams& p) {
  const int l = threadIdx.x % LPR;
  Lane a;
  a.on = 8 * l < p.K;
  a.turns = 8 * l < p.R;
  const bool apart = a.turns && !p.interleaved;
  a.o[0] = apart ? 4 * l : 8 * l;
  a.o[1] = apart ? 4 * l + p.R / 2 : 8 * l + 4;
  a.c[0] = a.c[1] = make_float2(1.f, 1.f);
  a.n[0] = a.n[1] = make_float2(0.f, 0.f);
  return a;
}

// The angles of a token.
template <int LPR>
__device__ __forceinline__ void load_angles(const QkParams& p, long long token, int t, bool valid,
                                            Lane& a) {
  if (!valid || !a.turns) return;
  const int pos = p.pos != nullptr ? __ldg(p.pos + token) : t;
  if (pos < 0 || pos >= p.P) {
    if (atomicCAS(&p.status[0], 0, kStatusBounds) == 0) atomicExch(&p.status[1], CHK_QK_POS);
    const float nan = __int_as_float(0x7fffffff);
    a.c[0] = a.c[1] = a.n[0] = a.n[1] = make_float2(nan, nan);
    return;
  }
  const size_t at = static_cast<size_t>(pos) * (p.R / 2) + 4 * (threadIdx.x % LPR);
  const float4 c = __ldg(reinterpret_cast<const float4*>(p.cs + at));
  const float4 n = __ldg(reinterpret_cast<const float4*>(p.sn + at));
  a.c[0] = make_float2(c.x, c.y);
  a.c[1] = make_float2(c.z, c.w);
  a.n[0] = make_float2(n.x, n.y);
  a.n[1] = make_float2(n.z, n.w);
}

// u[0..1], u[2..3]: the lane's quads as pairs; turned in place by the angles
// (TURN = 1) or back (-1).
template <int TURN>
__device__ __forceinline__ void rotate(const QkParams& p, const Lane& a, float2 (&u)[4]) {
  if (p.R == 0) return;
  if (p.interleaved) {  // (2i, 2i + 1) is one of the pairs
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float c = (j & 1) ? a.c[j / 2].y : a.c[j / 2].x;
      const float n = TURN * ((j & 1) ? a.n[j / 2].y : a.n[j / 2].x);
      const float2 r = make_float2(fmaf(u[j].x, c, -u[j].y * n), fmaf(u[j].y, c, u[j].x * n));
      u[j] = a.turns ? r : u[j];  // (1 and 0 in place of c and n would make NaN of a partner's inf)
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // first quad with second
    const float2 n = a.n[j], m = make_float2(-n.x, -n.y);
    const float2 x = u[j], y = u[2 + j];
    const float2 xr = fma2(y, TURN > 0 ? m : n, mul2(x, a.c[j]));
    const float2 yr = fma2(x, TURN > 0 ? n : m, mul2(y, a.c[j]));
    u[j] = a.turns ? xr : x;
    u[2 + j] = a.turns ? yr : y;
  }
}

template <bool F32>
struct RawRow {
  Raw<F32, 4> q[2];
};
template <bool F32>
__device__ __forceinline__ RawRow<F32> row_zero() {
  return RawRow<F32>{{raw_zero<F32, 4>(), raw_zero<F32, 4>()}};
}
template <bool F32>
__device__ __forceinline__ RawRow<F32> row_load(const typename Elem<F32>::T* src, const Lane& a) {
  return RawRow<F32>{{raw_load<F32, 4>(src + a.o[0]), raw_load<F32, 4>(src + a.o[1])}};
}
template <bool F32>
__device__ __forceinline__ void row_unpack(const RawRow<F32>& r, float2 (&o)[4]) {
  float2 t[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    raw_unpack2<F32, 4>(r.q[i], t);
    o[2 * i] = t[0];
    o[2 * i + 1] = t[1];
  }
}
template <bool F32>
__device__ __forceinline__ void row_store(typename Elem<F32>::T* dst, const Lane& a, const float2 (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 t[2] = {o[2 * i], o[2 * i + 1]};
    raw_store<F32, 4>(dst + a.o[i], raw_pack2<F32, 4>(t));
  }
}

template <bool F32>
__device__ __forceinline__ void load_weight(const QkParams& p, const void* w, const Lane& a, float2 (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = make_float2(1.f, 1.f);
  if (w != nullptr && a.on && in_range(p.status, a.o[0], 4, p.K, CHK_QK_PARAM) &&
      in_range(p.status, a.o[1], 4, p.K, CHK_QK_PARAM))
    row_unpack<F32>(row_load<F32>(static_cast<const typename Elem<F32>::T*>(w), a), o);
}

// A lane group takes heads g, g + split, ... of one token, queries first, then
// keys, U at a time.
template <bool F32, int LPR>
__global__ void __launch_bounds__(kThreads, F32 ? 2 : 3) qk_fwd_kernel(const QkParams p) {
  using E = typename Elem<F32>::T;
  constexpr int U = 4;  // rows in flight
  const long long gid = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / LPR;
  const long long token = gid / p.split;
  const int g = static_cast<int>(gid - token * p.split);
  Lane a = lane_of<LPR>(p);
  const bool valid = token < p.tokens && a.on;
  const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<long long>(b) * p.T);
  const float inv_k = 1.f / static_cast<float>(p.K);
  const int step = p.split * p.K;
  load_angles<LPR>(p, token, t, valid, a);
  auto heads = [&](const void* src, long long row, int n, const void* weight, void* dst) {
    const E* in = static_cast<const E*>(src) + row + g * p.K;
    E* out = static_cast<E*>(dst) + (token * n + g) * p.K;
    const size_t extent = static_cast<size_t>(p.tokens) * n * p.K;
    const int steps = (n + p.split - 1) / p.split;  // the same for every lane: shuffles below
    RawRow<F32> next[U];
    auto load = [&](int s0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = valid && g + (s0 + u) * p.split < n && in_range(p.status, t, 1, p.T, CHK_QK_IN);
        next[u] = on ? row_load<F32>(in, a) : row_zero<F32>();
        in += step;
      }
    };
    load(0);
    float2 w[4];
    load_weight<F32>(p, weight, a, w);
    for (int s0 = 0; s0 < steps; s0 += U) {
      RawRow<F32> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = next[u];
      if (s0 + U < steps) load(s0 + U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s0 + u >= steps) break;
        float2 x[4];
        row_unpack<F32>(r[u], x);
        const float2 ss = fma2(x[0], x[0], fma2(x[1], x[1], fma2(x[2], x[2], mul2(x[3], x[3]))));
        const float2 rs = both(rsqrtf(fmaf(row_sum<LPR>(ss.x + ss.y), inv_k, p.eps)));
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(x[j], rs), w[j]);
        rotate<1>(p, a, x);
        if (valid && g + (s0 + u) * p.split < n &&
            in_range(p.status, out - static_cast<E*>(dst), p.K, extent, CHK_QK_OUT))
          row_store<F32>(out, a, x);
        out += step;
      }
    }
  };
  heads(p.q, b * p.qb + t * p.qt, p.Nq, p.wq, p.qo);
  if (p.Nk > 0) heads(p.k, b * p.kb + t * p.kt, p.Nk, p.wk, p.ko);
}

// As the forward kernel, with the groups walking over the tokens: a lane
// keeps its features' shares of dwq and dwk in registers throughout.
template <bool F32, bool G32, int LPR>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_kernel(const QkParams p) {
  using E = typename Elem<F32>::T;
  using G = typename Elem<G32>::T;
  let_next_begin();
  constexpr int U = 2, kGroups = kThreads / LPR;
  __shared__ float sums[2][kGroups][8 * LPR + 1];
  const float inv_k = 1.f / static_cast<float>(p.K);
  Lane a = lane_of<LPR>(p);
  float2 wq[4], wk[4], dwq[4], dwk[4];
  load_weight<F32>(p, p.wq, a, wq);
  load_weight<F32>(p, p.wk, a, wk);
#pragma unroll
  for (int j = 0; j < 4; ++j) dwq[j] = dwk[j] = make_float2(0.f, 0.f);
  const long long items = p.tokens * p.split;
  const int step = p.split * p.K;
  // i0: the CTA's first group, the same for all of its warps
  for (long long i0 = static_cast<long long>(blockIdx.x) * kGroups; i0 < items;
       i0 += static_cast<long long>(gridDim.x) * kGroups) {
    const long long item = i0 + threadIdx.x / LPR;
    const long long token = item / p.split;
    const int g = static_cast<int>(item - token * p.split);
    const bool valid = item < items && a.on;
    const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<long long>(b) * p.T);
    load_angles<LPR>(p, token, t, valid, a);
    auto heads = [&](const void* src, long long row, const void* grad, int n, const float2 (&w)[4],
                     float2 (&dw)[4], void* dst) {
      const E* in = static_cast<const E*>(src) + row + g * p.K;
      const size_t first = static_cast<size_t>(token * n + g) * p.K;
      const G* gin = static_cast<const G*>(grad) + first;
      E* out = static_cast<E*>(dst) + first;
      const size_t extent = static_cast<size_t>(p.tokens) * n * p.K;
      const int steps = (n + p.split - 1) / p.split;
      RawRow<F32> nx[U];
      RawRow<G32> ny[U];
      auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool on = valid && g + (s0 + u) * p.split < n && in_range(p.status, t, 1, p.T, CHK_QK_IN) &&
                          in_range(p.status, gin - static_cast<const G*>(grad), p.K, extent, CHK_QK_IN);
          nx[u] = on ? row_load<F32>(in, a) : row_zero<F32>();
          ny[u] = on ? row_load<G32>(gin, a) : row_zero<G32>();
          in += step;
          gin += step;
        }
      };
      load(0);
      for (int s0 = 0; s0 < steps; s0 += U) {
        RawRow<F32> rx[U];
        RawRow<G32> ry[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = nx[u];
          ry[u] = ny[u];
        }
        if (s0 + U < steps) load(s0 + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (s0 + u >= steps) break;
          const bool on = valid && g + (s0 + u) * p.split < n;
          float2 x[4], du[4];
          row_unpack<F32>(rx[u], x);
          row_unpack<G32>(ry[u], du);
          rotate<-1>(p, a, du);
          const float2 ss = fma2(x[0], x[0], fma2(x[1], x[1], fma2(x[2], x[2], mul2(x[3], x[3]))));
          const float2 rs = both(rsqrtf(fmaf(row_sum<LPR>(ss.x + ss.y), inv_k, p.eps)));
          float2 dot = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = mul2(x[j], rs);                   // xh
            if (on) dw[j] = fma2(du[j], x[j], dw[j]);  // a head that is not there has, for eps = 0, xh = NaN
            du[j] = mul2(du[j], w[j]);               // g
            dot = fma2(du[j], x[j], dot);
          }
          // Lanes past the row's end hold zeros, or NaN times zero when eps = 0:
          // they must not enter the row's sum.
          const float2 mean = both(-row_sum<LPR>(a.on ? dot.x + dot.y : 0.f) * inv_k);
#pragma unroll
          for (int j = 0; j < 4; ++j) du[j] = mul2(rs, fma2(x[j], mean, du[j]));
          if (on && in_range(p.status, out - static_cast<E*>(dst), p.K, extent, CHK_QK_OUT))
            row_store<F32>(out, a, du);
          out += step;
        }
      }
    };
    heads(p.q, b * p.qb + t * p.qt, p.dqo, p.Nq, wq, dwq, p.dq);
    if (p.Nk > 0) heads(p.k, b * p.kb + t * p.kt, p.dko, p.Nk, wk, dwk, p.dk);
  }
  if (a.on) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int f = a.o[j / 2] + 2 * (j & 1), grp = threadIdx.x / LPR;
      sums[0][grp][f] = dwq[j].x;
      sums[0][grp][f + 1] = dwq[j].y;
      sums[1][grp][f] = dwk[j].x;
      sums[1][grp][f + 1] = dwk[j].y;
    }
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
// unless that leaves fewer than 1,024 threads for each of 152 SMs.  64 heads of 64:
// B=1 T=1024 9.2 us (one group 19.7, four times as many 10.7), B=8 T=2048 44.6
// (50.7, 51.0).  Ten heads of 128 at T=2048 would like one group: 7.5 instead of 9.1.
int qk_split(const m2rnn_qk_shape* s) {
  const long long tokens = static_cast<long long>(s->B) * s->T;
  const int heads = s->Nq > s->Nk ? s->Nq : s->Nk, lpr = lanes_per_row(s->K);
  if (tokens <= 0) return 1;
  const long long want = (152LL * 1024 / lpr + tokens - 1) / tokens;
  return static_cast<int>(want < 1 ? 1 : want > heads ? heads : want);
}

// CTAs of the gradient kernel: two resident ones for each of 152 SMs, so that the
// groups keep their sums of dw through many tokens.
int qk_bwd_parts(const m2rnn_qk_shape* s) {
  const long long groups = static_cast<long long>(s->B) * s->T * qk_split(s);
  const long long per_cta = kThreads / lanes_per_row(s->K);
  const long long need = (groups + per_cta - 1) / per_cta;
  return static_cast<int>(need < 152 * 2 ? need : 152 * 2);
}

cudaError_t launch_qk_fwd(const QkParams& p, bool f32, cudaStream_t st) {
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

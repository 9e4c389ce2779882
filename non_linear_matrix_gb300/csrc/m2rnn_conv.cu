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
// All three kernels are bound by HBM traffic, with instruction issue close behind
// (the backward kernel takes about 40 for each pair of values).  A thread owns a few
// neighbouring channels and walks along time with the last W rows of F
// (backward: and of dz) in registers, so each value is loaded once apart from the
// W - 1 rows before a thread's run, which its neighbour has just pulled into
// L2; the next rows are loaded while these are worked on.  Neighbouring lanes own
// neighbouring channels: every row is read in whole lines.  Channels are few per
// thread (4 forward, 2 backward) so that 24 warps fit on an SM: with 8 (16-byte
// loads) the forward kernel took 77 us instead of 53 (B=1 T=65536 C=1152, 302 MB:
// 5.7 TB/s), with 4 the backward one 110 us instead of 37 (B=8 T=4096 C=640,
// 126 MB: 3.4 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"
#include "m2rnn_vec.cuh"

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

// sigmoid(z) = 1 / (1 + e^-z); e^-z = inf gives 0.
template <bool F32>
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  if constexpr (F32) {
    return make_float2(1.f / (1.f + expf(-z.x)), 1.f / (1.f + expf(-z.y)));
  } else {  // the approximations' error (about 2^-21) is far below the output's rounding (2^-9)
    const float2 x = mul2(z, both(-1.4426950408889634f));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
    e = add2(e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
  }
}

// Row m of F for channels c0.. of batch item b (m in [0, T + W - 1)).  CONST: see raw_load.
template <bool F32, int VEC, int W, bool CONST = true>
__device__ __forceinline__ Raw<F32, VEC> row_of(const ConvParams& p, int b, long long m, int c0) {
  using E = typename Elem<F32>::T;
  if (m >= W - 1) {
    const long long t = m - (W - 1);
    if (!in_range(p.status, static_cast<size_t>(t), 1, p.T, CHK_CONV_IN) ||
        !in_range(p.status, c0, VEC, p.C, CHK_CONV_IN))
      return raw_zero<F32, VEC>();
    return raw_load<F32, VEC, CONST>(static_cast<const E*>(p.x) + b * p.xb + t * p.xt + c0);
  }
  if (p.state == nullptr) return raw_zero<F32, VEC>();
  const size_t at = (static_cast<size_t>(b) * (W - 1) + m) * p.C + c0;
  if (!in_range(p.status, at, VEC, static_cast<size_t>(p.B) * (W - 1) * p.C, CHK_CONV_IN))
    return raw_zero<F32, VEC>();
  return raw_load<F32, VEC, CONST>(static_cast<const E*>(p.state) + at);
}

// The taps of VEC channels, as pairs of channels for each tap, and their bias.
template <bool F32, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvParams& p, int c0, float2 (&w)[W][VEC / 2],
                                          float2 (&bias)[VEC / 2]) {
  using E = typename Elem<F32>::T;
  float t[VEC * W], bb[VEC];
#pragma unroll
  for (int j = 0; j < VEC * W; ++j) t[j] = 0.f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) bb[j] = 0.f;
  if (in_range(p.status, c0, VEC, p.C, CHK_CONV_PARAM)) {
    const E* src = static_cast<const E*>(p.w) + static_cast<size_t>(c0) * W;
#pragma unroll
    for (int g = 0; g < W; ++g) {  // VEC * W values, VEC at a time
      float x[VEC];
      load_vec<F32, VEC>(src + g * VEC, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) t[g * VEC + e] = x[e];
    }
    if (p.bias != nullptr) load_vec<F32, VEC>(static_cast<const E*>(p.bias) + c0, bb);
  }
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    bias[j] = make_float2(bb[2 * j], bb[2 * j + 1]);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i][j] = make_float2(t[2 * j * W + i], t[(2 * j + 1) * W + i]);
  }
}

// z of a thread's channels from the rows f[0..W-1], in pairs.
template <int VEC, int W>
__device__ __forceinline__ void filter(const float2 (&f)[W][VEC / 2], const float2 (&w)[W][VEC / 2],
                                       const float2 (&bias)[VEC / 2], float2 (&z)[VEC / 2]) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    z[j] = bias[j];
#pragma unroll
    for (int i = 0; i < W; ++i) z[j] = fma2(w[i][j], f[i][j], z[j]);
  }
}
// One thread: VEC channels x TT tokens.
template <bool F32, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, F32 ? 2 : 3) conv_fwd_kernel(const ConvParams p) {
  using E = typename Elem<F32>::T;
  constexpr int U = 4, H = VEC / 2;  // rows in flight per thread
  const int cv = p.C / VEC;
  const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (item >= static_cast<long long>(p.B) * p.nT * cv) return;
  const int c0 = static_cast<int>(item % cv) * VEC;
  const long long run = item / cv;
  const int b = static_cast<int>(run / p.nT);
  const int t0 = static_cast<int>(run - static_cast<long long>(b) * p.nT) * p.TT, t1 = min(p.T, t0 + p.TT);
  float2 w[W][H], bias[H], f[W][H];
  Raw<F32, VEC> next[U], last[W - 1];  // F[t .. t+W-2] as they lie in memory
#pragma unroll
  for (int i = 0; i < W - 1; ++i) last[i] = row_of<F32, VEC, W>(p, b, t0 + i, c0);
  const E* x = static_cast<const E*>(p.x) + b * p.xb + t0 * p.xt + c0;
  const size_t extent = static_cast<size_t>(p.B) * p.T * p.C;
  E* y = static_cast<E*>(p.y) + (static_cast<size_t>(b) * p.T + t0) * p.C + c0;
  auto load = [&](int t) {  // the rows t .. t + U - 1, as far as they are the run's
    if (t + U <= t1 && in_range(p.status, t, U, p.T, CHK_CONV_IN)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        next[u] = raw_load<F32, VEC>(x);
        x += p.xt;
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        next[u] = t + u < t1 && in_range(p.status, t + u, 1, p.T, CHK_CONV_IN) ? raw_load<F32, VEC>(x)
                                                                               : raw_zero<F32, VEC>();
        x += p.xt;
      }
    }
  };
  auto token = [&](const Raw<F32, VEC>& r) {
    raw_unpack2<F32, VEC>(r, f[W - 1]);
    float2 z[H];
    filter<VEC, W>(f, w, bias, z);
    if (SILU) {
#pragma unroll
      for (int j = 0; j < H; ++j) z[j] = mul2(z[j], sigmoid2<F32>(z[j]));
    }
    if (in_range(p.status, y - static_cast<E*>(p.y), VEC, extent, CHK_CONV_OUT))
      raw_store<F32, VEC>(y, raw_pack2<F32, VEC>(z));
    y += p.C;
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
#pragma unroll
      for (int j = 0; j < H; ++j) f[i][j] = f[i + 1][j];
  };
  load(t0);
  load_taps<F32, VEC, W>(p, c0, w, bias);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) raw_unpack2<F32, VEC>(last[i], f[i]);
  int t = t0;
  for (; t + U <= t1; t += U) {
    Raw<F32, VEC> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = next[u];
    load(t + U);
#pragma unroll
    for (int u = 0; u < U; ++u) token(r[u]);
  }
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (t + u < t1) token(next[u]);
  if (t1 == p.T && p.state_out != nullptr) {  // f now holds F's last W - 1 rows
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const size_t sat = (static_cast<size_t>(b) * (W - 1) + i) * p.C + c0;
      if (in_range(p.status, sat, VEC, static_cast<size_t>(p.B) * (W - 1) * p.C, CHK_CONV_OUT))
        raw_store<F32, VEC>(static_cast<E*>(p.state_out) + sat, raw_pack2<F32, VEC>(f[i]));
    }
  }
}

// One thread: 4 channels of one sequence; the state may be updated in place, so it
// is read by plain loads.
template <bool F32, int W, bool SILU>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p) {
  using E = typename Elem<F32>::T;
  constexpr int VEC = 4;
  const int cv = p.C / VEC;
  const long long item = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  if (item >= static_cast<long long>(p.B) * cv) return;
  const int c0 = static_cast<int>(item % cv) * VEC, b = static_cast<int>(item / cv);
  Raw<F32, VEC> r[W];
  float2 f[W][VEC / 2], w[W][VEC / 2], bias[VEC / 2], o[VEC / 2];
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = row_of<F32, VEC, W, false>(p, b, i, c0);
  load_taps<F32, VEC, W>(p, c0, w, bias);
#pragma unroll
  for (int i = 0; i < W; ++i) raw_unpack2<F32, VEC>(r[i], f[i]);
  filter<VEC, W>(f, w, bias, o);
  if (SILU) {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) o[j] = mul2(o[j], sigmoid2<F32>(o[j]));
  }
  const size_t yat = static_cast<size_t>(b) * p.C + c0;
  if (in_range(p.status, yat, VEC, static_cast<size_t>(p.B) * p.C, CHK_CONV_OUT))
    raw_store<F32, VEC>(static_cast<E*>(p.y) + yat, raw_pack2<F32, VEC>(o));
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const size_t at = (static_cast<size_t>(b) * (W - 1) + i) * p.C + c0;
    if (in_range(p.status, at, VEC, static_cast<size_t>(p.B) * (W - 1) * p.C, CHK_CONV_OUT))
      raw_store<F32, VEC>(static_cast<E*>(p.state_out) + at, r[i + 1]);
  }
}

// A warp takes 64 channels (2 per lane) and runs of TT rows of F; a run [m0, m0 +
// TT) writes dF there and adds dz's products for tokens in it.  The eight
// warps' sums are added in warp order, the CTAs' by sum_parts_kernel.
template <bool F32, bool G32, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, F32 ? 2 : 3) conv_bwd_kernel(const ConvParams p) {
  using E = typename Elem<F32>::T;
  using G = typename Elem<G32>::T;
  let_next_begin();
  constexpr int VEC = 2, kWarps = kThreads / 32, U = 4;
  __shared__ float sums[kWarps][32 * VEC * (W + 1)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (blockIdx.x * 32 + lane) * VEC;
  const bool active = c0 < p.C;
  const long long rows = static_cast<long long>(p.T) + W - 1;
  const size_t xn = static_cast<size_t>(p.B) * p.T * p.C;
  const size_t sn = static_cast<size_t>(p.B) * (W - 1) * p.C;
  float2 dw[W], db = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W; ++i) dw[i] = make_float2(0.f, 0.f);
  if (active) {
    float2 w[W][1], bias[1];
    load_taps<F32, VEC, W>(p, c0, w, bias);
    const long long runs = static_cast<long long>(p.B) * p.nT;
    for (long long g = static_cast<long long>(blockIdx.y) * kWarps + warp; g < runs;
         g += static_cast<long long>(gridDim.y) * kWarps) {
      const int b = static_cast<int>(g / p.nT);
      const long long m0 = (g - static_cast<long long>(b) * p.nT) * p.TT;
      const int m1 = static_cast<int>(m0 + p.TT < rows ? m0 + p.TT : rows);
      const int first = static_cast<int>(m0 - (W - 1) > 0 ? m0 - (W - 1) : 0);
      const int tend = min(p.T, m1);  // tokens to be read
      float2 f[W][1], dz[W];          // dz[i]: of token t - (W-1) + i
#pragma unroll
      for (int i = 0; i < W; ++i) f[i][0] = dz[i] = make_float2(0.f, 0.f);
      const E* x = static_cast<const E*>(p.x) + b * p.xb + first * p.xt + c0;
      const G* dy = static_cast<const G*>(p.dy) + (static_cast<size_t>(b) * p.T + first) * p.C + c0;
      E* dx = static_cast<E*>(p.dx) + (static_cast<size_t>(b) * p.T + first) * p.C + c0;  // row m - (W-1)
      dx -= static_cast<size_t>(W - 1) * p.C;
      Raw<F32, VEC> nx[U];
      Raw<G32, VEC> ng[U];
      auto load = [&](int t) {  // tokens t .. t + U - 1, as far as they are to be read
        if (t + U <= tend && in_range(p.status, t, U, p.T, CHK_CONV_IN)) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            nx[u] = raw_load<F32, VEC>(x);
            ng[u] = raw_load<G32, VEC>(dy);
            x += p.xt;
            dy += p.C;
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const bool on = t + u < tend && in_range(p.status, t + u, 1, p.T, CHK_CONV_IN);
            nx[u] = on ? raw_load<F32, VEC>(x) : raw_zero<F32, VEC>();
            ng[u] = on ? raw_load<G32, VEC>(dy) : raw_zero<G32, VEC>();
            x += p.xt;
            dy += p.C;
          }
        }
      };
      // dz of the next token into dz[W - 1], its row into f[W - 1]
      auto enter = [&](const Raw<F32, VEC>& rx, const Raw<G32, VEC>& rg) {
        float2 gy[1];
        raw_unpack2<F32, VEC>(rx, f[W - 1]);
        raw_unpack2<G32, VEC>(rg, gy);
        dz[W - 1] = gy[0];
        if (SILU) {
          float2 z[1];
          filter<VEC, W>(f, w, bias, z);
          const float2 s = sigmoid2<F32>(z[0]);
          // s (1 + z (1 - s)); at z = +-inf the inner product is 0 times inf: NaN, as in the formula
          const float2 q = fma2(z[0], fma2(s, both(-1.f), both(1.f)), both(1.f));
          dz[W - 1] = mul2(gy[0], mul2(s, q));
        }
      };
      auto products = [&](float2 (&o)[1]) {
        o[0] = mul2(w[0][0], dz[W - 1]);
        dw[0] = fma2(dz[W - 1], f[0][0], dw[0]);
#pragma unroll
        for (int i = 1; i < W; ++i) {
          o[0] = fma2(w[i][0], dz[W - 1 - i], o[0]);
          dw[i] = fma2(dz[W - 1], f[i][0], dw[i]);
        }
        db = add2(db, dz[W - 1]);
      };
      auto leave = [&]() {
        dx += p.C;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          f[i][0] = f[i + 1][0];
          dz[i] = dz[i + 1];
        }
      };
      // any token of the run, its edges among them
      auto token = [&](int m, const Raw<F32, VEC>& rx, const Raw<G32, VEC>& rg) {
        enter(rx, rg);
        if (m >= p.T) dz[W - 1] = make_float2(0.f, 0.f);
        if (m >= m0) {
          float2 o[1];
          products(o);
          if (m >= p.T && p.dstate_out != nullptr) {
            const size_t at = (static_cast<size_t>(b) * (W - 1) + (m - p.T)) * p.C + c0;
            float2 ds[1];
            if (in_range(p.status, at, VEC, sn, CHK_CONV_IN)) {
              raw_unpack2<F32, VEC>(raw_load<F32, VEC>(static_cast<const E*>(p.dstate_out) + at), ds);
              o[0] = add2(o[0], ds[0]);
            }
          }
          if (m >= W - 1) {
            if (in_range(p.status, dx - static_cast<E*>(p.dx), VEC, xn, CHK_CONV_OUT))
              raw_store<F32, VEC>(dx, raw_pack2<F32, VEC>(o));
          } else if (p.dstate != nullptr) {
            const size_t at = (static_cast<size_t>(b) * (W - 1) + m) * p.C + c0;
            if (in_range(p.status, at, VEC, sn, CHK_CONV_OUT))
              raw_store<F32, VEC>(static_cast<E*>(p.dstate) + at, raw_pack2<F32, VEC>(o));
          }
        }
        leave();
      };
      load(first);
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
        if (first + i < rows)
          raw_unpack2<F32, VEC>(row_of<F32, VEC, W>(p, b, first + i, c0), f[i]);
      const int inner = m0 > W - 1 ? static_cast<int>(m0) : W - 1;  // from here to tend: no edge
      for (int t = first; t < m1; t += U) {
        Raw<F32, VEC> rx[U];
        Raw<G32, VEC> rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = nx[u];
          rg[u] = ng[u];
        }
        load(t + U);
        if (t >= inner && t + U <= tend) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float2 o[1];
            enter(rx[u], rg[u]);
            products(o);
            if (in_range(p.status, dx - static_cast<E*>(p.dx), VEC, xn, CHK_CONV_OUT))
              raw_store<F32, VEC>(dx, raw_pack2<F32, VEC>(o));
            leave();
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (t + u < m1) token(t + u, rx[u], rg[u]);
        }
      }
    }
  }
  // the part's layout: dw [C][W], then dbias [C]
#pragma unroll
  for (int i = 0; i < W; ++i) {
    sums[warp][lane * VEC * W + i] = dw[i].x;
    sums[warp][(lane * VEC + 1) * W + i] = dw[i].y;
  }
  sums[warp][32 * VEC * W + lane * VEC] = db.x;
  sums[warp][32 * VEC * W + lane * VEC + 1] = db.y;
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
  constexpr int VEC = 4;
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
  const dim3 grid((p.C + 63) / 64, p.nparts);
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
// 2,048 threads for each SM, 4 tokens at least.  B=8 T=4096 C=640: 17.2 us, asking
// for 8,192 26.7, for 512 16.4; T=2048 C=640: 4.7 (4.7, 4.8).
int conv_fwd_tokens(const m2rnn_conv_shape* s, int sms) {
  const long long per_token = static_cast<long long>(s->B) * (s->C / 4);
  int tt = 32;
  while (tt > 4 && per_token * ((s->T + tt - 1) / tt) < 2048LL * sms) tt /= 2;
  return tt;
}

// CTAs of eight warps for 64 channels each, as many as are resident (456: three
// for each of 152 SMs) and no more, so that they end together and the parts
// stay few; the sequences are cut so that each warp has one run, 8 rows at
// least.  B=8 T=4096 C=640: 37 us, with 228 CTAs 57, with 912 41.
void conv_bwd_plan(const m2rnn_conv_shape* s, int* TT, int* nT, int* nparts) {
  const long long rows = static_cast<long long>(s->T) + s->W - 1;
  const long long groups = (s->C + 63) / 64;
  const long long parts = 456 / groups > 1 ? 456 / groups : 1;
  long long per_item = parts * 8 / s->B;  // runs of a sequence
  if (per_item < 1) per_item = 1;
  long long tt = (rows + per_item - 1) / per_item;
  if (tt < 8) tt = 8;
  *TT = static_cast<int>(tt);
  *nT = static_cast<int>((rows + tt - 1) / tt);
  const long long need = (static_cast<long long>(s->B) * *nT + 7) / 8;
  *nparts = static_cast<int>(need < parts ? need : parts);
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

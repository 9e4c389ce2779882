// m2rnn_scan_step.cu -- one token of the selective scan for many sequences,
// the state carried in HBM between calls:
//
//     dt = softplus(a + beta),  H' = exp(-alpha dt) H + dt k v^T,  y = H'^T q + w_r (.) v
//
// A step reads and writes the whole fp32 state (2 K V 4 bytes per head)
// against a few hundred bytes of inputs: bound by HBM traffic.  A warp owns a
// head; a lane owns 4 neighbouring columns of every (128 / V)-th row, so the
// state moves in 16-byte accesses over whole lines, each element once, and
// the readout's sum over rows ends in a few shuffles within the warp.  2048
// sequences of 32 heads of 64 x 16 (542 MB) take 87 us: 6.2 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"
#include "m2rnn_gate.cuh"
#include "m2rnn_vec.cuh"

namespace m2rnn {
namespace {

constexpr int kWarps = 4;

template <int V, bool F32>
__global__ void __launch_bounds__(32 * kWarps) scan_step_kernel(const ScanStepParams p) {
  using E = typename Elem<F32>::T;
  constexpr int LPC = V / 4;       // lanes per row
  constexpr int RPP = 32 / LPC;    // rows per pass of the warp
  constexpr int U = 8;             // rows in flight per lane
  const long long head = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (head >= static_cast<long long>(p.B) * p.N) return;
  const int lane = threadIdx.x & 31, row0 = lane / LPC, col = (lane % LPC) * 4;
  const int b = static_cast<int>(head / p.N), n = static_cast<int>(head % p.N);
  const int group = n / (p.N / p.Nq);
  const size_t base = static_cast<size_t>(head) * p.K * V;
  const size_t extent = static_cast<size_t>(p.B) * p.N * p.K * V;
  if (!in_range(p.status, b, 1, p.B, CHK_SCAN_IN) || !in_range(p.status, group, 1, p.Nq, CHK_SCAN_IN))
    return;
  const E* q = static_cast<const E*>(p.q) + b * p.qb + static_cast<size_t>(group) * p.K;
  const E* k = static_cast<const E*>(p.k) + b * p.kb + static_cast<size_t>(group) * p.K;
  const E* vp = static_cast<const E*>(p.v) + b * p.vb + static_cast<size_t>(n) * V + col;
  float v[4], y[4] = {0.f, 0.f, 0.f, 0.f}, f = 0.f, dt = 0.f;
  for (int r0 = row0; r0 < p.K; r0 += RPP * U) {
    float4 h[U];
    float kk[U], qq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      h[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      kk[u] = qq[u] = 0.f;
      if (r < p.K && in_range(p.status, base + static_cast<size_t>(r) * V + col, 4, extent,
                              CHK_SCAN_STATE)) {
        h[u] = *reinterpret_cast<const float4*>(p.H_in + base + static_cast<size_t>(r) * V + col);
        kk[u] = to_f32(k[r]);
        qq[u] = to_f32(q[r]);
      }
    }
    if (r0 == row0) {  // the gate, while the first rows of the state are on their way
      load_vec<F32, 4>(vp, v);
      dt = gate_softplus(to_f32(static_cast<const E*>(p.a)[b * p.ab + n]) +
                         to_f32(static_cast<const E*>(p.beta)[n]));
      f = expf(-to_f32(static_cast<const E*>(p.alpha)[n]) * dt);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      if (r >= p.K) break;
      const float kd = kk[u] * dt;
      h[u].x = fmaf(f, h[u].x, kd * v[0]);
      h[u].y = fmaf(f, h[u].y, kd * v[1]);
      h[u].z = fmaf(f, h[u].z, kd * v[2]);
      h[u].w = fmaf(f, h[u].w, kd * v[3]);
      y[0] = fmaf(qq[u], h[u].x, y[0]);
      y[1] = fmaf(qq[u], h[u].y, y[1]);
      y[2] = fmaf(qq[u], h[u].z, y[2]);
      y[3] = fmaf(qq[u], h[u].w, y[3]);
      if (in_range(p.status, base + static_cast<size_t>(r) * V + col, 4, extent, CHK_SCAN_STATE))
        *reinterpret_cast<float4*>(p.H_out + base + static_cast<size_t>(r) * V + col) = h[u];
    }
  }
#pragma unroll
  for (int m = LPC; m < 32; m *= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += __shfl_xor_sync(0xffffffffu, y[j], m);
  if (row0 != 0) return;
  if (p.w_r != nullptr) {
    float w[4];
    load_vec<F32, 4>(static_cast<const E*>(p.w_r) + static_cast<size_t>(n) * V + col, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(w[j], v[j], y[j]);
  }
  const size_t at = static_cast<size_t>(head) * V + col;
  if (in_range(p.status, at, 4, static_cast<size_t>(p.B) * p.N * V, CHK_SCAN_OUT))
    store_vec<F32, 4>(static_cast<E*>(p.y) + at, y);
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepParams& p, int V, bool f32, cudaStream_t st) {
  const long long heads = static_cast<long long>(p.B) * p.N;
  const unsigned grid = static_cast<unsigned>((heads + kWarps - 1) / kWarps);
  if (V == 16) {
    if (f32)
      scan_step_kernel<16, true><<<grid, 32 * kWarps, 0, st>>>(p);
    else
      scan_step_kernel<16, false><<<grid, 32 * kWarps, 0, st>>>(p);
  } else {
    if (f32)
      scan_step_kernel<32, true><<<grid, 32 * kWarps, 0, st>>>(p);
    else
      scan_step_kernel<32, false><<<grid, 32 * kWarps, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace m2rnn

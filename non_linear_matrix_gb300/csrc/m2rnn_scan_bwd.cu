// m2rnn_scan_bwd.cu -- the scan's backward pass after the states: the chunk
// kernels (m2rnn_scan_bwd.cuh), then the sums over what several CTAs share,
// in a fixed order.
#include "m2rnn_scan.cuh"

namespace m2rnn {

cudaError_t launch_scan_bwd_bf16_lo(const ScanParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_bf16_hi(const ScanParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_f32_lo(const ScanParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd_f32_hi(const ScanParams& p, cudaStream_t st);

namespace {

// dq and dk from their shares; a thread sums 4 neighbouring values.
template <bool F32>
__global__ void __launch_bounds__(256) add_shares_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  let_next_begin();
  await_before();
  const size_t n = static_cast<size_t>(p.B) * p.T * p.Nq * p.K;
  const size_t at = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= 2 * n) return;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int h = 0; h < p.hsplit; ++h) {
    const size_t from = h * 2 * n + at;
    if (!in_range(p.status, from, 4, p.hsplit * 2 * n, CHK_SCAN_WS)) return;
    const float4 x = *reinterpret_cast<const float4*>(p.dqk + from);
    s[0] += x.x;
    s[1] += x.y;
    s[2] += x.z;
    s[3] += x.w;
  }
  store_vec<F32, 4>(at < n ? static_cast<E*>(p.dq) + at : static_cast<E*>(p.dk) + (at - n), s);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanParams& p, bool f32, cudaStream_t st) {
  cudaError_t e;
  if (f32)
    e = p.K <= 32 ? launch_scan_bwd_f32_lo(p, st) : launch_scan_bwd_f32_hi(p, st);
  else
    e = p.K <= 32 ? launch_scan_bwd_bf16_lo(p, st) : launch_scan_bwd_bf16_hi(p, st);
  if (e != cudaSuccess) return e;
  if (p.hsplit > 1) {
    const size_t n4 = static_cast<size_t>(p.B) * p.T * p.Nq * p.K / 2;  // 2 n / 4
    const dim3 grid(static_cast<unsigned>((n4 + 255) / 256));
    e = f32 ? launch_after(add_shares_kernel<true>, grid, 256, 0, st, p)
            : launch_after(add_shares_kernel<false>, grid, 256, 0, st, p);
    if (e != cudaSuccess) return e;
  }
  const SumOut o{{p.dalpha, p.dbeta, p.dw_r}, {p.N, p.N, p.N * p.V}};
  return launch_sum_parts(p.part, p.B * p.nc, o, p.status, CHK_SCAN_PARAM, st);
}

}  // namespace m2rnn

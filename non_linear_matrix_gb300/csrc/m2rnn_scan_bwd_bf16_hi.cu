// m2rnn_scan_bwd_bf16_hi.cu -- the scan's gradient kernels for bf16 inputs and
// K = 64 or 128 (compiled apart: the build runs them in parallel).
#include "m2rnn_scan_bwd.cuh"

namespace m2rnn {

cudaError_t launch_scan_bwd_bf16_hi(const ScanParams& p, cudaStream_t st) {
  if (p.K == 64)
    return p.V == 16 ? scan::launch_bwd_kt<false, 8, 16>(p, st) : scan::launch_bwd_kt<false, 8, 32>(p, st);
  return p.V == 16 ? scan::launch_bwd_kt<false, 16, 16>(p, st) : scan::launch_bwd_kt<false, 16, 32>(p, st);
}

}  // namespace m2rnn

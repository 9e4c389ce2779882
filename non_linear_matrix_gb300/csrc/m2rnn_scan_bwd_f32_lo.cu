// m2rnn_scan_bwd_f32_lo.cu -- the scan's gradient kernels for f32 inputs and
// K = 16 or 32 (compiled apart: the build runs them in parallel).
#include "m2rnn_scan_bwd.cuh"

namespace m2rnn {

cudaError_t launch_scan_bwd_f32_lo(const ScanParams& p, cudaStream_t st) {
  if (p.K == 16)
    return p.V == 16 ? scan::launch_bwd_kt<true, 2, 16>(p, st) : scan::launch_bwd_kt<true, 2, 32>(p, st);
  return p.V == 16 ? scan::launch_bwd_kt<true, 4, 16>(p, st) : scan::launch_bwd_kt<true, 4, 32>(p, st);
}

}  // namespace m2rnn

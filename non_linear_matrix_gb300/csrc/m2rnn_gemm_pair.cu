// m2rnn_gemm_pair.cu -- instances of the product kernel: gated products and the
// 8-bit ones.
#include "m2rnn_gemm.cuh"

namespace m2rnn {

cudaError_t launch_gemm_grad(const GemmParams& p, const GemmKind& k, int sms, cudaStream_t st);

cudaError_t launch_gemm(const GemmParams& p, const GemmKind& k, int sms, cudaStream_t st) {
  switch (k.epi) {
    case EPI_GLU:
      if (k.f32) return launch_cfg<GemmCfg<EPI_GLU, false, true, false, false, 128, 1>>(p, sms, st);
      return k.bn == 256 ? launch_cfg<GemmCfg<EPI_GLU, false, false, false, false, 256, 2>>(p, sms, st)
                         : launch_cfg<GemmCfg<EPI_GLU, false, false, false, false, 128, 1>>(p, sms, st);
    case EPI_GLU8:
      return k.bn == 256 ? launch_cfg<GemmCfg<EPI_GLU8, true, false, false, false, 256, 2>>(p, sms, st)
                         : launch_cfg<GemmCfg<EPI_GLU8, true, false, false, false, 128, 1>>(p, sms, st);
    case EPI_LIN8:
      return k.bn == 256 ? launch_cfg<GemmCfg<EPI_LIN8, true, false, false, false, 256, 2>>(p, sms, st)
                         : launch_cfg<GemmCfg<EPI_LIN8, true, false, false, false, 128, 1>>(p, sms, st);
    default:
      return launch_gemm_grad(p, k, sms, st);
  }
}

// Accumulator columns of a tile: 256, by a pair of CTAs over 256 rows, where there are
// as many tiles as pairs; otherwise 128, by a CTA over 128 rows.  fp32: 128, whose sums fit
// the registers.
int gemm_bn(int epi, bool f32, long long m, int n, int nbatch, int sms) {
  if (f32) return 128;
  const bool pair = epi == EPI_GLU || epi == EPI_DGLU || epi == EPI_GLU8;
  const int cols = pair ? 128 : 256;
  const long long tiles = (m + 255) / 256 * ((n + cols - 1) / cols) * nbatch;
  return 2 * tiles >= sms ? 256 : 128;
}

}  // namespace m2rnn

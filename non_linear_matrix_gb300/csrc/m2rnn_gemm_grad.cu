// m2rnn_gemm_grad.cu -- instances of the product kernel for the gated products'
// gradients.
#include "m2rnn_gemm.cuh"

namespace m2rnn {

cudaError_t launch_gemm_grad(const GemmParams& p, const GemmKind& k, int sms, cudaStream_t st) {
  if (k.epi == EPI_DGLU) {
    if (k.f32) return launch_cfg<GemmCfg<EPI_DGLU, false, true, false, false, 128, 1>>(p, sms, st);
    return k.bn == 256 ? launch_cfg<GemmCfg<EPI_DGLU, false, false, false, false, 256, 2>>(p, sms, st)
                       : launch_cfg<GemmCfg<EPI_DGLU, false, false, false, false, 128, 1>>(p, sms, st);
  }
  if (!k.a_mn) {  // dx
    if (k.f32)
      return k.rows == 256 ? launch_cfg<GemmCfg<EPI_STORE, false, true, false, true, 128, 2>>(p, sms, st)
                           : launch_cfg<GemmCfg<EPI_STORE, false, true, false, true, 128, 1>>(p, sms, st);
    return k.bn == 256 ? launch_cfg<GemmCfg<EPI_STORE, false, false, false, true, 256, 2>>(p, sms, st)
                       : launch_cfg<GemmCfg<EPI_STORE, false, false, false, true, 128, 1>>(p, sms, st);
  }
  if (k.f32)
      return k.rows == 256 ? launch_cfg<GemmCfg<EPI_STORE, false, true, true, true, 128, 2>>(p, sms, st)
                           : launch_cfg<GemmCfg<EPI_STORE, false, true, true, true, 128, 1>>(p, sms, st);
  return k.bn == 256 ? launch_cfg<GemmCfg<EPI_STORE, false, false, true, true, 256, 2>>(p, sms, st)
                     : launch_cfg<GemmCfg<EPI_STORE, false, false, true, true, 128, 1>>(p, sms, st);
}

}  // namespace m2rnn

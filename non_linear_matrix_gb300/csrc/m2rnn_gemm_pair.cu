// m2rnn_gemm_pair.cu -- instances of the product kernel: gated products and the
// 8-bit ones.
#include "m2rnn_gemm.cuh"

namespace m2rnn {

cudaError_t launch_gemm_grad(const GemmParams& p, const GemmKind& k, int sms, cudaStream_t st);

cudaError_t launch_gemm(const GemmParams& p, const GemmKind& k, int sms, cudaStream_t st) {
  switch (k.epi) {
    case EPI_GLU:
      if (k.f32)
        return k.rows == 256 ? launch_cfg<GemmCfg<EPI_GLU, false, true, false, false, 128, 2>>(p, sms, st)
                             : launch_cfg<GemmCfg<EPI_GLU, false, true, false, false, 128, 1>>(p, sms, st);
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

// Tiles of 256 x 256 by a pair of CTAs where there are as many as pairs (76, two to each of
// 152 SMs); otherwise 128 x 128 by a CTA.  fp32: 256 x 128 by a pair, whose
// terms and sums fit, or 128 x 128 by a CTA, which takes a fifth longer for its tile (shared memory
// feeds the products), where that makes fewer waves, and for the gradients of g and u, whose six
// planes then find room to pass through shared memory (backward pass M=8192 D=512 F=2048 432
// -> 408 us, M=4096 D=2048 F=4096 equal).
// The tiles beyond whole waves are cut along K into as many parts as leave every pair or
// CTA one, each of 16 K tiles (fp32, whose K tiles are six products: 4) at least, and not where
// the whole is shorter than three of those: joining the parts takes 2 us and a launch of the
// host's, 16 K tiles 2 to 4.  With bf16 operands all tiles are cut where one chain of
// sums over all segments would be longer than 512 K tiles (16,384 tokens in a weight's gradient,
// 32,768 with one term): each of its four steps
// per K tile cuts the sum off, by up to 3.1 2^-24 of it (measured, terms of one sign), so that a
// chain loses at most 2^-12.3 of its sum.  So are they with fp32 operands (unless few tiles are cut into more
// parts anyway): there 512 K tiles are 128 chunks, whose sums are rounded as they are added one
// after the other, and the roundings of longer runs show (weights' gradients over a million
// tokens 1.26e-6 instead of 8e-7).  The gated products themselves are cut only in fp32 and where
// the tiles are at most half as many as run at once: their parts want g and u in memory (M=169
// D=1888 F=136 36 -> 23 us forward, 72 -> 49 backward); their longest run is D = 2^16, 256 chunks.
GemmPlan gemm_plan(int epi, bool f32, long long m, int n, int nbatch, int nseg, int kt) {
  constexpr int kSms = 152;
  const bool pair = epi == EPI_GLU || epi == EPI_DGLU || epi == EPI_GLU8;
  GemmPlan q{};
  const auto tiles = [&](int rows, int bn) {
    const int cols = pair ? bn / 2 : bn;
    q.bn = bn;
    q.rows = rows;
    q.mt = static_cast<int>((m + rows - 1) / rows);
    q.nt = (n + cols - 1) / cols;
    q.nbatch = nbatch;
    return q.mt * q.nt * nbatch;
  };
  int count, at_once = kSms / 2;
  if (f32) {
    const int singles = tiles(128, 128), waves = (singles + kSms - 1) / kSms;
    count = tiles(256, 128);
    if (epi == EPI_DGLU || 5 * waves < 4 * ((count + at_once - 1) / at_once)) {
      count = tiles(128, 128);
      at_once = kSms;
    }
  } else if ((count = tiles(256, 256)) < at_once) {
    count = tiles(128, 128);
    at_once = kSms;
  }
  q.whole = count;
  q.split = 1;
  if (epi != EPI_STORE && !(f32 && 2 * count <= at_once)) return q;
  constexpr long long kChain = 512;
  const long long chain = static_cast<long long>(nseg) * kt;
  const int rest = count % at_once, least = f32 ? 4 : 16;  // (K tiles of a part)
  int split = rest == 0 || chain < 3 * least ? 1 : at_once / rest;
  if (split > chain / least) split = static_cast<int>(chain / least);
  if (split > kt) split = kt;
  const int need = static_cast<int>((chain + kChain - 1) / kChain);
  if (need > 1 && !(f32 && rest == count && split >= need)) {
    q.whole = 0;
    q.split = need;
    q.nparts = count * q.split;
    q.parts_bytes = static_cast<size_t>(q.nparts) * q.rows * q.bn * sizeof(float);
    return q;
  }
  if (split < 2) return q;
  q.whole = count - rest;
  q.split = split;
  q.nparts = rest * split;
  q.parts_bytes = static_cast<size_t>(q.nparts) * q.rows * q.bn * sizeof(float);
  return q;
}

}  // namespace m2rnn

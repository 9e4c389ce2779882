// m2rnn_scan_out.cu -- the outputs of the selective scan, chunk by chunk, from
// the states before the chunks:
//
//     y_i = 2^S(start,i) H^T q_i + sum_{j<=i} (q_i.k_j) 2^S(j,i) dt_j v_j + w_r (.) v_i
//
// A CTA takes one chunk of one query/key group: q k^T (64 x 64, fp32) is
// formed once, a warp keeping its 16 rows in registers for all heads; then the
// head blocks pass by, each bringing its v tile and state.  For each head
// the weights are made in registers from q k^T, in the layout that the next
// product takes as its A operand.  Warp w of CTA x works on rows 16 ((w + x)
// mod 4)..: the row blocks differ in causal work, and a warp's place decides
// which quarter of the SM it runs on.
#include "m2rnn_scan.cuh"

namespace m2rnn {
namespace scan {
namespace {

template <bool F32>
int out_smem_bytes(int K) {
  constexpr int P = Terms<F32>::in, PS = Terms<F32>::state;
  return 2 * P * kChunk * (K + 8) * 2 + P * kChunk * kVLd * 2 + PS * kCols * K * 2 +
         (F32 ? 0 : kChunk * kVLd * 2) + 3 * 4 * kChunk * 4;
}

template <bool F32, int V>
__global__ void __launch_bounds__(kThreads) out_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  constexpr int P = Terms<F32>::in, PS = Terms<F32>::state, PW = Terms<F32>::prob;
  constexpr int HB = kCols / V, NT = V / 8;  // heads per block, column tiles per head
  extern __shared__ __align__(128) unsigned char smem[];
  const int K = p.K, ld = K + 8;
  const uint32_t qs = ptx::smem_addr(smem), ks_ = qs + P * kChunk * ld * 2,
                 vs = ks_ + P * kChunk * ld * 2, hs = vs + P * kChunk * kVLd * 2,
                 ys = hs + PS * kCols * K * 2;
  // per head: sum of l from the 16-block's start to the token; the same less
  // log2 dt (bf16) or as it is (fp32); dt
  float* loc = reinterpret_cast<float*>(smem + (ys - qs) + (F32 ? 0 : kChunk * kVLd * 2));
  float* locj = loc + HB * kChunk;
  float* dts = locj + HB * kChunk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
  const int rt = (warp + blockIdx.x) & 3;  // the warp's 16 rows
  const int c = blockIdx.x % p.nc;
  const int rest = blockIdx.x / p.nc, part = rest % p.hsplit;
  const int group = (rest / p.hsplit) % p.Nq, b = rest / p.hsplit / p.Nq;
  const int t0 = c * kChunk, rows = min(kChunk, p.T - t0);
  const int per = (p.nhb + p.hsplit - 1) / p.hsplit;
  const int hb0 = part * per, hb1 = min(p.nhb, hb0 + per);
  if (hb0 >= hb1) return;
  const E* q = static_cast<const E*>(p.q) + b * p.qb + t0 * p.qt + static_cast<size_t>(group) * K;
  const E* k = static_cast<const E*>(p.k) + b * p.kb + t0 * p.kt + static_cast<size_t>(group) * K;
  load_tile<F32>(qs, q, p.qt, rows, K, K, ld, p.status, p.T - t0);
  load_tile<F32>(ks_, k, p.kt, rows, K, K, ld, p.status, p.T - t0);
  ptx::cp_async_commit();

  const size_t sd_extent = static_cast<size_t>(p.B) * p.N * p.nc * kChunk;
  const size_t hs_extent = state_at(p, PS, p.B, 0, 0);
  auto fetch = [&](int hb) {
    const Place w = place_of(p, b, group * p.nhb + hb);
    const E* v = static_cast<const E*>(p.v) + b * p.vb + t0 * p.vt + static_cast<size_t>(w.head0) * V;
    load_tile<F32>(vs, v, p.vt, rows, w.heads * V, kCols, kVLd, p.status, p.T - t0);
    const size_t at = state_at(p, PS, b, group * p.nhb + hb, c);
    if (in_range(p.status, at, PS * kCols * K, hs_extent, CHK_SCAN_WS))
      load_linear(hs, p.Hs + at, PS * kCols * K * 2);
    ptx::cp_async_commit();
    for (int e = threadIdx.x; e < w.heads * kChunk; e += kThreads) {
      const size_t sat = (static_cast<size_t>(b) * p.N + w.head0 + e / kChunk) * p.nc * kChunk + t0 + e % kChunk;
      float2 s = make_float2(0.f, 0.f);
      if (in_range(p.status, sat, 1, sd_extent, CHK_SCAN_WS)) s = p.sd[sat];
      loc[e] = s.x;
      locj[e] = F32 ? s.x : s.x - log2f(s.y);  // dt = 0: +inf, a weight of 0
      if (F32) dts[e] = s.y;
    }
  };
  fetch(hb0);
  cp_async_wait<1>();
  __syncthreads();

  float gm[8][4];  // q k^T: rows 16 rt + g [+8], column tile nt
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) gm[nt][i] = 0.f;
  for (int kk = 0; kk < K / 16; ++kk) {
    uint32_t a[P][4];
    load_a<P>(a, qs, ld, 16 * rt, 16 * kk);
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      if (jb > rt) break;
      uint32_t b0[P][2], b1[P][2];
      load_b2<P>(b0, b1, ks_, ld, 16 * jb, 16 * kk);
      mma_terms<P, P>(gm[2 * jb], a, b0);
      mma_terms<P, P>(gm[2 * jb + 1], a, b1);
    }
  }

  const E* w_r = static_cast<const E*>(p.w_r);
  E* y = static_cast<E*>(p.y);
  const size_t y_extent = static_cast<size_t>(p.B) * p.T * p.N * V;
  for (int hb = hb0; hb < hb1; ++hb) {
    const Place w = place_of(p, b, group * p.nhb + hb);
    cp_async_wait<0>();
    __syncthreads();
    float acc[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    // from the state: q H
    for (int kk = 0; kk < K / 16; ++kk) {
      uint32_t a[P][4];
      load_a<P>(a, qs, ld, 16 * rt, 16 * kk);
#pragma unroll
      for (int v8 = 0; v8 < 8; v8 += 2) {
        if (v8 >= w.heads * NT) break;
        uint32_t b0[PS][2], b1[PS][2];
        state_b2<PS>(b0, b1, hs, K, v8, kk);
        mma_terms<P, PS>(acc[v8], a, b0);
        mma_terms<P, PS>(acc[v8 + 1], a, b1);
      }
    }
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      if (h >= w.heads) break;
      const float* lo = loc + h * kChunk;
      const float* lj = locj + h * kChunk;
      const float li0 = lo[16 * rt + g], li1 = lo[16 * rt + g + 8];
      {  // decay since the chunk's start
        float off = 0.f;
#pragma unroll
        for (int k4 = 0; k4 < 3; ++k4) off += k4 < rt ? lo[16 * k4 + 15] : 0.f;
        const float e0 = ex2(off + li0), e1 = ex2(off + li1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[h * NT + nt][0] *= e0;
          acc[h * NT + nt][1] *= e0;
          acc[h * NT + nt][2] *= e1;
          acc[h * NT + nt][3] *= e1;
        }
      }
      // within the chunk; s0, s1: sum of l from the start of j's block to i
      float s0 = li0, s1 = li1;
#pragma unroll
      for (int jj = 3; jj >= 0; --jj) {
        if (jj > rt) continue;
        if (jj < rt) {
          s0 += lo[16 * jj + 15];
          s1 += lo[16 * jj + 15];
        }
        uint32_t a[PW][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int nt = 2 * jj + u;
          const float2 s = *reinterpret_cast<const float2*>(lj + 8 * nt + c2);
          float m0 = gm[nt][0] * ex2(s0 - s.x), m1 = gm[nt][1] * ex2(s0 - s.y);
          float m2 = gm[nt][2] * ex2(s1 - s.x), m3 = gm[nt][3] * ex2(s1 - s.y);
          if (F32) {
            const float2 d = *reinterpret_cast<const float2*>(dts + h * kChunk + 8 * nt + c2);
            m0 *= d.x; m1 *= d.y; m2 *= d.x; m3 *= d.y;
          }
          if (jj == rt) {  // j <= i
            const int j = 8 * u + c2;
            m0 = j <= g ? m0 : 0.f;
            m1 = j + 1 <= g ? m1 : 0.f;
            m2 = j <= g + 8 ? m2 : 0.f;
            m3 = j + 1 <= g + 8 ? m3 : 0.f;
          }
          uint32_t t0_[PW], t1_[PW];
          split<PW>(m0, m1, t0_);
          split<PW>(m2, m3, t1_);
#pragma unroll
          for (int s2 = 0; s2 < PW; ++s2) {
            a[s2][2 * u] = t0_[s2];
            a[s2][2 * u + 1] = t1_[s2];
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
          uint32_t b0[P][2], b1[P][2];
          load_b2_t<P>(b0, b1, vs, kVLd, 16 * jj, h * V + 8 * nt);
          mma_terms<PW, P>(acc[h * NT + nt], a, b0);
          mma_terms<PW, P>(acc[h * NT + nt + 1], a, b1);
        }
      }
    }
    // + w_r (.) v, and out
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt >= w.heads * NT) break;
      float2 wr = make_float2(0.f, 0.f);
      if (w_r != nullptr) {
        const E* src = w_r + static_cast<size_t>(w.head0) * V + 8 * nt + c2;
        wr = make_float2(to_f32(src[0]), to_f32(src[1]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * rt + g + 8 * h;
        uint32_t x[P];
#pragma unroll
        for (int s = 0; s < P; ++s)
          x[s] = ptx::lds_u32(vs + s * kChunk * kVLd * 2 + (r * kVLd + 8 * nt + c2) * 2);
        const float2 v = join<P>(x);
        const float y0 = fmaf(wr.x, v.x, acc[nt][2 * h]), y1 = fmaf(wr.y, v.y, acc[nt][2 * h + 1]);
        if constexpr (F32) {
          const size_t at = ((static_cast<size_t>(b) * p.T + t0 + r) * p.N + w.head0) * V + 8 * nt + c2;
          if (r < rows && in_range(p.status, at, 2, y_extent, CHK_SCAN_OUT))
            *reinterpret_cast<float2*>(y + at) = make_float2(y0, y1);
        } else {
          ptx::sts_u32(ys + (r * kVLd + 8 * nt + c2) * 2, ptx::pack_bf16x2(y0, y1));
        }
      }
    }
    if constexpr (!F32) {
      __syncwarp();  // the warp's own 16 rows, in 16-byte pieces
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = 16 * rt + it * 4 + (lane >> 3), col = (lane & 7) * 8;
        if (r >= rows || col >= w.heads * V) continue;
        const uint4 u = ptx::lds_u32x4(ys + (r * kVLd + col) * 2);
        const size_t at = ((static_cast<size_t>(b) * p.T + t0 + r) * p.N + w.head0) * V + col;
        if (in_range(p.status, at, 8, y_extent, CHK_SCAN_OUT))
          *reinterpret_cast<uint4*>(y + at) = u;
      }
    }
    __syncthreads();  // v, the state and the sums may be overwritten
    if (hb + 1 < hb1) fetch(hb + 1);
  }
}

template <bool F32, int V>
cudaError_t run(const ScanParams& p, cudaStream_t st) {
  const int smem = out_smem_bytes<F32>(p.K);
  auto kern = out_kernel<F32, V>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const long long grid = static_cast<long long>(p.B) * p.Nq * p.hsplit * p.nc;
  kern<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_out(const ScanParams& p, bool f32, cudaStream_t st) {
  if (p.V == 16) return f32 ? scan::run<true, 16>(p, st) : scan::run<false, 16>(p, st);
  return f32 ? scan::run<true, 32>(p, st) : scan::run<false, 32>(p, st);
}

}  // namespace m2rnn

// m2rnn_few.cu -- the gated products and the 8-bit product for few tokens, and the
// split of fp32 matrices into bf16 terms.
//
// With few tokens the weights' bytes are the work: each is used for M tokens only.  A
// CTA takes 16 rows of the weights (of both, for a pair) and its warps share K in
// pieces.  A lane's 16-byte load is its part of two mma.sync fragments as it comes:
// which k stands where in a fragment does not matter as long as the tokens' fragment is
// permuted alike, so no weight passes through shared memory.  The warps' sums are
// added in warp order.
#include "m2rnn_act.cuh"
#include "m2rnn_ffn.h"
#include "m2rnn_vec.cuh"

namespace m2rnn {
namespace {

__device__ __forceinline__ void mma_e4m3_16832(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a lane loads at a time: 16 bytes of bf16 or e4m3, 32 of fp32 (8 elements).
template <bool E4M3, bool F32>
struct Piece {
  static constexpr int ELEMS = E4M3 ? 16 : 8, WORDS = F32 ? 8 : 4;
  uint32_t w[WORDS];
};

template <bool E4M3, bool F32>
__device__ __forceinline__ void load_piece(Piece<E4M3, F32>& r, const uint8_t* src, size_t off, bool in, size_t extent,
                                           int* status) {
  constexpr int E = E4M3 ? 1 : F32 ? 4 : 2;
  constexpr int N = Piece<E4M3, F32>::ELEMS, W = Piece<E4M3, F32>::WORDS;
  if (in && in_range(status, off, N, extent, CHK_GLU_IN)) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + off * E) + i);
      r.w[4 * i] = u.x;
      r.w[4 * i + 1] = u.y;
      r.w[4 * i + 2] = u.z;
      r.w[4 * i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = 0u;
  }
}

// Three bf16 terms of 8 fp32 values, as 4 packed words each.
__device__ __forceinline__ void split8(const uint32_t (&w)[8], uint32_t (&t)[3][4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // (only the first can pass bf16's range)
    const float lo = bf16_term(v[2 * i]), hi = bf16_term(v[2 * i + 1]);
    t[0][i] = ptx::pack_bf16x2(lo, hi);
    v[2 * i] = isfinite(lo) ? v[2 * i] - lo : 0.f;
    v[2 * i + 1] = isfinite(hi) ? v[2 * i + 1] - hi : 0.f;
  }
#pragma unroll
  for (int k = 1; k < 3; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[k][i] = ptx::pack_bf16x2(v[2 * i], v[2 * i + 1]);
      v[2 * i] -= ptx::bf16x2_lo(t[k][i]);
      v[2 * i + 1] -= ptx::bf16x2_hi(t[k][i]);
    }
}

// NT: groups of 8 tokens; PAIR: two weights; UN: pieces in flight.
template <int EPI, bool E4M3, bool F32, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) few_kernel(FewParams p) {
  constexpr bool PAIR = EPI != EPI_LIN8;
  constexpr int NW = PAIR ? 2 : 1, TOK = 8 * NT;
  constexpr int UN = F32 ? 1 : NT <= 2 ? 4 : 2;
  using P = Piece<E4M3, F32>;
  constexpr int STEP = 4 * P::ELEMS;  // k of a piece of a warp
  extern __shared__ float sums[];     // [WARPS][NW][TOK][17]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int f0 = blockIdx.x * 16;
  const size_t w_ext = static_cast<size_t>(p.F) * p.D, x_ext = static_cast<size_t>(p.M - 1) * p.x_row + p.D;
  const uint8_t* wp[2] = {static_cast<const uint8_t*>(p.w0), static_cast<const uint8_t*>(p.w1)};
  const uint8_t* xp = static_cast<const uint8_t*>(p.x);
  // fp32: sums of the small products apart from the leading ones
  constexpr int NS = F32 ? 2 : 1;
  float acc[NS][NW][NT][4];
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[s][m][t][i] = 0.f;
  const bool r0 = f0 + g < p.F, r1 = f0 + g + 8 < p.F;
  for (int k0 = warp * UN * STEP; k0 < p.D; k0 += WARPS * UN * STEP) {
    P a[UN][NW][2];
#pragma unroll
    for (int q = 0; q < UN; ++q) {
      const int k = k0 + q * STEP + c * P::ELEMS;
      const bool in = k < p.D;
#pragma unroll
      for (int m = 0; m < NW; ++m) {
        load_piece<E4M3, F32>(a[q][m][0], wp[m], static_cast<size_t>(f0 + g) * p.D + k, in && r0, w_ext, p.status);
        load_piece<E4M3, F32>(a[q][m][1], wp[m], static_cast<size_t>(f0 + g + 8) * p.D + k, in && r1, w_ext, p.status);
      }
    }
#pragma unroll
    for (int q = 0; q < UN; ++q) {
      const int k = k0 + q * STEP + c * P::ELEMS;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = 8 * t + g;
        P b;
        load_piece<E4M3, F32>(b, xp, static_cast<size_t>(tok) * p.x_row + k, k < p.D && tok < p.M, x_ext, p.status);
        if constexpr (F32) {
          uint32_t bt[3][4];
          split8(b.w, bt);
#pragma unroll
          for (int m = 0; m < NW; ++m) {
            uint32_t at0[3][4], at1[3][4];
            split8(a[q][m][0].w, at0);
            split8(a[q][m][1].w, at1);
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
              for (int j = 0; j < 3 - i; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t af[4] = {at0[i][2 * h], at1[i][2 * h], at0[i][2 * h + 1], at1[i][2 * h + 1]};
                  if (i + j == 0) {  // from zero, added with rounding
                    float d[4];
                    ptx::mma_bf16_16816_zero(d, af, bt[j][2 * h], bt[j][2 * h + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[0][m][t][e] += d[e];
                  } else {
                    ptx::mma_bf16_16816(acc[NS - 1][m][t], af, bt[j][2 * h], bt[j][2 * h + 1]);
                  }
                }
          }
        } else {
#pragma unroll
          for (int m = 0; m < NW; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t af[4] = {a[q][m][0].w[2 * h], a[q][m][1].w[2 * h], a[q][m][0].w[2 * h + 1],
                                      a[q][m][1].w[2 * h + 1]};
              if constexpr (E4M3)
                mma_e4m3_16832(acc[0][m][t], af, b.w[2 * h], b.w[2 * h + 1]);
              else
                ptx::mma_bf16_16816(acc[0][m][t], af, b.w[2 * h], b.w[2 * h + 1]);
            }
        }
      }
    }
  }
  // accumulator: (row g, tokens 2c, 2c+1), (row g + 8, the same)
#pragma unroll
  for (int m = 0; m < NW; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = acc[0][m][t][i];
        if constexpr (F32) v += acc[1][m][t][i];
        sums[((warp * NW + m) * TOK + 8 * t + 2 * c + (i & 1)) * 17 + g + 8 * (i >> 1)] = v;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * TOK; i += WARPS * 32) {
    const int r = i & 15, tok = i >> 4, f = f0 + r;
    if (f >= p.F || tok >= p.M) continue;
    float s[NW];
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      s[m] = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s[m] += sums[((w * NW + m) * TOK + tok) * 17 + r];
    }
    float o;
    if constexpr (E4M3) {
      const float sa = in_range(p.status, tok, 1, p.M, CHK_GLU_IN) ? __ldg(p.sa + tok) : 0.f;
      const bool in = in_range(p.status, f, 1, p.F, CHK_GLU_IN);
      s[0] *= sa * (in ? __ldg(p.sb0 + f) : 0.f);
      if constexpr (PAIR) s[NW - 1] *= sa * (in ? __ldg(p.sb1 + f) : 0.f);
    }
    if constexpr (PAIR) {
      o = (F32 ? act_of(s[0], p.act) : act2(both(s[0]), p.act).x) * s[NW - 1];
    } else {
      o = s[0];
      const size_t at = static_cast<size_t>(tok) * p.res_row + f;
      if (p.res != nullptr &&
          in_range(p.status, at, 1, static_cast<size_t>(p.M - 1) * p.res_row + p.F, CHK_GLU_IN))
        o += __bfloat162float(static_cast<const __nv_bfloat16*>(p.res)[at]);
    }
    const size_t at = static_cast<size_t>(tok) * p.F + f;
    if (!in_range(p.status, at, 1, static_cast<size_t>(p.M) * p.F, CHK_GLU_OUT)) continue;
    if constexpr (F32)
      static_cast<float*>(p.out)[at] = o;
    else
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
  }
}

template <int EPI, bool E4M3, bool F32, int NT, int WARPS>
cudaError_t launch_warps(const FewParams& p, cudaStream_t st) {
  constexpr int NW = EPI != EPI_LIN8 ? 2 : 1;
  constexpr int smem = WARPS * NW * 8 * NT * 17 * 4;
  if (smem > 48 * 1024) {
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !ready[dev]) {
      e = cudaFuncSetAttribute(few_kernel<EPI, E4M3, F32, NT, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      if (dev < 64) ready[dev] = true;
    }
  }
  few_kernel<EPI, E4M3, F32, NT, WARPS><<<(p.F + 15) / 16, WARPS * 32, smem, st>>>(p);
  return cudaGetLastError();
}
// 16 warps where each of 152 SMs gets one CTA at most and a row has 4 KB, so that every warp has
// a run of pieces; 8 otherwise.  us for 8 tokens, 8 and 16 warps: the 8-bit product D=5632
// F=2048 8.1, 6.5; gated, bf16, D=2048 F=2432 7.4, 6.8, D=1024 F=2048 (2 KB) 4.8, 5.2; D=2048
// F=5632 (352 CTAs) 10.3, 13.7.
template <int EPI, bool E4M3, bool F32, int NT>
cudaError_t launch_nt(const FewParams& p, cudaStream_t st) {
  constexpr int E = E4M3 ? 1 : F32 ? 4 : 2;
  if constexpr (NT <= 2) {
    if (p.F <= 16 * 152 && p.D * E >= 4096) return launch_warps<EPI, E4M3, F32, NT, 16>(p, st);
  }
  return launch_warps<EPI, E4M3, F32, NT, 8>(p, st);
}
template <int EPI, bool E4M3, bool F32>
cudaError_t launch_t(const FewParams& p, cudaStream_t st) {
  return p.M <= 8    ? launch_nt<EPI, E4M3, F32, 1>(p, st)
         : p.M <= 16 ? launch_nt<EPI, E4M3, F32, 2>(p, st)
         : p.M <= 32 ? launch_nt<EPI, E4M3, F32, 4>(p, st)
                     : launch_nt<EPI, E4M3, F32, 8>(p, st);
}

// A row to 64 threads, 8 elements of each at a turn; blockIdx.y: the matrix.
__global__ void __launch_bounds__(256) split_kernel(const __grid_constant__ SplitParams p) {
  let_next_begin();
  const int which = blockIdx.y, vecs = p.D / 8;
  const float* src = which == 0 ? p.src[0] : which == 1 ? p.src[1] : p.src[2];
  __nv_bfloat16* dst = which == 0 ? p.dst[0] : which == 1 ? p.dst[1] : p.dst[2];
  const long long M = which == 0 ? p.M[0] : which == 1 ? p.M[1] : p.M[2];
  const long long from = which == 0 ? p.row[0] : which == 1 ? p.row[1] : p.row[2];
  const size_t plane = static_cast<size_t>(M) * p.pitch, extent = static_cast<size_t>(M - 1) * from + p.D;
  for (long long r = blockIdx.x * 4LL + (threadIdx.x >> 6); r < M; r += gridDim.x * 4LL)
    for (int v = threadIdx.x & 63; v < vecs; v += 64) {
      const size_t at = static_cast<size_t>(r) * from + 8 * v, to = static_cast<size_t>(r) * p.pitch + 8 * v;
      if (!in_range(p.status, at, 8, extent, CHK_GLU_IN)) continue;
      const Raw<true, 8> x = raw_load<true, 8>(src + at);
      uint32_t t[3][4];
      split8(x.w, t);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (in_range(p.status, k * plane + to, 8, 3 * plane, CHK_GLU_WS))
          *reinterpret_cast<uint4*>(dst + k * plane + to) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
    }
}

}  // namespace

cudaError_t launch_few(const FewParams& p, int epi, bool e4m3, bool f32, cudaStream_t st) {
  if (epi == EPI_LIN8) return launch_t<EPI_LIN8, true, false>(p, st);
  if (e4m3) return launch_t<EPI_GLU8, true, false>(p, st);
  return f32 ? launch_t<EPI_GLU, false, true>(p, st) : launch_t<EPI_GLU, false, false>(p, st);
}

cudaError_t launch_split(const SplitParams& p, cudaStream_t st) {
  split_kernel<<<dim3(912, p.n), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace m2rnn

// m2rnn_gemm.cuh -- the product kernel of the feed-forward operators.
//
// out = sum over segments and K of A B^T.  A tile is 128 rows x BN accumulator columns of
// one CTA, or 256 x BN of a pair of CTAs (CG = 2), each of which holds half of the rows of A
// and of B, so that a byte of B in shared memory serves twice as many rows.
// One persistent CTA per SM: a warp that issues the tensor-map copies into a ring of
// K tiles (128 bytes of K each), a warp whose elected thread issues tcgen05.mma, and four
// warps that turn finished accumulators into outputs.  Tensor memory holds two
// accumulators, so that the products of the next tile run meanwhile.
//
// PAIR (gated products): the accumulator's halves are the products with two weights'
// rows of the same numbers, so g and u of an output meet in one thread.
//
// fp32: operands come as three bf16 terms each (x = x0 + x1 + x2, |x1| <= 2^-9 |x|,
// |x2| <= 2^-18 |x|), and the six products down to 2^-27 are segments of one sum, the
// small ones first.  The tensor core cuts its sums off where it should round, which
// drifts along a long sum; so K is taken in chunks whose accumulators are added with
// rounding in registers.
#pragma once
#include "m2rnn_act.cuh"
#include "m2rnn_ffn.h"
#include "m2rnn_tc5.cuh"
#include "m2rnn_vec.cuh"

namespace m2rnn {

template <int EPI_, bool E4M3_, bool F32_, bool A_MN_, bool B_MN_, int BN_, int CG_>
struct GemmCfg {
  static constexpr int EPI = EPI_, BN = BN_, CG = CG_;
  static constexpr int BM = 128 * CG, BR = BN / CG;  // rows of a tile; B's rows in a CTA
  static constexpr bool E4M3 = E4M3_, F32 = F32_, A_MN = A_MN_, B_MN = B_MN_;
  static constexpr bool PAIR = EPI == EPI_GLU || EPI == EPI_DGLU || EPI == EPI_GLU8;
  static constexpr int OUT_N = PAIR ? BN / 2 : BN;  // output columns of a tile
  static constexpr int KT = E4M3 ? 128 : 64;        // elements of a K tile
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BR * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int SMEM = STAGES * STAGE + 1024;
  static constexpr int TCOLS = 2 * BN;
  static constexpr int THREADS = 192;
};

__device__ __forceinline__ void gave_up(int* status, int site) {
  if (atomicCAS(&status[0], 0, kStatusTimeout) == 0) atomicExch(&status[1], site);
}

struct TileAt {
  int batch, m, n;
};
// Tiles in groups of 16 rows of tiles, rows fastest: what runs at the same time shares
// its B columns and, between neighbours, its A rows in L2.
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
  const int per = p.mt * p.nt;
  TileAt r;
  r.batch = t / per;
  t -= r.batch * per;
  const int group = t / (16 * p.nt), first = group * 16;
  const int rows = min(16, p.mt - first);
  t -= group * 16 * p.nt;
  r.m = first + t % rows;
  r.n = t / rows;
  return r;
}

template <class C>
__device__ __forceinline__ void issue_tile(const GemmParams& p, uint32_t dst, uint32_t bar, const TileAt& t, int rank,
                                           int seg, int kt) {
  const int k = kt * C::KT;
  const int az = p.az[seg] + t.batch * p.az_step, bz = p.bz[seg];
  const int m = t.m * C::BM + rank * 128;
  if constexpr (C::A_MN) {
    tc5::copy_box<C::CG>(dst, &p.a, m, k, az, bar);
    tc5::copy_box<C::CG>(dst + 8192, &p.a, m + 64, k, az, bar);
  } else {
    tc5::copy_box<C::CG>(dst, &p.a, k, m, az, bar);
  }
  const uint32_t b = dst + C::A_BYTES;
  if constexpr (C::PAIR) {
    const int n = t.n * C::OUT_N;
    if constexpr (C::CG == 2) {  // a weight to each CTA
      tc5::copy_box<2>(b, rank ? &p.b1 : &p.b0, k, n, bz, bar);
    } else {
      tc5::copy_box<1>(b, &p.b0, k, n, bz, bar);
      tc5::copy_box<1>(b + C::B_BYTES / 2, &p.b1, k, n, bz, bar);
    }
  } else {
    const int n = t.n * C::OUT_N + rank * C::BR;
    const CUtensorMap* map = p.bi[seg] ? &p.b1 : &p.b0;
    if constexpr (C::B_MN) {
#pragma unroll
      for (int i = 0; i < C::BR / 64; ++i) tc5::copy_box<C::CG>(b + 8192 * i, map, n + 64 * i, k, bz, bar);
    } else {
      tc5::copy_box<C::CG>(b, map, k, n, bz, bar);
    }
  }
}

// 32 outputs of one row, `cols` of them inside the matrix (a multiple of 8).
template <bool F32>
__device__ __forceinline__ void store32(void* out, size_t at, int cols, const float (&v)[32], size_t extent,
                                        int* status, int site) {
  using T = typename Elem<F32>::T;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (8 * i < cols && in_range(status, at + 8 * i, 8, extent, site)) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = v[8 * i + j];
      store_vec<F32, 8>(static_cast<T*>(out) + at + 8 * i, o);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void load32(const void* in, size_t at, int cols, float (&v)[32], size_t extent,
                                       int* status, int site) {
  using T = typename Elem<F32>::T;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (8 * i < cols && in_range(status, at + 8 * i, 8, extent, site))
      raw_unpack<F32, 8>(raw_load<F32, 8, false>(static_cast<const T*>(in) + at + 8 * i), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * i + j] = o[j];
  }
}

// The bf16 terms of fp32 values: each the rounding of what the ones before leave.  A
// value that is not finite is its own first term.
__device__ __forceinline__ void next_term(float (&v)[32], float (&t)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    t[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
    v[i] = isfinite(t[i]) ? v[i] - t[i] : 0.f;
  }
}

// One row's 32 columns from their accumulators (g, u: the pair, or the product in g).
template <class C>
__device__ __forceinline__ void finish32(const GemmParams& p, const TileAt& t, long long row, int col, float (&g)[32],
                                         float (&u)[32]) {
  const int cols = min(32, p.N - col);
  if (row >= p.M || cols <= 0) return;
  const size_t at = static_cast<size_t>(row) * p.N + col, extent = static_cast<size_t>(p.M) * p.N;
  if constexpr (C::EPI == EPI_GLU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] = act_of<C::F32>(g[i], p.act) * u[i];
    store32<C::F32>(p.out[0], at, cols, g, extent, p.status, CHK_GLU_OUT);
  } else if constexpr (C::EPI == EPI_DGLU) {
    float d[32];
    load32<C::F32>(p.in, at, cols, d, extent, p.status, CHK_GLU_IN);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float a, s;
      act_grad<C::F32>(g[i], p.act, a, s);
      g[i] = d[i] * u[i] * s;
      u[i] = d[i] * a;
    }
    // Rounded to bf16 (bf16 inputs): they are operands of the products to come.  fp32 inputs:
    // three terms, which hold the value.
    constexpr int terms = C::F32 ? 3 : 1;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[0]);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int k = 0; k < terms; ++k) {
        const size_t plane = static_cast<size_t>(which * terms + k) * extent;
        if constexpr (C::F32)
          next_term(which ? u : g, d);
        else {
#pragma unroll
          for (int i = 0; i < 32; ++i) d[i] = which ? u[i] : g[i];
        }
        store32<false>(out, plane + at, cols, d, 2 * terms * extent, p.status, CHK_GLU_WS);
      }
    }
  } else if constexpr (C::EPI == EPI_STORE) {
    store32<C::F32>(t.batch ? p.out[1] : p.out[0], at, cols, g, extent, p.status, CHK_GLU_OUT);
  } else {
    const float sa = __ldg(p.sa + row);
    const size_t n = static_cast<size_t>(p.N);
    if constexpr (C::EPI == EPI_GLU8) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const bool in = i < cols && in_range(p.status, col + i, 1, n, CHK_GLU_IN);
        const float s0 = in ? __ldg(p.sb0 + col + i) : 0.f, s1 = in ? __ldg(p.sb1 + col + i) : 0.f;
        g[i] = act_of<false>(g[i] * (sa * s0), p.act) * (u[i] * (sa * s1));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const bool in = i < cols && in_range(p.status, col + i, 1, n, CHK_GLU_IN);
        g[i] *= sa * (in ? __ldg(p.sb0 + col + i) : 0.f);
      }
      if (p.in != nullptr) {
        load32<false>(p.in, static_cast<size_t>(row) * p.in_row + col, cols, u,
                      static_cast<size_t>(p.M - 1) * p.in_row + n, p.status, CHK_GLU_IN);
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] += u[i];
      }
    }
    store32<false>(p.out[0], at, cols, g, extent, p.status, CHK_GLU_OUT);
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) gemm_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * C::STAGES + 5];
  __shared__ uint32_t tslot;
  const uint32_t base = (ptx::smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t full = ptx::smem_addr(&bars[0]), empty = full + 8 * C::STAGES;
  const uint32_t tfull = empty + 8 * C::STAGES, tempty = tfull + 16, drain = tempty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = C::CG == 2 ? static_cast<int>(tc5::cta_rank()) : 0;
  const int first = blockIdx.x / C::CG, stride = gridDim.x / C::CG;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      ptx::mbar_init(full + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(tfull + 8 * i, 1);
      ptx::mbar_init(tempty + 8 * i, 4 * C::CG);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_init_fence();
  }
  if (warp == 5) tc5::alloc<C::CG>(ptx::smem_addr(&tslot), C::TCOLS);
  tc5::fence_before();
  __syncthreads();
  if constexpr (C::CG == 2) tc5::cluster_sync();
  tc5::fence_after();
  const uint32_t tm = tslot;
  let_next_begin();
  await_before();

  const int tiles = p.mt * p.nt * p.nbatch, nchunk = (p.kt + p.kc - 1) / p.kc;
  if (warp == 4) {
    if (tc5::elect_one()) {
      tc5::prefetch_map(&p.a);
      tc5::prefetch_map(&p.b0);
      tc5::prefetch_map(&p.b1);
      const uint32_t full0 = C::CG == 2 ? tc5::map_to(full, 0) : full;
      int it = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const TileAt at = tile_at(p, t);
        for (int c = 0; c < nchunk && ok; ++c)
          for (int s = 0; s < p.nseg && ok; ++s)
            for (int k = c * p.kc; k < min(p.kt, (c + 1) * p.kc); ++k, ++it) {
              const int st = it % C::STAGES, round = it / C::STAGES;
              if (!ptx::mbar_wait(empty + 8 * st, (round & 1) ^ 1, p.limit_ns)) {
                ok = false;
                break;
              }
              // (the pair's copies are counted in the first CTA, whose thread issues the products)
              if (rank == 0) tc5::arrive_expect(full + 8 * st, C::CG * C::STAGE);
              issue_tile<C>(p, base + st * C::STAGE, full0 + 8 * st, at, rank, s, k);
            }
      }
      // The last products have been done, and have said so, before a CTA of a pair goes.
      for (int i = max(0, it - C::STAGES); i < it && ok && C::CG == 2; ++i)
        ok = ptx::mbar_wait(empty + 8 * (i % C::STAGES), (i / C::STAGES) & 1, p.limit_ns);
      if (!ok) {  // copies in flight land before the CTA goes
        gave_up(p.status, SITE_GEMM_COPY);
        for (int i = max(0, it - C::STAGES); i < it && rank == 0; ++i)
          ptx::mbar_wait(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, p.limit_ns);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    if (rank == 0 && tc5::elect_one()) {
      constexpr uint32_t id = tc5::idesc(C::BM, C::BN, C::E4M3, C::A_MN, C::B_MN);
      constexpr uint32_t a_step = C::A_MN ? 2048 : 32, b_step = C::B_MN ? 2048 : 32;
      int it = 0, acc = 0;
      bool ok = true;
      int site = SITE_GEMM_MMA;
      for (int t = first; t < tiles && ok; t += stride)
        for (int c = 0; c < nchunk && ok; ++c, ++acc) {
          const int ab = acc & 1;
          if (!tc5::wait_released<C::CG>(tempty + 8 * ab, ((acc >> 1) & 1) ^ 1, p.limit_ns)) {
            ok = false;
            break;
          }
          tc5::fence_after();
          bool add = false;
          for (int s = 0; s < p.nseg && ok; ++s)
            for (int k = c * p.kc; k < min(p.kt, (c + 1) * p.kc); ++k, ++it) {
              const int st = it % C::STAGES;
              if (!ptx::mbar_wait(full + 8 * st, (it / C::STAGES) & 1, p.limit_ns)) {
                ok = false;
                break;
              }
              tc5::fence_after();
              const uint32_t sa = base + st * C::STAGE, sb = sa + C::A_BYTES;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                tc5::mma<C::E4M3, C::CG>(tm + ab * C::BN, tc5::sdesc(sa + i * a_step, C::A_MN ? 8192 : 16, 1024),
                                  tc5::sdesc(sb + i * b_step, C::B_MN ? 8192 : 16, 1024), id, add);
                add = true;
              }
              tc5::commit<C::CG>(empty + 8 * st);
            }
          if (ok) tc5::commit<C::CG>(tfull + 8 * ab);
        }
      if (!ok) {
        gave_up(p.status, site);
        tc5::commit<C::CG>(drain);
        if (!ptx::mbar_wait(drain, 0, p.limit_ns)) gave_up(p.status, SITE_GEMM_DRAIN);
      }
    }
    __syncwarp();
  } else {
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tempty0 = C::CG == 2 ? tc5::map_to(tempty, 0) : tempty;
    const auto release = [&](int ab) {  // the accumulator has been read
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (C::CG == 2)
          tc5::arrive_cluster(tempty0 + 8 * ab);
        else
          ptx::mbar_arrive(tempty0 + 8 * ab);
      }
    };
    int acc = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += stride) {
      const TileAt at = tile_at(p, t);
      const long long row = static_cast<long long>(at.m) * C::BM + rank * 128 + warp * 32 + lane;
      const int col0 = at.n * C::OUT_N;
      if constexpr (C::F32) {
        float sum[C::BN / 32][32];
        for (int c = 0; c < nchunk; ++c, ++acc) {
          const int ab = acc & 1;
          ok = ptx::mbar_wait(tfull + 8 * ab, (acc >> 1) & 1, p.limit_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc5::fence_after();
#pragma unroll
          for (int b = 0; b < C::BN / 32; ++b) {
            float v[32];
            tc5::ld32(tm + lanes + ab * C::BN + 32 * b, v);
            tc5::wait_ld(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[b][i] = c == 0 ? v[i] : sum[b][i] + v[i];
          }
          release(ab);
        }
        if (ok) {
#pragma unroll
          for (int b = 0; b < C::OUT_N / 32; ++b)
            finish32<C>(p, at, row, col0 + 32 * b, sum[b], sum[C::PAIR ? b + C::OUT_N / 32 : b]);
        }
      } else {
        const int ab = acc & 1;
        ok = ptx::mbar_wait(tfull + 8 * ab, (acc >> 1) & 1, p.limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc5::fence_after();
          const uint32_t ta = tm + lanes + ab * C::BN;
#pragma unroll 1
          for (int b = 0; b < C::OUT_N / 32; ++b) {
            float g[32], u[32];
            __syncwarp();
            tc5::ld32(ta + 32 * b, g);
            if constexpr (C::PAIR) tc5::ld32(ta + C::OUT_N + 32 * b, u);
            tc5::wait_ld(g);
            if constexpr (C::PAIR) tc5::wait_ld(u);
            if (b == C::OUT_N / 32 - 1) release(ab);
            finish32<C>(p, at, row, col0 + 32 * b, g, u);
          }
        }
        ++acc;
      }
    }
    if (!ok && lane == 0) gave_up(p.status, SITE_GEMM_OUT);
  }
  tc5::fence_before();
  __syncthreads();
  if constexpr (C::CG == 2) tc5::cluster_sync();
  tc5::fence_after();
  if (warp == 5) tc5::dealloc<C::CG>(tm, C::TCOLS);
}

template <class C>
cudaError_t launch_cfg(const GemmParams& p, int sms, cudaStream_t st) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  const long long tiles = static_cast<long long>(p.mt) * p.nt * p.nbatch, most = sms / C::CG;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C::CG;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(C::CG * (tiles < most ? tiles : most)));
  c.blockDim = dim3(C::THREADS);
  c.dynamicSmemBytes = C::SMEM;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = C::CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&c, gemm_kernel<C>, p);
}

}  // namespace m2rnn

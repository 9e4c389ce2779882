// m2rnn_gemm.cuh -- the product kernel of the feed-forward operators.
//
// out = sum over segments and K of A B^T.  A tile is 128 rows x BN accumulator columns of
// one CTA, or 256 x BN of a pair of CTAs (CG = 2), each of which holds half of the rows of A
// and of B, so that a byte of B in shared memory serves twice as many rows.
// One persistent CTA per SM: a warp that issues the tensor-map copies into a ring of
// K tiles (128 bytes of K each), a warp whose elected thread issues tcgen05.mma, and eight
// warps that turn finished accumulators into outputs.  Tensor memory holds two sets of
// accumulators, so that the products of the next tile run meanwhile.
//
// PAIR (gated products): the accumulator's halves are the products with two weights'
// rows of the same numbers, so g and u of an output meet in one thread.
//
// fp32: operands come as three bf16 terms each (x = x0 + x1 + x2, |x1| <= 2^-9 |x|,
// |x2| <= 2^-18 |x|); a K tile holds all terms of both, and the six products down to
// 2^-27 are formed from it.  The tensor core cuts its sums off where it should round, which
// drifts along a long sum; so the leading products and the small ones have accumulators of
// their own, and K is taken in chunks whose sums are added with rounding in registers.
//
// A last wave of few tiles is cut along K (`split` parts each, fp32 sums in memory that
// join_parts_kernel adds in order), so that it takes 1/split of a wave; so are all tiles of
// very long sums.
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
  static constexpr int TERMS = F32 ? 3 : 1;
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BR * 128;  // of a term
  static constexpr int STAGE = TERMS * (A_BYTES + B_BYTES);
  static constexpr int STAGES = 216 * 1024 / STAGE;  // (6 of 32 KB, 3 of 72 KB, 2 of 96 KB)
  // bf16 outputs and what they read pass through 2 KB of each output warp (where there is room)
  static constexpr int STAGED = F32 && CG == 2 ? 0 : 2048;
  static constexpr int SMEM = STAGES * STAGE + 1024 + 8 * STAGED;
  static constexpr int ACC = F32 ? 2 * BN : BN;  // columns of a set of accumulators
  static constexpr int TCOLS = 2 * ACC;
  static constexpr int OUT_WARPS = 8, THREADS = 32 * (OUT_WARPS + 2);
  static constexpr int BLOCKS = OUT_N / 32 / 2;  // blocks of 32 output columns of a warp
};

// How long a kernel that gave up waits for its own copies and products.
constexpr uint64_t kDrainNs = 1000000000ull;

__device__ __forceinline__ void gave_up(int* status, int site) {
  if (atomicCAS(&status[0], 0, kStatusTimeout) == 0) atomicExch(&status[1], site);
}

// A unit of work: a tile, or the part `part` of a tile of the last wave.
struct TileAt {
  int batch, m, n, k0, k1, part;  // part < 0: the whole tile
};
// Tiles in groups of 16 rows of tiles, rows fastest: what runs at the same time shares
// its B columns and, between neighbours, its A rows in L2.
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
  TileAt r;
  r.k0 = 0;
  r.k1 = p.kt;
  r.part = -1;
  if (t >= p.whole) {
    r.part = t - p.whole;
    t = p.whole + r.part / p.split;
    const int i = r.part % p.split;
    r.k0 = static_cast<int>(static_cast<long long>(p.kt) * i / p.split);
    r.k1 = static_cast<int>(static_cast<long long>(p.kt) * (i + 1) / p.split);
  }
  const int per = p.mt * p.nt;
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
  const int m = t.m * C::BM + rank * 128;
#pragma unroll
  for (int term = 0; term < C::TERMS; ++term) {
    const uint32_t a = dst + term * C::A_BYTES;
    const int az = C::F32 ? (seg + t.batch) * 3 + term : seg + t.batch * p.aterms;
    if constexpr (C::A_MN) {
      tc5::copy_box<C::CG>(a, &p.a, m, k, az, bar);
      tc5::copy_box<C::CG>(a + 8192, &p.a, m + 64, k, az, bar);
    } else {
      tc5::copy_box<C::CG>(a, &p.a, k, m, az, bar);
    }
    const uint32_t b = dst + C::TERMS * C::A_BYTES + term * C::B_BYTES;
    if constexpr (C::PAIR) {
      const int n = t.n * C::OUT_N;
      if constexpr (C::CG == 2) {  // a weight to each CTA
        tc5::copy_box<2>(b, rank ? &p.b1 : &p.b0, k, n, term, bar);
      } else {
        tc5::copy_box<1>(b, &p.b0, k, n, term, bar);
        tc5::copy_box<1>(b + C::B_BYTES / 2, &p.b1, k, n, term, bar);
      }
    } else {
      const int n = t.n * C::OUT_N + rank * C::BR;
      const CUtensorMap* map = seg >= (C::F32 ? 1 : p.aterms) ? &p.b1 : &p.b0;
      if constexpr (C::B_MN) {
#pragma unroll
        for (int i = 0; i < C::BR / 64; ++i) tc5::copy_box<C::CG>(b + 8192 * i, map, n + 64 * i, k, term, bar);
      } else {
        tc5::copy_box<C::CG>(b, map, k, n, term, bar);
      }
    }
  }
}

// 32 fp32 values of one row, `cols` of them inside the matrix (a multiple of 8).
__device__ __forceinline__ void store32(void* out, size_t at, int cols, const float (&v)[32], size_t extent,
                                        int* status, int site) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (8 * i < cols && in_range(status, at + 8 * i, 8, extent, site)) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = v[8 * i + j];
      store_vec<true, 8>(static_cast<float*>(out) + at + 8 * i, o);
    }
  }
}
__device__ __forceinline__ void load32(const void* in, size_t at, int cols, float (&v)[32], size_t extent,
                                       int* status, int site) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (8 * i < cols && in_range(status, at + 8 * i, 8, extent, site))
      raw_unpack<true, 8>(raw_load<true, 8, false>(static_cast<const float*>(in) + at + 8 * i), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * i + j] = o[j];
  }
}

// 32 scales (the same ones for the whole warp).  Plain loads, as of everything here: a kernel
// before may still write what this one reads when it becomes resident (await_before).
__device__ __forceinline__ void load32_scales(const float* in, int at, int cols, float (&v)[32], size_t extent,
                                             int* status) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (8 * i < cols && in_range(status, at + 8 * i, 8, extent, CHK_GLU_IN))
      raw_unpack<true, 8>(raw_load<true, 8, false>(in + at + 8 * i), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * i + j] = o[j];
  }
}

// The next bf16 term of fp32 values: the rounding of what the terms before leave (the first one cut
// off where rounding would pass bf16's largest value; a value that is not finite is its own
// first term).
template <bool FIRST>
__device__ __forceinline__ void next_term(float (&v)[32], float (&t)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    t[i] = FIRST ? bf16_term(v[i]) : __bfloat162float(__float2bfloat16_rn(v[i]));
    v[i] = !FIRST || isfinite(t[i]) ? v[i] - t[i] : 0.f;
  }
}

// What the rounding to bf16 leaves of v (0 where that is infinite or NaN, which stays so in the sum).
__device__ __forceinline__ void leave_rest(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const uint32_t w = ptx::pack_bf16x2(v[i], v[i + 1]);
    const float2 r = fma2(make_float2(ptx::bf16x2_lo(w), ptx::bf16x2_hi(w)), both(-1.f), make_float2(v[i], v[i + 1]));
    v[i] = isfinite(r.x) ? r.x : 0.f;
    v[i + 1] = isfinite(r.y) ? r.y : 0.f;
  }
}

// A warp's block of 32 rows of 32 bf16 columns on its way between memory, where four lanes
// hold a row's 64 bytes (eight rows to an instruction), and a row per lane.  In the warp's 2 KB
// the 16-byte pieces of a row are exchanged by its number, so that neither side has
// bank conflicts.
__device__ __forceinline__ uint32_t piece_at(uint32_t buf, int row, int piece) {
  return buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
struct Block {  // rows and columns of the matrix that the block covers, from `at` on
  size_t at, row;
  long long rows;
  int cols;
  size_t extent;
};
__device__ __forceinline__ void block_load(uint4 (&v)[4], const __nv_bfloat16* src, const Block& k, int lane,
                                           int* status) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), c = lane & 3;
    const size_t at = k.at + r * k.row + 8 * c;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < k.rows && 8 * c < k.cols && in_range(status, at, 8, k.extent, CHK_GLU_IN))
      v[i] = *reinterpret_cast<const uint4*>(src + at);
  }
}
// What block_load took, as the lane's row.
__device__ __forceinline__ void block_rows(const uint4 (&v)[4], uint32_t buf, int lane, float (&o)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sts128(piece_at(buf, 8 * i + (lane >> 2), lane & 3), v[i]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 u = ptx::lds_u32x4(piece_at(buf, lane, i));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[8 * i + 2 * j] = ptx::bf16x2_lo(w[j]);
      o[8 * i + 2 * j + 1] = ptx::bf16x2_hi(w[j]);
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void block_store(__nv_bfloat16* dst, const Block& k, uint32_t buf, int lane,
                                            const float (&o)[32], int* status, int site) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sts128(piece_at(buf, lane, i),
           make_uint4(ptx::pack_bf16x2(o[8 * i], o[8 * i + 1]), ptx::pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                      ptx::pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), ptx::pack_bf16x2(o[8 * i + 6], o[8 * i + 7])));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), c = lane & 3;
    const size_t at = k.at + r * k.row + 8 * c;
    const uint4 u = ptx::lds_u32x4(piece_at(buf, r, c));
    if (r < k.rows && 8 * c < k.cols && in_range(status, at, 8, k.extent, site))
      *reinterpret_cast<uint4*>(dst + at) = u;
  }
  __syncwarp();
}

// fp32 sums of a part of a tile: [part][rows of a tile][BN], `col` of the output (a pair's second
// product behind the first).
template <class C>
__device__ __forceinline__ void store_part(const GemmParams& p, const TileAt& t, long long row, int col,
                                           const float (&g)[32], int second = 0) {
  if (row >= p.M || col >= p.N) return;
  const size_t tile = static_cast<size_t>(C::BM) * C::BN;
  const size_t at = t.part * tile + static_cast<size_t>(row - static_cast<long long>(t.m) * C::BM) * C::BN +
                    (col - t.n * C::OUT_N + second * C::OUT_N);
  store32(p.parts, at, 32, g, tile * p.nparts, p.status, CHK_GLU_WS);
}

// Where the output's block of a warp's 32 rows from row0 on lies, with `pitch` elements to a row.
__device__ __forceinline__ Block block_of(const GemmParams& p, long long row0, int col, long long pitch) {
  Block k;
  k.row = static_cast<size_t>(pitch);
  k.at = static_cast<size_t>(row0) * k.row + col;
  k.rows = p.M - row0;
  k.cols = min(32, p.N - col);
  k.extent = static_cast<size_t>(p.M - 1) * k.row + p.N;
  return k;
}

// A block's outputs from its accumulators (g, u: the pair, or the product in g); `in`: what
// block_load took of dh or res.
template <class C>
__device__ __forceinline__ void finish_bf16(const GemmParams& p, const TileAt& t, long long row0, int col, int lane,
                                            uint32_t buf, float (&g)[32], float (&u)[32], const uint4 (&in)[4]) {
  const Block k = block_of(p, row0, col, C::EPI == EPI_DGLU ? p.pitch : p.N);
  if constexpr (C::EPI == EPI_GLU) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 h = mul2(act2(make_float2(g[i], g[i + 1]), p.act), make_float2(u[i], u[i + 1]));
      g[i] = h.x;
      g[i + 1] = h.y;
    }
    block_store(static_cast<__nv_bfloat16*>(p.out[0]), k, buf, lane, g, p.status, CHK_GLU_OUT);
  } else if constexpr (C::EPI == EPI_DGLU) {
    float d[32];
    block_rows(in, buf, lane, d);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 dh = make_float2(d[i], d[i + 1]);
      float2 a, s;
      act_grad2(make_float2(g[i], g[i + 1]), p.act, a, s);
      const float2 dg = mul2(mul2(dh, make_float2(u[i], u[i + 1])), s), du = mul2(dh, a);
      g[i] = dg.x;
      g[i + 1] = dg.y;
      u[i] = du.x;
      u[i + 1] = du.y;
    }
    // Rounded to bf16, as operands of the products to come; what the rounding leaves follows as a
    // second term.
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[0]);
    const size_t plane = static_cast<size_t>(p.M) * p.pitch;
    if (p.aterms == 1) {
      block_store(out, k, buf, lane, g, p.status, CHK_GLU_WS);
      block_store(out + plane, k, buf, lane, u, p.status, CHK_GLU_WS);
    } else {
      block_store(out, k, buf, lane, g, p.status, CHK_GLU_WS);
      leave_rest(g);
      block_store(out + plane, k, buf, lane, g, p.status, CHK_GLU_WS);
      block_store(out + 2 * plane, k, buf, lane, u, p.status, CHK_GLU_WS);
      leave_rest(u);
      block_store(out + 3 * plane, k, buf, lane, u, p.status, CHK_GLU_WS);
    }
  } else if constexpr (C::EPI == EPI_STORE) {
    if (t.part >= 0)
      store_part<C>(p, t, row0 + lane, col, g);
    else
      block_store(static_cast<__nv_bfloat16*>(t.batch ? p.out[1] : p.out[0]), k, buf, lane, g, p.status, CHK_GLU_OUT);
  } else {
    const float sa = lane < k.rows && in_range(p.status, row0 + lane, 1, p.M, CHK_GLU_IN) ? p.sa[row0 + lane] : 0.f;
    const size_t n = static_cast<size_t>(p.N);
    float s[32];
    load32_scales(p.sb0, col, k.cols, s, n, p.status);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 v = mul2(make_float2(g[i], g[i + 1]), mul2(both(sa), make_float2(s[i], s[i + 1])));
      g[i] = v.x;
      g[i + 1] = v.y;
    }
    if constexpr (C::EPI == EPI_GLU8) {
      load32_scales(p.sb1, col, k.cols, s, n, p.status);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 v = mul2(make_float2(u[i], u[i + 1]), mul2(both(sa), make_float2(s[i], s[i + 1])));
        const float2 h = mul2(act2(make_float2(g[i], g[i + 1]), p.act), v);
        g[i] = h.x;
        g[i + 1] = h.y;
      }
    } else if (p.in != nullptr) {
      block_rows(in, buf, lane, s);
#pragma unroll
      for (int i = 0; i < 32; ++i) g[i] += s[i];
    }
    block_store(static_cast<__nv_bfloat16*>(p.out[0]), k, buf, lane, g, p.status, CHK_GLU_OUT);
  }
}

// fp32: one row's 32 columns (all lanes of the warp are here).
template <class C>
__device__ __forceinline__ void finish_f32(const GemmParams& p, const TileAt& t, long long row0, int col, int lane,
                                           uint32_t buf, float (&g)[32], float (&u)[32]) {
  const long long row = row0 + lane;
  const int cols = row < p.M ? min(32, p.N - col) : 0;  // of the lane's row
  if (C::EPI != EPI_DGLU && cols <= 0) return;
  const size_t at = static_cast<size_t>(row) * p.N + col, extent = static_cast<size_t>(p.M) * p.N;
  if (t.part >= 0) {
    store_part<C>(p, t, row, col, g);
    if constexpr (C::PAIR) store_part<C>(p, t, row, col, u, 1);
    return;
  }
  if constexpr (C::EPI == EPI_GLU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] = act_of(g[i], p.act) * u[i];
    store32(p.out[0], at, cols, g, extent, p.status, CHK_GLU_OUT);
  } else if constexpr (C::EPI == EPI_DGLU) {
    static_assert(C::STAGED > 0, "the terms pass through shared memory");
    float d[32];
    load32(p.in, at, cols, d, extent, p.status, CHK_GLU_IN);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float a, s;
      act_grad(g[i], p.act, a, s);
      g[i] = d[i] * u[i] * s;
      u[i] = d[i] * a;
    }
    // as the three terms that the products to come take
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[0]);
    const size_t plane = static_cast<size_t>(p.M) * p.pitch;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k == 0)
          next_term<true>(which ? u : g, d);
        else
          next_term<false>(which ? u : g, d);
        block_store(out + (which * 3 + k) * plane, block_of(p, row0, col, p.pitch), buf, lane, d, p.status, CHK_GLU_WS);
      }
  } else {
    store32(t.batch ? p.out[1] : p.out[0], at, cols, g, extent, p.status, CHK_GLU_OUT);
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
      ptx::mbar_init(tempty + 8 * i, C::OUT_WARPS * C::CG);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_init_fence();
  }
  if (warp == C::OUT_WARPS + 1) tc5::alloc<C::CG>(ptx::smem_addr(&tslot), C::TCOLS);
  tc5::fence_before();
  __syncthreads();
  if constexpr (C::CG == 2) tc5::cluster_sync();
  tc5::fence_after();
  const uint32_t tm = tslot;
  let_next_begin();
  await_before();

  const int tiles = p.whole + p.nparts;
  if (warp == C::OUT_WARPS) {
    if (tc5::elect_one()) {
      tc5::prefetch_map(&p.a);
      tc5::prefetch_map(&p.b0);
      tc5::prefetch_map(&p.b1);
      const uint32_t full0 = C::CG == 2 ? tc5::map_to(full, 0) : full;
      int it = 0;
      bool ok = true;
      for (int t = p.inject_stall ? tiles : first; t < tiles && ok; t += stride) {
        const TileAt at = tile_at(p, t);
        for (int c = at.k0; c < at.k1 && ok; c += p.kc)
          for (int s = 0; s < p.nseg && ok; ++s)
            for (int k = c; k < min(at.k1, c + p.kc); ++k, ++it) {
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
        if (rank == 0) {
          for (int i = max(0, it - C::STAGES); i < it; ++i)
            ptx::mbar_wait(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, kDrainNs);
        } else {  // (they are counted in the other CTA: a thousand times what a copy takes)
          const uint64_t t0 = ptx::globaltimer_ns();
          while (ptx::globaltimer_ns() - t0 < 1000000) __nanosleep(1000);
        }
      }
    }
    __syncwarp();
  } else if (warp == C::OUT_WARPS + 1) {
    if (rank == 0 && tc5::elect_one()) {
      constexpr uint32_t id = tc5::idesc(C::BM, C::BN, C::E4M3, C::A_MN, C::B_MN);
      constexpr uint32_t a_step = C::A_MN ? 2048 : 32, b_step = C::B_MN ? 2048 : 32;
      int it = 0, acc = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const TileAt at = tile_at(p, t);
        for (int c = at.k0; c < at.k1 && ok; c += p.kc, ++acc) {
          const int ab = acc & 1;
          if (!tc5::wait_released<C::CG>(tempty + 8 * ab, ((acc >> 1) & 1) ^ 1, p.limit_ns)) {
            ok = false;
            break;
          }
          tc5::fence_after();
          const uint32_t lead = tm + ab * C::ACC, small = lead + C::BN;
          bool add = false;
          for (int s = 0; s < p.nseg && ok; ++s)
            for (int k = c; k < min(at.k1, c + p.kc); ++k, ++it) {
              const int st = it % C::STAGES;
              if (!ptx::mbar_wait(full + 8 * st, (it / C::STAGES) & 1, p.limit_ns)) {
                ok = false;
                break;
              }
              tc5::fence_after();
              const uint32_t sa = base + st * C::STAGE, sb = sa + C::TERMS * C::A_BYTES;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const auto ad = [&](int term) {
                  return tc5::sdesc(sa + term * C::A_BYTES + i * a_step, C::A_MN ? 8192 : 16, 1024);
                };
                const auto bd = [&](int term) {
                  return tc5::sdesc(sb + term * C::B_BYTES + i * b_step, C::B_MN ? 8192 : 16, 1024);
                };
                if constexpr (C::F32) {  // (a term of A is read once for its products)
                  tc5::mma<C::E4M3, C::CG, tc5::KEEP_FILL>(lead, ad(0), bd(0), id, add);
                  tc5::mma<C::E4M3, C::CG, tc5::KEEP_USE>(small, ad(0), bd(2), id, add);
                  tc5::mma<C::E4M3, C::CG, tc5::KEEP_LAST>(small, ad(0), bd(1), id, true);
                  tc5::mma<C::E4M3, C::CG, tc5::KEEP_FILL>(small, ad(1), bd(1), id, true);
                  tc5::mma<C::E4M3, C::CG, tc5::KEEP_LAST>(small, ad(1), bd(0), id, true);
                  tc5::mma<C::E4M3, C::CG>(small, ad(2), bd(0), id, true);
                } else {
                  tc5::mma<C::E4M3, C::CG>(lead, ad(0), bd(0), id, add);
                }
                add = true;
              }
              tc5::commit<C::CG>(empty + 8 * st);
            }
          if (ok) tc5::commit<C::CG>(tfull + 8 * ab);
        }
      }
      if (!ok) {
        gave_up(p.status, SITE_GEMM_MMA);
        tc5::commit<C::CG>(drain);
        if (!ptx::mbar_wait(drain, 0, kDrainNs)) gave_up(p.status, SITE_GEMM_DRAIN);
      }
    }
    __syncwarp();
  } else {
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int half = (warp >> 2) * C::BLOCKS;  // this warp's first block of columns
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
      const long long row0 = static_cast<long long>(at.m) * C::BM + rank * 128 + (warp & 3) * 32;
      const int col0 = at.n * C::OUT_N;
      if constexpr (C::F32) {
        const uint32_t buf = base + C::STAGES * C::STAGE + warp * C::STAGED;
        float sum[C::PAIR ? 2 : 1][C::BLOCKS][32];
        for (int c = at.k0; c < at.k1; c += p.kc, ++acc) {
          const int ab = acc & 1;
          ok = ptx::mbar_wait(tfull + 8 * ab, (acc >> 1) & 1, p.limit_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc5::fence_after();
#pragma unroll
          for (int w = 0; w < (C::PAIR ? 2 : 1); ++w)
#pragma unroll
            for (int b = 0; b < C::BLOCKS; ++b) {
              float v[32], r[32];
              const uint32_t ta = tm + lanes + ab * C::ACC + w * C::OUT_N + 32 * (half + b);
              tc5::ld32(ta, v);
              tc5::ld32(ta + C::BN, r);
              tc5::wait_ld(v);
              tc5::wait_ld(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[w][b][i] = c == at.k0 ? v[i] + r[i] : sum[w][b][i] + (v[i] + r[i]);
            }
          release(ab);
        }
        if (ok) {
#pragma unroll
          for (int b = 0; b < C::BLOCKS; ++b)
            finish_f32<C>(p, at, row0, col0 + 32 * (half + b), lane, buf, sum[0][b], sum[C::PAIR ? 1 : 0][b]);
        }
      } else {
        const int ab = acc & 1;
        const uint32_t buf = base + C::STAGES * C::STAGE + warp * C::STAGED;
        const bool reads = C::EPI == EPI_DGLU || (C::EPI == EPI_LIN8 && p.in != nullptr);
        const long long in_row = C::EPI == EPI_DGLU ? p.N : p.in_row;
        const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(p.in);
        uint4 next[4];  // of dh or res: in flight while the accumulators are waited for
        if (reads) block_load(next, in, block_of(p, row0, col0 + 32 * half, in_row), lane, p.status);
        ok = ptx::mbar_wait(tfull + 8 * ab, (acc >> 1) & 1, p.limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc5::fence_after();
          const uint32_t ta = tm + lanes + ab * C::ACC + 32 * half;
#pragma unroll 1
          for (int b = 0; b < C::BLOCKS; ++b) {
            float g[32], u[32];
            uint4 now[4];
            const int col = col0 + 32 * (half + b);
            __syncwarp();
            tc5::ld32(ta + 32 * b, g);
            if constexpr (C::PAIR) tc5::ld32(ta + C::OUT_N + 32 * b, u);
            if (reads) {
#pragma unroll
              for (int i = 0; i < 4; ++i) now[i] = next[i];
              if (b + 1 < C::BLOCKS) block_load(next, in, block_of(p, row0, col + 32, in_row), lane, p.status);
            }
            tc5::wait_ld(g);
            if constexpr (C::PAIR) tc5::wait_ld(u);
            if (b == C::BLOCKS - 1) release(ab);
            finish_bf16<C>(p, at, row0, col, lane, buf, g, u, now);
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
  if (warp == C::OUT_WARPS + 1) tc5::dealloc<C::CG>(tm, C::TCOLS);
}

// The parts of tiles that were cut, added in order, and (fp32 pairs) what finish_f32 makes of
// them.  A thread takes 8 columns of the output.
template <class C>
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ GemmParams p) {
  await_before();
  constexpr int VECS = C::OUT_N / 8;
  constexpr int PER = C::BM * VECS / 256;  // CTAs of a tile
  const size_t tile = static_cast<size_t>(C::BM) * C::BN;
  const int t = blockIdx.x / PER, v = blockIdx.x % PER * 256 + threadIdx.x;
  const int r = v / VECS, c = v % VECS * 8;
  const TileAt at = tile_at(p, p.whole + t * p.split);
  const long long row = static_cast<long long>(at.m) * C::BM + r;
  const int col = at.n * C::OUT_N + c;
  if (row >= p.M || col >= p.N) return;
  float s[C::PAIR ? 2 : 1][8] = {};
  for (int i = 0; i < p.split; ++i) {
    const size_t from = (static_cast<size_t>(t) * p.split + i) * tile + static_cast<size_t>(r) * C::BN + c;
#pragma unroll
    for (int w = 0; w < (C::PAIR ? 2 : 1); ++w) {
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (in_range(p.status, from + w * C::OUT_N, 8, tile * p.nparts, CHK_GLU_WS))
        raw_unpack<true, 8>(raw_load<true, 8, false>(p.parts + from + w * C::OUT_N), o);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[w][j] += o[j];
    }
  }
  const size_t to = static_cast<size_t>(row) * p.N + col, extent = static_cast<size_t>(p.M) * p.N;
  if constexpr (C::EPI == EPI_DGLU) {
    float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in_range(p.status, to, 8, extent, CHK_GLU_IN))
      raw_unpack<true, 8>(raw_load<true, 8, false>(static_cast<const float*>(p.in) + to), d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, e;
      act_grad(s[0][j], p.act, a, e);
      s[0][j] = d[j] * s[C::PAIR ? 1 : 0][j] * e;
      s[C::PAIR ? 1 : 0][j] = d[j] * a;
    }
    const size_t plane = static_cast<size_t>(p.M) * p.pitch, at8 = static_cast<size_t>(row) * p.pitch + col;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float& x = s[C::PAIR ? w : 0][j];
          o[j] = bf16_term(x);
          x = isfinite(o[j]) ? x - o[j] : 0.f;
        }
        if (in_range(p.status, (w * 3 + k) * plane + at8, 8, 6 * plane, CHK_GLU_WS))
          store_vec<false, 8>(static_cast<__nv_bfloat16*>(p.out[0]) + (w * 3 + k) * plane + at8, o);
      }
  } else {
    if constexpr (C::EPI == EPI_GLU) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0][j] = act_of(s[0][j], p.act) * s[C::PAIR ? 1 : 0][j];
    }
    if (in_range(p.status, to, 8, extent, CHK_GLU_OUT))
      store_vec<C::F32, 8>(static_cast<typename Elem<C::F32>::T*>(at.batch ? p.out[1] : p.out[0]) + to, s[0]);
  }
}

// (static: the `ready` of another build of the library in the same process is not this one's)
template <class C>
static cudaError_t launch_cfg(const GemmParams& p, int sms, cudaStream_t st) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  const int tiles = p.whole + p.nparts, most = sms / C::CG;
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
  e = cudaLaunchKernelEx(&c, gemm_kernel<C>, p);
  if constexpr (C::EPI == EPI_STORE || C::F32) {
    if (e == cudaSuccess && p.nparts > 0)
      e = launch_after(join_parts_kernel<C>, dim3(C::BM * C::OUT_N / 8 / 256 * (p.nparts / p.split)), 256, 0, st, p);
  }
  return e;
}

}  // namespace m2rnn

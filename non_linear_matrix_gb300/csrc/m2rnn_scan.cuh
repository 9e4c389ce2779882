// m2rnn_scan.cuh -- what the selective scan's kernels share.
//
// The scan  H_t = f_t H_{t-1} + dt_t k_t v_t^T,  y_t = H_t^T q_t + w_r (.) v_t  in chunks of
// 64 tokens.  With l_t = log2 f_t, S(j, i) = sum of l over (j, i] and H the
// state before the chunk,
//
//     y_i = 2^S(start,i) H^T q_i + sum_{j<=i} (q_i.k_j) 2^S(j,i) dt_j v_j  (+ w_r (.) v_i)
//     H'  = 2^S(start,end) H + sum_j 2^S(j,end) dt_j k_j v_j^T
//
// so a chunk is a handful of small matrix products.  Decays are powers of two
// of sums over (j, i] that are formed from sums over 16-token blocks: exact
// to a few 2^-24 of the sum itself, however long the sequence, never as
// differences of two long sums.
//
// Operands.  Products run on the tensor cores in bf16 with fp32 accumulation.
// A value that has more than 8 bits (a state, a decayed product, any fp32
// input) enters as a sum of bf16 terms, largest first: two terms hold 16
// bits (error at most 2^-18 of the value), three hold the whole fp32 value.  A
// product of values with PA and PB terms multiplies the pairs whose sizes
// matter, i + j < max(PA, PB).
//
// Head blocks.  A CTA works on 64 value columns at a time: 64 / V heads of
// one query/key group, which share q and k and the products q_i.k_j.
//
// States are kept transposed, as 8 x 8 blocks (value column, key row) of 128
// contiguous bytes, block (v8, k8) at (v8 K/8 + k8): what an accumulator of
// the state's product holds is a block's row, whole lines are written, and
// both the block and its transpose are operands without bank conflicts.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"
#include "m2rnn_gate.cuh"
#include "m2rnn_vec.cuh"
#include "ptx.cuh"

namespace m2rnn {
namespace scan {

constexpr int kThreads = 128;
constexpr int kVLd = kCols + 8;  // shared row of a value tile: 144 bytes, no bank conflicts
constexpr float kLog2e = 1.4426950408889634f;

template <bool F32>
struct Terms {
  static constexpr int in = F32 ? 3 : 1;     // of an input
  static constexpr int state = F32 ? 3 : 2;  // of a state or a decayed input
  static constexpr int prob = F32 ? 3 : 1;   // of a weight that only meets outputs of in_dtype
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The P bf16 terms of a pair of values, packed.
template <int P>
__device__ __forceinline__ void split(float a, float b, uint32_t (&t)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    t[i] = ptx::pack_bf16x2(a, b);
    if (i + 1 < P) {
      a -= ptx::bf16x2_lo(t[i]);
      b -= ptx::bf16x2_hi(t[i]);
    }
  }
}

// The pair of values that packed terms stand for (exact for an input's terms).
template <int P>
__device__ __forceinline__ float2 join(const uint32_t (&t)[P]) {
  float2 v = make_float2(ptx::bf16x2_lo(t[P - 1]), ptx::bf16x2_hi(t[P - 1]));
#pragma unroll
  for (int i = P - 2; i >= 0; --i) {
    v.x += ptx::bf16x2_lo(t[i]);
    v.y += ptx::bf16x2_hi(t[i]);
  }
  return v;
}

// acc += A B over the terms' pairs that matter, smallest first.
template <int PA, int PB>
__device__ __forceinline__ void mma_terms(float (&acc)[4], const uint32_t (&a)[PA][4],
                                          const uint32_t (&b)[PB][2]) {
  constexpr int most = (PA > PB ? PA : PB) - 1;
#pragma unroll
  for (int s = most; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < PB) ptx::mma_bf16_16816(acc, a[i], b[j][0], b[j][1]);
    }
}

// ---- tiles ------------------------------------------------------------------
//
// A tile holds 64 tokens' rows of up to `width` elements as P planes of
// [64][ld] bf16, ld = width + 8: rows 16 bytes off a multiple of 128 (or 32),
// so eight rows' 16-byte pieces lie in different banks.

// Fills a tile from global rows; rows at or past `rows` and columns at or past
// `cols` become zero.  bf16 by asynchronous copies, fp32 through registers as
// three terms.
template <bool F32>
__device__ __forceinline__ void load_tile(uint32_t dst, const void* src_, long long stride, int rows,
                                          int cols, int width, int ld, int* status, int row_extent) {
  using E = typename Elem<F32>::T;
  const E* src = static_cast<const E*>(src_);
  const int per_row = width / 8;
  for (int e = threadIdx.x; e < kChunk * per_row; e += kThreads) {
    const int r = e / per_row, c = (e - r * per_row) * 8;
    bool on = r < rows && c < cols;
    if (on) on = in_range(status, r, 1, row_extent, CHK_SCAN_IN);
    const uint32_t d = dst + (r * ld + c) * 2;
    const E* s = on ? src + r * stride + c : src;
    if constexpr (!F32) {
      cp_async16_zfill(d, s, on);
    } else {
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (on) load_vec<true, 8>(s, x);
      uint32_t t[4][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) split<3>(x[2 * i], x[2 * i + 1], t[i]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(d + p * kChunk * ld * 2),
                     "r"(t[0][p]), "r"(t[1][p]), "r"(t[2][p]), "r"(t[3][p])
                     : "memory");
    }
  }
}

// Copies `bytes` (a multiple of 16) as they are.
__device__ __forceinline__ void load_linear(uint32_t dst, const void* src, int bytes) {
  for (int e = threadIdx.x * 16; e < bytes; e += kThreads * 16)
    ptx::cp_async16(dst + e, static_cast<const char*>(src) + e);
}

// Address of a lane's row for ldmatrix of the 16 x 16 piece at (r0, c0) of a
// tile: the four 8 x 8 matrices in the order (r0, c0), (r0+8, c0), (r0, c0+8),
// (r0+8, c0+8): as it is, an A operand whose rows are the tile's rows.
__device__ __forceinline__ uint32_t piece_rc(uint32_t tile, int ld, int r0, int c0) {
  const int lane = threadIdx.x & 31;
  return tile + ((r0 + (lane & 15)) * ld + c0 + (lane >> 4) * 8) * 2;
}
// The same with the middle two matrices exchanged: (r0, c0), (r0, c0+8),
// (r0+8, c0), (r0+8, c0+8).  Plain: B operands (contraction along the tile's
// columns) of n = rows r0.. and r0+8..; transposed: an A operand whose rows are
// the tile's columns.
__device__ __forceinline__ uint32_t piece_cr(uint32_t tile, int ld, int r0, int c0) {
  const int lane = threadIdx.x & 31;
  return tile + ((r0 + (lane & 7) + (lane >> 4) * 8) * ld + c0 + ((lane >> 3) & 1) * 8) * 2;
}

template <int P>
__device__ __forceinline__ void load_a(uint32_t (&a)[P][4], uint32_t tile, int ld, int r0, int c0) {
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4(a[p], piece_rc(tile + p * kChunk * ld * 2, ld, r0, c0));
}
// A operand whose rows are the tile's columns c0.. and whose contraction runs
// over the tile's rows r0..
template <int P>
__device__ __forceinline__ void load_a_t(uint32_t (&a)[P][4], uint32_t tile, int ld, int r0, int c0) {
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4_t(a[p], piece_cr(tile + p * kChunk * ld * 2, ld, r0, c0));
}
// B operands, contraction over the tile's columns c0.., n = rows r0.. (first)
// and r0+8.. (second).
template <int P>
__device__ __forceinline__ void load_b2(uint32_t (&b0)[P][2], uint32_t (&b1)[P][2], uint32_t tile,
                                        int ld, int r0, int c0) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t r[4];
    ldsm4(r, piece_cr(tile + p * kChunk * ld * 2, ld, r0, c0));
    b0[p][0] = r[0]; b0[p][1] = r[1]; b1[p][0] = r[2]; b1[p][1] = r[3];
  }
}
// B operands, contraction over the tile's rows r0.., n = columns c0.. (first)
// and c0+8.. (second).
template <int P>
__device__ __forceinline__ void load_b2_t(uint32_t (&b0)[P][2], uint32_t (&b1)[P][2], uint32_t tile,
                                          int ld, int r0, int c0) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t r[4];
    ldsm4_t(r, piece_rc(tile + p * kChunk * ld * 2, ld, r0, c0));
    b0[p][0] = r[0]; b0[p][1] = r[1]; b1[p][0] = r[2]; b1[p][1] = r[3];
  }
}

// B operands from a state's blocks: contraction over key rows 16 ks.., n =
// value columns 8 v8.. and 8 v8 + 8..
template <int P>
__device__ __forceinline__ void state_b2(uint32_t (&b0)[P][2], uint32_t (&b1)[P][2], uint32_t state,
                                         int K, int v8, int ks) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  const uint32_t at = state + (((v8 + (m >> 1)) * (K / 8) + 2 * ks + (m & 1)) * 64 + (lane & 7) * 8) * 2;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t r[4];
    ldsm4(r, at + p * kCols * K * 2);
    b0[p][0] = r[0]; b0[p][1] = r[1]; b1[p][0] = r[2]; b1[p][1] = r[3];
  }
}
// B operands from a state's transposed blocks: contraction over value columns
// 8 v8 .. 8 v8 + 15, n = key rows 8 k8.. and 8 k8 + 8..
template <int P>
__device__ __forceinline__ void state_bt2(uint32_t (&b0)[P][2], uint32_t (&b1)[P][2],
                                          uint32_t state, int K, int v8, int k8) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  const uint32_t at = state + (((v8 + (m & 1)) * (K / 8) + k8 + (m >> 1)) * 64 + (lane & 7) * 8) * 2;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t r[4];
    ldsm4_t(r, at + p * kCols * K * 2);
    b0[p][0] = r[0]; b0[p][1] = r[1]; b1[p][0] = r[2]; b1[p][1] = r[3];
  }
}

// ---- places -------------------------------------------------------------------

struct Place {
  int b, group, hb;  // batch item, query/key group, head block within the group
  int head0, heads;  // first head of the block and how many it has
};
__device__ __forceinline__ Place place_of(const ScanParams& p, int b, int gb) {
  Place w;
  w.b = b;
  w.group = gb / p.nhb;
  w.hb = gb - w.group * p.nhb;
  const int per = kCols / p.V;
  w.head0 = w.group * p.hpg + w.hb * per;
  w.heads = min(per, p.hpg - w.hb * per);
  return w;
}

__device__ __forceinline__ size_t state_at(const ScanParams& p, int terms, int b, int gb, int c) {
  return ((static_cast<size_t>(b) * p.Nq * p.nhb + gb) * p.nc + c) * terms * kCols * p.K;
}

}  // namespace scan
}  // namespace m2rnn

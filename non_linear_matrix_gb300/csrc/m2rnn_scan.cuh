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
// to a few 2^-24 of the sum itself, however long the sequence.  Between blocks only
// sums of parts are formed.  Within a block S(j,i) is a difference of two sums from
// the block's start, which a token that forgets (l near -160) makes large: each is
// held as a rounded sum and what the rounding left, and so is the difference.
//
// Operands.  Products run on the tensor cores (mma.sync) in bf16 with fp32
// accumulation.  A value of more than 8 bits enters as a sum of bf16 terms,
// largest first; three terms hold a whole fp32 value.  A product of values
// with PA and PB terms multiplies the pairs that matter, i + j < max(PA, PB).
// bf16 inputs are one term.  What ends in fp32 (states, gradients of
// parameters) is made from three-term operands, and states enter the readout as
// such.  A weight (and R in dv) that only meets an output rounded to bf16 enters
// with two, 2^-17 of itself and far below that rounding's 2^-9.  With one term,
// states' too, the scan's part of y was off by 2.35e-3 (relative 2-norm) where
// the rounding alone is 1.68e-3, dk and dv likewise; B=1 T=65536 N=64 took 290 us
// instead of 380, with one term for the weights only 325.
//
// Head blocks.  A CTA works on 64 value columns at a time: 64 / V heads of
// one query/key group, which share q and k and the products q_i.k_j.
//
// States are kept transposed, as 8 x 8 blocks (value column, key row), block
// (v8, k8) at (v8 K/8 + k8), fp32 in global memory, bf16 terms of 128
// contiguous bytes in shared memory: what an accumulator of the state's product
// holds is a row of a block, whole lines are written, and both the block and
// its transpose are operands without bank conflicts.
//
// Segments.  Along the chunks the state is a chain.  It is cut into segments
// that run at the same time, each from zero; a small kernel then carries the
// states from segment to segment, and whoever reads a state adds
// 2^S(segment's start, chunk) times the state at the segment's start.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "m2rnn_block.h"
#include "m2rnn_check.cuh"
#include "m2rnn_gate.cuh"
#include "m2rnn_vec.cuh"
#include "ptx.cuh"

namespace m2rnn {
namespace scan {

constexpr int kThreads = 128;  // that fill a tile together
constexpr int kVLd = kCols + 8;  // shared row of a value tile: 144 bytes, no bank conflicts
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLo = static_cast<float>(1.4426950408889634 - kLog2e);

template <bool F32>
struct Terms {
  static constexpr int in = F32 ? 3 : 1;   // of an input
  static constexpr int state = 3;          // of a state or decayed input
  static constexpr int out = F32 ? 3 : 2;  // of a weight that only meets an output
};

__device__ __forceinline__ float2 pair(const float (&x)[4], int half) {
  return make_float2(x[2 * half], x[2 * half + 1]);
}
__device__ __forceinline__ void set_pair(float (&x)[4], int half, float2 v) {
  x[2 * half] = v.x;
  x[2 * half + 1] = v.y;
}

// a + b rounded, and what the rounding left of it (Knuth's two-sum; exact).
__device__ __forceinline__ float two_sum(float a, float b, float& left) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  left = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s;
}

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

// Barrier 1, of `threads` threads: some only announce themselves.
__device__ __forceinline__ void bar_arrive(int threads) {
  asm volatile("bar.arrive 1, %0;" ::"r"(threads) : "memory");
}
__device__ __forceinline__ void bar_wait(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
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

__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// The P bf16 terms of a pair of values, packed.
template <int P>
__device__ __forceinline__ void split(float2 v, uint32_t (&t)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    t[i] = ptx::pack_bf16x2(v.x, v.y);
    // v - term is exact: the sign bit flips in both halves at once
    if (i + 1 < P) {
      const uint32_t n = t[i] ^ 0x80008000u;
      v = add2(v, make_float2(ptx::bf16x2_lo(n), ptx::bf16x2_hi(n)));
    }
  }
}

// Which of two packed bf16 values are infinite or NaN: their sign bits' places.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
}
// The pair with those values replaced by 0.
__device__ __forceinline__ uint32_t finite_only(uint32_t x) {
  return x & ~((not_finite(x) >> 15) * 0xffffu);
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

// A tensor core cuts its sum off where it should round (by 0.37 of the last
// place on average where the accumulator is much larger or smaller than the
// products, 0.05 from zero, measured): a long chain drifts towards zero, and one
// that runs through a state does so from chunk to chunk.  So where both sides
// have three terms, the leading product and the others' sum start from zero and
// are added with rounding, and the states' products start from zero per chunk.

// acc += A B over the terms' pairs that matter, smallest first, for N
// accumulators that share A, term by term across them: a product's result is
// ready about 20 clocks after its issue, so consecutive products go to different
// accumulators.
template <int PA, int PB, int N>
__device__ __forceinline__ void mma_terms_n(float (&acc)[N][4], const uint32_t (&a)[PA][4],
                                            const uint32_t (&b)[N][PB][2]) {
  constexpr int most = (PA > PB ? PA : PB) - 1;
  constexpr bool apart = PA == 3 && PB == 3;
  float top[N][4], rest[N][4];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) top[n][i] = rest[n][i] = 0.f;
#pragma unroll
  for (int s = most; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < PB)
#pragma unroll
        for (int n = 0; n < N; ++n)
          ptx::mma_bf16_16816(!apart ? acc[n] : s == 0 ? top[n] : rest[n], a[i], b[n][j][0], b[n][j][1]);
    }
  if (apart)
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        set_pair(acc[n], h, add2(pair(acc[n], h), add2(pair(top[n], h), pair(rest[n], h))));
}
template <int PA, int PB>
__device__ __forceinline__ void mma_terms(float (&acc)[4], const uint32_t (&a)[PA][4],
                                          const uint32_t (&b)[PB][2]) {
  mma_terms_n<PA, PB, 1>(reinterpret_cast<float(&)[1][4]>(acc), a,
                         reinterpret_cast<const uint32_t(&)[1][PB][2]>(b));
}

// Lets a kernel take `bytes` of dynamic shared memory: asked once per kernel
// and device.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- tiles ------------------------------------------------------------------
//
// A tile holds 64 tokens' rows of up to `width` elements as P planes of
// [64][ld] bf16, ld = width + 8: rows 16 bytes off a multiple of 128 (or 32),
// so eight rows' 16-byte pieces lie in different banks.

// Fills a tile from global rows; rows at or past `rows` and columns at or past
// `cols` become zero.  bf16 by asynchronous copies, fp32 through registers as
// three terms.  tid: the caller's place among kThreads threads.
template <bool F32, int WIDTH>
__device__ __forceinline__ void load_tile(int tid, uint32_t dst, const void* src_, long long stride,
                                          int rows, int cols, int* status, int row_extent) {
  using E = typename Elem<F32>::T;
  constexpr int per_row = WIDTH / 8, ld = WIDTH + 8, step = kThreads / per_row;  // rows per pass
  const int r0 = tid / per_row, c = (tid % per_row) * 8;
  const bool col_on = c < cols;
  const E* src = static_cast<const E*>(src_);
  const E* s = src + r0 * stride + c;
  uint32_t d = dst + (r0 * ld + c) * 2;
#pragma unroll
  for (int i = 0; i < kChunk / step; ++i) {
    const int r = r0 + i * step;
    const bool on = col_on && r < rows && in_range(status, r, 1, row_extent, CHK_SCAN_IN);
    if constexpr (!F32) {
      cp_async16_zfill(d, on ? s : src, on);
    } else {
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (on) load_vec<true, 8>(s, x);
      uint32_t t[4][3];
#pragma unroll
      for (int j = 0; j < 4; ++j) split<3>(make_float2(x[2 * j], x[2 * j + 1]), t[j]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(d + p * kChunk * ld * 2),
                     "r"(t[0][p]), "r"(t[1][p]), "r"(t[2][p]), "r"(t[3][p])
                     : "memory");
    }
    s += step * stride;
    d += step * ld * 2;
  }
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

// The 16-row block of warp w of four.  The blocks differ in causal work and a
// warp's place decides which quarter of its SM it runs on: the order turns from
// CTA to CTA such that the CTAs that an SM holds at a time (152 apart) differ.
__device__ __forceinline__ int row_block(int w) { return (w + (blockIdx.x >> 3)) & 3; }

// ---- places -------------------------------------------------------------------

struct Place {
  int b, group, hb;  // batch item, query/key group, head block within the group
  int head0, heads;  // first head of the block and how many it has
};
// Head block hb of a group (no division: this is done once per head block).
__device__ __forceinline__ Place place_in(const ScanParams& p, int per, int b, int group, int hb) {
  Place w;
  w.b = b;
  w.group = group;
  w.hb = hb;
  w.head0 = group * p.hpg + hb * per;
  w.heads = min(per, p.hpg - hb * per);
  return w;
}
__device__ __forceinline__ Place place_of(const ScanParams& p, int b, int gb) {
  const int group = gb / p.nhb;
  return place_in(p, kCols / p.V, b, group, gb - group * p.nhb);
}

// A segment's first state is the one its predecessor ended with; the first
// segment starts from the given state itself.
struct StateRef {
  const float* own;    // 64 x K, before the chunk, from the segment's start
  size_t at;           // its first element's place
  const float* start;  // 64 x K, at the segment's start (NULL: nothing to add)
  const float* dec;    // [heads * nc]: log2 decay from there, head h's at h * nc
};
// seg: the segment that made the chunk's state.
__device__ __forceinline__ StateRef state_ref(const ScanParams& p, const float* local,
                                              const float* ends, const float* dec, const Place& w,
                                              int c, int seg) {
  const size_t pair = (static_cast<size_t>(w.b) * p.Nq + w.group) * p.nhb + w.hb, tile = kCols * p.K;
  StateRef r;
  r.at = (pair * p.nc + c) * tile;
  r.own = local + r.at;
  r.start = seg == 0 ? nullptr : ends + (pair * p.nseg + seg - 1) * tile;
  r.dec = dec + (static_cast<size_t>(w.b) * p.N + w.head0) * p.nc + c;
  return r;
}

// Eight values of a state (a row of a block), element e of the tile: the loads,
// and apart from them the sum, so that several rows' loads can be in flight.  Plain
// loads, never the read-only path: a kernel that await_before holds back is resident
// while its predecessors still write the states and decays, and a load that
// promises read-only memory may be moved in front of the wait.
struct StateRow {
  float4 a, b, s, t;
  float dec;
};
template <int K, int V>
__device__ __forceinline__ StateRow state_load(const ScanParams& p, const StateRef& r, int e) {
  StateRow x;
  x.a = *reinterpret_cast<const float4*>(r.own + e);
  x.b = reinterpret_cast<const float4*>(r.own + e)[1];
  x.s = x.t = make_float4(0.f, 0.f, 0.f, 0.f);
  x.dec = 0.f;
  if (r.start != nullptr) {
    x.s = *reinterpret_cast<const float4*>(r.start + e);
    x.t = reinterpret_cast<const float4*>(r.start + e)[1];
    x.dec = r.dec[static_cast<size_t>(e / (K * V)) * p.nc];
  }
  return x;
}
__device__ __forceinline__ void state_sum(const StateRow& r, float2 (&x)[4]) {
  const float2 d = both(ex2(r.dec));
  x[0] = make_float2(r.a.x, r.a.y);
  x[1] = make_float2(r.a.z, r.a.w);
  x[2] = make_float2(r.b.x, r.b.y);
  x[3] = make_float2(r.b.z, r.b.w);
  x[0] = fma2(make_float2(r.s.x, r.s.y), d, x[0]);
  x[1] = fma2(make_float2(r.s.z, r.s.w), d, x[1]);
  x[2] = fma2(make_float2(r.t.x, r.t.y), d, x[2]);
  x[3] = fma2(make_float2(r.t.z, r.t.w), d, x[3]);
}

// Asks for a state's own tile to be in L2 by the time it is fetched.
__device__ __forceinline__ void state_prefetch(int tid, const StateRef& r, int n) {
  for (int e = tid * 32; e < n; e += kThreads * 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(r.own + e));
}

// Writes a state row's P terms into the shared tile.
template <int P, int K>
__device__ __forceinline__ void put_state_row(uint32_t tile, int e, const float2 (&x)[4]) {
  uint32_t t[4][P];
#pragma unroll
  for (int j = 0; j < 4; ++j) split<P>(x[j], t[j]);
#pragma unroll
  for (int q = 0; q < P; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tile + (q * kCols * K + e) * 2),
                 "r"(t[0][q]), "r"(t[1][q]), "r"(t[2][q]), "r"(t[3][q])
                 : "memory");
}

// A chunk's gate values of the block's heads: [heads][4][64] floats.
__device__ __forceinline__ void load_gate(int tid, uint32_t dst, const ScanParams& p, const Place& w,
                                          int c) {
  const int o = (tid & 63) * 4;  // 64 threads bring a head's 1,024 bytes
  const size_t extent = static_cast<size_t>(p.B) * p.N * p.nc * kGate;
  for (int h = tid >> 6; h < w.heads; h += kThreads / 64) {
    const size_t at = ((static_cast<size_t>(w.b) * p.N + w.head0 + h) * p.nc + c) * kGate + o;
    if (in_range(p.status, at, 4, extent, CHK_SCAN_WS)) ptx::cp_async16(dst + (h * kGate + o) * 4, p.gate + at);
  }
}

// Two neighbouring values (at an even place).
template <bool F32>
__device__ __forceinline__ float2 load_pair(const typename Elem<F32>::T* src) {
  float2 o[1];
  raw_unpack2<F32, 2>(raw_load<F32, 2>(src), o);
  return o[0];
}

}  // namespace scan
}  // namespace m2rnn

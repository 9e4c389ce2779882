// m2rnn_scan_bwd.cuh -- the gradients of the selective scan, chunk by chunk,
// from the states H before the chunks and the gradients R that reach the
// states after them.  With u_i = dy_i, E_ij = u_i.v_j, G_ij = q_i.k_j and
// L_ij = 2^S(j,i) dt_j for j <= i (0 above):
//
//     dq_i = 2^S(start,i) H u_i + sum_{j<=i} E_ij L_ij k_j         (summed over a group's heads)
//     dk_j = 2^S(j,end) dt_j R v_j + sum_{i>=j} E_ij L_ij q_i      (likewise)
//     dv_j = 2^S(j,end) dt_j R^T k_j + sum_{i>=j} G_ij L_ij u_i + w_r (.) u_j
//
// The decay of token t lies on every path from before t to t or later, so
// with D = E (.) G (.) L and the parts of q_i.dq_i and k_j.dk_j that go through
// the states, Pin_i and Uin_j (per head),
//
//     dl_t = 2^S(start,end) <R, H> + sum_{j<t} Uin_j + sum_{i>=t} Pin_i + sum_{i>=t>j} D_ij
//     da_t = sigmoid(a + beta) ((Uin_t + sum_i D_it) / dt_t - alpha dl_t)
//     dalpha = - sum dt dl,  dbeta = sum da,  dw_r = sum u (.) v
//
// (dl_t: with respect to the natural logarithm of the decay.)  Its last sum is
// formed without differences, which would leave errors of the size of all of D in
// it where the decay is strong: block by block of 16 tokens, from D's row sums and
// column sums over whole blocks, and within t's own block as [i >= t] D^T on the
// tensor cores (D in three terms), summed over j < t.
//
// A CTA takes one chunk of one group and walks over its head blocks: dq and
// dk, and the sum over heads of E L, stay with it, so neither needs a sum over
// CTAs (unless the head blocks are shared out, then their shares are added in
// order).  Eight warps in two sides.  Warps 0 to 3 take dq and dk through the
// states, 32 rows x half of the K columns each (a state's operand then serves two
// products, and the shared-memory pipe is what this kernel loads most), <R, H>,
// dw_r and the gate; warps 4 to 7 dv and everything within the chunk, 16 rows j
// each, and the fetching of the next head block.  G and the sum of E L wait in
// shared memory, in the order of the accumulators' lanes (in registers they
// spilled: 336 us instead of 245).  The products within the chunk are formed with j
// along the rows, which leaves G L in the registers as the A operand of dv.
// Between different 16-token blocks L is a product of a row's and a column's
// factor, as in the forward pass.  States enter with three bf16 terms where a
// value that stays in fp32 depends on them (dl) and with two for dv.
//
// Bound by latency and the shared-memory pipe (54 % of its cycles; 37 % of issue
// slots, 18 % of the tensor pipe's): B=8 T=4096 N=32 K=64 V=16 takes 250 us (235 with
// one-term weights).  An earlier state of it, 248 us, took 173 without the products within the chunk,
// 206 without the fetching, 222 without the states' side and 241 without the gate.
// The chunk's side is uneven (row block 0 has four blocks, row block 3 one), yet
// handing one over to row block 3's warp gained nothing (269 us: more spills).
#pragma once
#include "m2rnn_scan.cuh"

namespace m2rnn {
namespace scan {
namespace {

template <bool F32, int KT, int V>
struct BwdSmem {
  static constexpr int P = Terms<F32>::in, PS = Terms<F32>::state, K = 8 * KT, HB = kCols / V;
  static constexpr int key = P * kChunk * (K + 8) * 2, val = P * kChunk * kVLd * 2;
  static constexpr int state = PS * kCols * K * 2;
  static constexpr int tri = 20 * 512;  // G, or the sum of E L: 8 - 2 rt tiles of row block rt
  static constexpr int q = 0, k = q + key, v = k + key, u = v + val, h = u + val;
  static constexpr int r = F32 ? h : h + state;  // fp32: R takes H's place
  static constexpr int KH = KT >= 4 ? 2 : 1;     // parts that the K columns are cut into
  static constexpr int g = r + state, f = g + tri;
  static constexpr int gate = f + (F32 ? 0 : tri);  // fp32 keeps the sum in registers
  // Per head and token, from the first half of the K columns: Pin, Uin [HB][64];
  // column sums of D by row block rt: in the columns of its own block the sums over
  // i >= t > j, then the later blocks' column sums; shares of <R, H>.  What else
  // there is per head and token has its place in the 16 bytes behind the tiles' rows
  // (see spare).
  static constexpr int through = gate + HB * kGate * 4;
  static constexpr int cols = through + 2 * HB * kChunk * 4;
  static constexpr int rh = cols + 160 * HB * 4;
  static constexpr int bytes = rh + 32 * 4;
};

__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// d (16 x 8) += A (16 x 8, a0: rows 0..7, a1: 8..15) B (8 x 8).
__device__ __forceinline__ void mma_bf16_1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(b));
}

// Two neighbouring values of an output in its element type.
template <bool F32>
__device__ __forceinline__ void store2(typename Elem<F32>::T* dst, float a, float b) {
  if constexpr (F32)
    *reinterpret_cast<float2*>(dst) = make_float2(a, b);
  else
    *reinterpret_cast<uint32_t*>(dst) = ptx::pack_bf16x2(a, b);
}

template <bool F32, int KT, int V>
__global__ void __launch_bounds__(2 * kThreads, F32 || KT == 16 ? 1 : 2) bwd_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  using S = BwdSmem<F32, KT, V>;
  constexpr int P = S::P, PS = S::PS, PO = Terms<F32>::out, K = S::K, HB = S::HB, NT = V / 8;
  constexpr int ld = K + 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = ptx::smem_addr(smem);
  const uint32_t qs = base + S::q, ks = base + S::k, vs = base + S::v, us = base + S::u,
                 hs = base + S::h, rs = base + S::r;
  const float* gate = reinterpret_cast<const float*>(smem + S::gate);
  float* Pin = reinterpret_cast<float*>(smem + S::through);
  float* Uin = Pin + HB * kChunk;
  float* rh = reinterpret_cast<float*>(smem + S::rh);
  float* Pcol = reinterpret_cast<float*>(smem + S::cols);  // see col_at
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
  const int rt = row_block(warp & 3);                  // its 16 rows (the chunk's side)
  const bool sside = warp < 4;                         // the states' side
  const int tid = threadIdx.x & (kThreads - 1);        // within the side
  // column i of row block r's sums for head h (columns 16 r and on)
  auto col_at = [&](int r, int h, int i) { return HB * (r * 64 - 8 * r * (r - 1)) + h * (64 - 16 * r) + i - 16 * r; };
  const int c = blockIdx.x % p.nc;
  const int rest = blockIdx.x / p.nc, share = rest % p.hsplit;
  const int group = (rest / p.hsplit) % p.Nq, b = rest / p.hsplit / p.Nq;
  const int t0 = c * kChunk, rows = min(kChunk, p.T - t0);
  const int per = (p.nhb + p.hsplit - 1) / p.hsplit;
  const int hb0 = share * per, hb1 = min(p.nhb, hb0 + per);
  const E* q = static_cast<const E*>(p.q) + b * p.qb + t0 * p.qt + static_cast<size_t>(group) * K;
  const E* k = static_cast<const E*>(p.k) + b * p.kb + t0 * p.kt + static_cast<size_t>(group) * K;
  if (sside) {
    load_tile<F32, K>(tid, qs, q, p.qt, rows, K, p.status, p.T - t0);
    load_tile<F32, K>(tid, ks, k, p.kt, rows, K, p.status, p.T - t0);
    ptx::cp_async_commit();
  }

  const size_t st_extent = static_cast<size_t>(p.B) * p.Nq * p.nhb * p.nc * kCols * K;
  const size_t tok_extent = static_cast<size_t>(p.B) * p.T * p.N;  // tokens x heads
  const long long ut = static_cast<long long>(p.N) * V;
  const int hseg = c / p.cps, rseg = (p.nc - 1 - c) / p.cps;
  auto ref_h = [&](const Place& w) { return state_ref(p, p.Hl, p.Hseg, p.cdec, w, c, hseg); };
  auto ref_r = [&](const Place& w) { return state_ref(p, p.Rl, p.Rseg, p.rdec, w, c, rseg); };
  // `threads` threads bring a state's tile, two rows each in flight.
  auto fetch_state = [&](int thread, int threads, uint32_t dst, const StateRef& r,
                         int n) {
    constexpr int U = 2;
    const int step = threads * 8;
#pragma unroll 1
    for (int e0 = thread * 8; e0 < n; e0 += U * step) {
      StateRow x[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * step;
        on[u] = e < n && in_range(p.status, r.at + e, 8, st_extent, CHK_SCAN_WS);
        if (on[u]) x[u] = state_load<K, V>(p, r, e);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on[u]) {
          float2 z[4];
          state_sum(x[u], z);
          put_state_row<PS, K>(dst, e0 + u * step, z);
        }
    }
  };
  auto fetch_h = [&](int hb, int thread, int threads) {
    const Place w = place_in(p, HB, b, group, hb);
    fetch_state(thread, threads, hs, ref_h(w), w.heads * V * K);
  };
  auto fetch_rest = [&](int hb) {
    const Place w = place_in(p, HB, b, group, hb);
    const E* v = static_cast<const E*>(p.v) + b * p.vb + t0 * p.vt + static_cast<size_t>(w.head0) * V;
    const E* u = static_cast<const E*>(p.dy) + (static_cast<size_t>(b) * p.T + t0) * ut +
                 static_cast<size_t>(w.head0) * V;
    load_tile<F32, kCols>(tid, vs, v, p.vt, rows, w.heads * V, p.status, p.T - t0);
    load_tile<F32, kCols>(tid, us, u, ut, rows, w.heads * V, p.status, p.T - t0);
    load_gate(tid, base + S::gate, p, w, c);
    ptx::cp_async_commit();
    if (!F32) fetch_state(tid, kThreads, rs, ref_r(w), w.heads * V * K);
  };
  // fp32: R in H's place, and <R, H> with H from memory, in shares of 256
  // elements (a warp's pass).
  auto fetch_r_late = [&](int hb) {
    const Place w = place_in(p, HB, b, group, hb);
    const StateRef fh = ref_h(w), fr = ref_r(w);
#pragma unroll 1
    for (int e = tid * 8; e < w.heads * V * K; e += kThreads * 8) {
      // (a warp's 256 elements together: its lanes sum below)
      if (!in_range(p.status, fh.at + e / 256 * 256, 256, st_extent, CHK_SCAN_WS)) continue;
      const StateRow xr = state_load<K, V>(p, fh, e), yr = state_load<K, V>(p, fr, e);
      float2 x[4], y[4];
      state_sum(xr, x);
      state_sum(yr, y);
      put_state_row<PS, K>(rs, e, y);
      const float2 d = fma2(x[0], y[0], fma2(x[1], y[1], fma2(x[2], y[2], mul2(x[3], y[3]))));
      float s = d.x + d.y;
#pragma unroll
      for (int m = 16; m >= 1; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (lane == 0) rh[e / 256] = s;
    }
  };
  // The 16 bytes behind each row of a tile keep bank conflicts away and hold one
  // value per head: the second half's shares of Pin (u) and Uin (v), the row
  // sums of D over later blocks (q) and over the row's own block (k).
  auto spare = [&](int tile, int width, int h, int row) {
    return reinterpret_cast<float*>(smem + tile + (row * (width + 8) + width) * 2) + h;
  };
  let_next_begin();
  await_before();  // (q and k are inputs)
  if (sside) {
    fetch_h(hb0, tid, kThreads);
    cp_async_wait<0>();
  } else {
    fetch_rest(hb0);
  }
  __syncthreads();

  const E* w_r = static_cast<const E*>(p.w_r);
  float* part = p.part + (static_cast<size_t>(b) * p.nc + c) * p.N * (2 + V);
  const size_t part_extent = static_cast<size_t>(p.N) * (2 + V);
  if (sside) {
    constexpr int KH = S::KH, NK = KT / KH;  // column tiles of a warp
    const int row0 = 32 * (warp & 1), n0 = NK * (warp >> 1);
    const bool works = (warp >> 1) < KH;     // K = 16 has one part only
    float dq[2][NK][4], dk[2][NK][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int nt = 0; nt < NK; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[m][nt][i] = dk[m][nt][i] = 0.f;
    // Through a state: out += scale_row (A state^T), and the rows' products with
    // `with`'s rows (q or k), for one head; scale[m]: of rows 16 m + g, + 8.
    auto through = [&](int tile_at, uint32_t state, uint32_t with, int h, const float2 (&scale)[2],
                       float (&out)[2][NK][4], float* sums) {
      const uint32_t tile = base + tile_at;
      uint32_t a[2][V / 16][P][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int vv = 0; vv < V / 16; ++vv)
          load_a<P>(a[m][vv], tile, kVLd, row0 + 16 * m, h * V + 16 * vv);
      float d[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int nt = 0; nt < NK; nt += 2) {
        uint32_t bb[V / 16][2][PS][2];
#pragma unroll
        for (int vv = 0; vv < V / 16; ++vv)
          state_bt2<PS>(bb[vv][0], bb[vv][1], state, K, h * NT + 2 * vv, n0 + nt);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int vv = 0; vv < V / 16; ++vv) mma_terms_n<P, PS, 2>(x, a[m][vv], bb[vv]);
          uint32_t y[P][4];
          load_a<P>(y, with, ld, row0 + 16 * m, 8 * (n0 + nt));
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // (row g, tile nt), (g + 8, nt), (g, nt + 1), (g + 8, nt + 1)
            uint32_t t[P];
#pragma unroll
            for (int s = 0; s < P; ++s) t[s] = y[s][r];
            const float2 z = pair(x[r >> 1], r & 1), f = join<P>(t);
            float(&o)[4] = out[m][nt + (r >> 1)];
            set_pair(o, r & 1, fma2(both((r & 1) ? scale[m].y : scale[m].x), z, pair(o, r & 1)));
            d[m][r & 1] = fmaf(f.x, z.x, fmaf(f.y, z.y, d[m][r & 1]));
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float y0 = quad_sum(d[m][0]) * scale[m].x, y1 = quad_sum(d[m][1]) * scale[m].y;
        const int r = row0 + 16 * m + g;
        if ((lane & 3) == 0) {
          if (n0 == 0) {
            sums[h * kChunk + r] = y0;
            sums[h * kChunk + r + 8] = y1;
          } else {
            *spare(tile_at, kCols, h, r) = y0;
            *spare(tile_at, kCols, h, r + 8) = y1;
          }
        }
      }
    };
    for (int hb = hb0; hb < hb1; ++hb) {
      const Place w = place_in(p, HB, b, group, hb);
      __syncthreads();  // the head block is there
      if (hb + 1 < hb1) {
        const Place next = place_in(p, HB, b, group, hb + 1);
        state_prefetch(tid, ref_h(next), next.heads * V * K);
      }
      // the gate of head `warp`: 2^S(start,end), and its two tokens' parts
      float decay = 0.f, alpha = 0.f, dt[2], sg[2], ratio[2];
      if (warp < w.heads) {
        const int n = w.head0 + warp;
        const float* lo = gate + warp * kGate;
        decay = ex2((lo[15] + lo[31]) + (lo[47] + lo[63]));
        const E* a = static_cast<const E*>(p.a) + b * p.ab + n;
        alpha = to_f32(static_cast<const E*>(p.alpha)[n]);
        const float beta = to_f32(static_cast<const E*>(p.beta)[n]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
          if (2 * lane + e < rows && in_range(p.status, t0 + 2 * lane + e, 1, p.T, CHK_SCAN_IN))
            x = to_f32(a[(t0 + 2 * lane + e) * p.at]) + beta;
          dt[e] = gate_softplus(x);
          sg[e] = 1.f / (1.f + expf(-x));
          // sigmoid / softplus -> 1 as both vanish; a token with dt = 0 has no part of U
          ratio[e] = dt[e] > 0.f ? sg[e] / dt[e] : 1.f;
        }
      }
      if (works) {
#pragma unroll 1
        for (int h = 0; h < w.heads; ++h) {  // dq through H: 2^S(start,i)
          const float* lo = gate + h * kGate;
          float2 sc[2];
          float off = row0 ? lo[15] + lo[31] : 0.f;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sc[m] = make_float2(ex2(off + lo[row0 + 16 * m + g]), ex2(off + lo[row0 + 16 * m + g + 8]));
            off += lo[row0 + 15];
          }
          through(S::u, hs, qs, h, sc, dq, Pin);
        }
      }
      // dw_r: the diagonal of u^T v over the chunk, 16 columns per warp
      if (w_r != nullptr && 16 * warp < w.heads * V) {
        float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t a[P][4], b0[P][2], b1[P][2];
          load_a_t<P>(a, us, kVLd, 16 * s, 16 * warp);
          load_b2_t<P>(b0, b1, vs, kVLd, 16 * s, 16 * warp);
          mma_terms<P, P>(x0, a, b0);
          mma_terms<P, P>(x1, a, b1);
        }
        const size_t at = 2 * static_cast<size_t>(p.N) + static_cast<size_t>(w.head0) * V + 16 * warp + g;
        if ((lane & 3) == (g >> 1) && in_range(p.status, at, 9, part_extent, CHK_SCAN_PARAM)) {
          part[at] = (g & 1) ? x0[1] : x0[0];
          part[at + 8] = (g & 1) ? x1[3] : x1[2];
        }
      }
      if constexpr (F32) {  // R in H's place
        __syncthreads();
        __syncthreads();
      } else if (16 * warp < w.heads * V) {  // <R, H> of the warp's 16 columns: the diagonal of H^T R
        float z[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < KT / 2; ++kk) {
          uint32_t a[PS][4], bb[2][PS][2];
          const int m = lane >> 3;
          const uint32_t at = hs + (((2 * warp + (m & 1)) * KT + 2 * kk + (m >> 1)) * 64 + (lane & 7) * 8) * 2;
#pragma unroll
          for (int s = 0; s < PS; ++s) ldsm4(a[s], at + s * kCols * K * 2);
          state_b2<PS>(bb[0], bb[1], rs, K, 2 * warp, kk);
          mma_terms_n<PS, PS, 2>(z, a, bb);
        }
        float s = 0.f;
        if ((lane & 3) == (g >> 1)) s = (g & 1) ? z[0][1] + z[1][3] : z[0][0] + z[1][2];
#pragma unroll
        for (int m = 16; m >= 1; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (lane == 0) rh[warp] = s;
      }
      if (!F32) bar_arrive(2 * kThreads);  // done with H
      if (works) {
#pragma unroll 1
        for (int h = 0; h < w.heads; ++h) {  // dk through R: 2^S(j,end) dt_j
          const float* lo = gate + h * kGate;
          float2 sc[2];
          float off = row0 ? 0.f : lo[47] + lo[63];
#pragma unroll
          for (int m = 1; m >= 0; --m) {
            const float f = ex2(off);
            sc[m] = make_float2(lo[128 + row0 + 16 * m + g] * f, lo[128 + row0 + 16 * m + g + 8] * f);
            off += lo[row0 + 31];
          }
          through(S::v, rs, ks, h, sc, dk, Uin);
        }
      }
      __syncthreads();  // done with it; the others' sums are there
      if (F32 && hb + 1 < hb1) fetch_h(hb + 1, tid, kThreads);
      if (warp < w.heads) {  // the gate: one warp per head, two tokens per lane
        const int h = warp, n = w.head0 + h, t = 2 * lane, blk = lane >> 3;
        float2 ui = *reinterpret_cast<const float2*>(Uin + h * kChunk + t);
        float2 pi = *reinterpret_cast<const float2*>(Pin + h * kChunk + t);
        if (KH == 2) {
          ui = add2(ui, make_float2(*spare(S::v, kCols, h, t), *spare(S::v, kCols, h, t + 1)));
          pi = add2(pi, make_float2(*spare(S::u, kCols, h, t), *spare(S::u, kCols, h, t + 1)));
        }
        // sums of D over a token's own block (from itself on) and the later ones, and
        // what earlier blocks' columns hold for it
        const float2 own = make_float2(*spare(S::k, K, h, t), *spare(S::k, K, h, t + 1));
        const float2 later = make_float2(*spare(S::q, K, h, t), *spare(S::q, K, h, t + 1));
        const float2 within = *reinterpret_cast<const float2*>(Pcol + col_at(blk, h, t));
        float2 bw = pi;
        float far[4];  // for the tokens of block 0..3: the parts of tokens of other blocks
        far[0] = blk > 0 ? pi.x + pi.y : 0.f;
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          if (s < blk) bw = add2(bw, *reinterpret_cast<const float2*>(Pcol + col_at(s, h, t)));
          far[s + 1] = blk < s + 1 ? ui.x + ui.y : blk > s + 1 ? bw.x + bw.y : 0.f;
        }
        {  // their sums, a lane its own block's
          const bool b4 = lane & 16, b3 = lane & 8;
          float x = b4 ? far[2] : far[0], y = b4 ? far[3] : far[1];
          x += __shfl_xor_sync(0xffffffffu, b4 ? far[0] : far[2], 16);
          y += __shfl_xor_sync(0xffffffffu, b4 ? far[1] : far[3], 16);
          far[0] = b3 ? y : x;
          far[0] += __shfl_xor_sync(0xffffffffu, b3 ? x : y, 8);
#pragma unroll
          for (int m = 4; m >= 1; m /= 2) far[0] += __shfl_xor_sync(0xffffffffu, far[0], m);
        }
        const float2 fw = add2(ui, later);
        float inc = fw.x + fw.y, suf = bw.x + bw.y;
#pragma unroll
        for (int d = 1; d < 8; d *= 2) {
          const float up = __shfl_up_sync(0xffffffffu, inc, d, 8);
          const float dn = __shfl_down_sync(0xffffffffu, suf, d, 8);
          if ((lane & 7) >= d) inc += up;
          if ((lane & 7) + d < 8) suf += dn;
        }
        float before = __shfl_up_sync(0xffffffffu, inc, 1, 8), behind = __shfl_down_sync(0xffffffffu, suf, 1, 8);
        if ((lane & 7) == 0) before = 0.f;
        if ((lane & 7) == 7) behind = 0.f;
        constexpr int shares = F32 ? K * V / 256 : V / 16;
        float all = 0.f;
#pragma unroll
        for (int e = 0; e < shares; ++e) all += rh[h * shares + e];
        all = fmaf(all, decay, far[0]);
        const float dl[2] = {all + within.x + before + (behind + bw.y + bw.x),
                             all + within.y + (before + fw.x) + (behind + bw.y)};
        const float uu[2] = {fw.x + own.x, fw.y + own.y};
        float sa = 0.f, sb = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (t + e >= rows) continue;
          const float da = fmaf(ratio[e], uu[e], -alpha * sg[e] * dl[e]);
          sa = fmaf(-dt[e], dl[e], sa);
          sb += da;
          const size_t at = (static_cast<size_t>(b) * p.T + t0 + t + e) * p.N + n;
          if (in_range(p.status, at, 1, tok_extent, CHK_SCAN_OUT)) {
            if constexpr (F32)
              static_cast<float*>(p.da)[at] = da;
            else
              static_cast<__nv_bfloat16*>(p.da)[at] = __float2bfloat16_rn(da);
          }
        }
#pragma unroll
        for (int m = 16; m >= 1; m /= 2) {
          sa += __shfl_xor_sync(0xffffffffu, sa, m);
          sb += __shfl_xor_sync(0xffffffffu, sb, m);
        }
        if (lane == 0 && in_range(p.status, p.N + n, 1, part_extent, CHK_SCAN_PARAM)) {
          part[n] = sa;
          part[p.N + n] = sb;
        }
      }
    }
    __syncthreads();
    __syncthreads();  // the sum of E L is there
    if (!works) return;
    // dq and dk within the chunk
    const size_t qk_extent = static_cast<size_t>(p.B) * p.T * p.Nq * K;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int rb = (row0 >> 4) + m;  // 16-row block
#pragma unroll 1
      for (int jb = 0; jb <= rb; ++jb) {
        uint32_t a[PO][4];
        load_a_t<PO>(a, vs, kVLd, 16 * jb, 16 * rb);
#pragma unroll
        for (int nt = 0; nt < NK; nt += 2) {
          uint32_t b0[P][2], b1[P][2];
          load_b2_t<P>(b0, b1, ks, ld, 16 * jb, 8 * (n0 + nt));
          mma_terms<PO, P>(dq[m][nt], a, b0);
          mma_terms<PO, P>(dq[m][nt + 1], a, b1);
        }
      }
#pragma unroll 1
      for (int ib = rb; ib < 4; ++ib) {
        uint32_t a[PO][4];
        load_a<PO>(a, vs, kVLd, 16 * rb, 16 * ib);
#pragma unroll
        for (int nt = 0; nt < NK; nt += 2) {
          uint32_t b0[P][2], b1[P][2];
          load_b2_t<P>(b0, b1, qs, ld, 16 * ib, 8 * (n0 + nt));
          mma_terms<PO, P>(dk[m][nt], a, b0);
          mma_terms<PO, P>(dk[m][nt + 1], a, b1);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NK; ++nt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int r = row0 + 16 * m + g + 8 * hh;
          const size_t at = ((static_cast<size_t>(b) * p.T + t0 + r) * p.Nq + group) * K + 8 * (n0 + nt) + c2;
          if (r >= rows || !in_range(p.status, at, 2, qk_extent, CHK_SCAN_OUT)) continue;
          if (p.hsplit > 1) {
            float* dst = p.dqk + static_cast<size_t>(share) * 2 * qk_extent + at;
            *reinterpret_cast<float2*>(dst) = pair(dq[m][nt], hh);
            *reinterpret_cast<float2*>(dst + qk_extent) = pair(dk[m][nt], hh);
          } else {
            store2<F32>(static_cast<E*>(p.dq) + at, dq[m][nt][2 * hh], dq[m][nt][2 * hh + 1]);
            store2<F32>(static_cast<E*>(p.dk) + at, dk[m][nt][2 * hh], dk[m][nt][2 * hh + 1]);
          }
        }
    }
    return;
  }

  // Tile n of the row block (columns 16 rt + 8 n..) of G and of the sum of E L.
  const int rb = 16 * rt;
  float4* gt = reinterpret_cast<float4*>(smem + S::g) + rt * (9 - rt) * 32 + lane;
  float4* ft = reinterpret_cast<float4*>(smem + S::f) + rt * (9 - rt) * 32 + lane;
  // G with j along the rows, for the tiles with i >= j
#pragma unroll 1
  for (int k4 = 0; rt + k4 < 4; ++k4) {
    float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KT / 2; ++kk) {
      uint32_t a[P][4], b0[P][2], b1[P][2];
      load_a<P>(a, ks, ld, rb, 16 * kk);
      load_b2<P>(b0, b1, qs, ld, rb + 16 * k4, 16 * kk);
      mma_terms<P, P>(x0, a, b0);
      mma_terms<P, P>(x1, a, b1);
    }
    gt[64 * k4] = make_float4(x0[0], x0[1], x0[2], x0[3]);
    gt[64 * k4 + 32] = make_float4(x1[0], x1[1], x1[2], x1[3]);
    if (!F32) ft[64 * k4] = ft[64 * k4 + 32] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  E* dv_out = static_cast<E*>(p.dv) + ((static_cast<size_t>(b) * p.T + t0 + rb + g) * p.N +
                                       static_cast<size_t>(group) * p.hpg) * V + c2;
  const size_t dv_8 = 8 * static_cast<size_t>(p.N) * V;  // 8 rows further on
  float* pcol = Pcol + HB * (rt * 64 - 8 * rt * (rt - 1)) + c2;
  const int pcol_h = 64 - rb;
  float dsum[8][4];  // sum over heads of E L, tile n (fp32)
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) dsum[nt][i] = 0.f;
  for (int hb = hb0; hb < hb1; ++hb) {
    const Place w = place_in(p, HB, b, group, hb);
    cp_async_wait<0>();
    __syncthreads();
    if (F32) {  // R in H's place
      __syncthreads();
      fetch_r_late(hb);
      __syncthreads();
    }
    if (hb + 1 < hb1) {
      const Place next = place_in(p, HB, b, group, hb + 1);
      state_prefetch(tid, ref_r(next), next.heads * V * K);
    }
#pragma unroll 1
    for (int h = 0; h < w.heads; ++h) {
      const float* lo = gate + h * kGate;
      const float* lj = lo + rb + g;                   // of rows g; g + 8 further on the others
      const float end0 = lj[128], end1 = lj[128 + 8];  // 2^S(j, block's end) dt_j
      float w0, w1;                                    // 2^S(j, end) dt_j
      {
        float off = 0.f;
        for (int i4 = rt + 1; i4 < 4; ++i4) off += lo[16 * i4 + 15];
        off = ex2(off);
        w0 = end0 * off;
        w1 = end1 * off;
      }
      // dv through R
      float dv[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) dv[nt][i] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KT / 2; ++kk) {
        uint32_t a[P][4];
        load_a<P>(a, ks, ld, 16 * rt, 16 * kk);
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
          uint32_t b0[PO][2], b1[PO][2];
          state_b2<PO>(b0, b1, rs, K, h * NT + nt, kk);
          mma_terms<P, PO>(dv[nt], a, b0);
          mma_terms<P, PO>(dv[nt + 1], a, b1);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        set_pair(dv[nt], 0, mul2(pair(dv[nt], 0), both(w0)));
        set_pair(dv[nt], 1, mul2(pair(dv[nt], 1), both(w1)));
      }
      // within the chunk
      uint32_t va[V / 16][P][4];
#pragma unroll
      for (int vv = 0; vv < V / 16; ++vv) load_a<P>(va[vv], vs, kVLd, 16 * rt, h * V + 16 * vv);
      float2 ur0 = make_float2(0.f, 0.f), ur1 = ur0;  // row sums of D over later blocks
      float* ph = pcol + h * pcol_h;
      const float* li_at = lo + rb + c2;
      float between = 0.f;  // sum of l over the blocks between j's and i's
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {  // columns i of block rt + k4
        if (rt + k4 > 3) break;
        if (k4 > 1) between += lo[rb + 16 * k4 - 1];
        float e[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int vv = 0; vv < V / 16; ++vv) {
          uint32_t b0[P][2], b1[P][2];
          load_b2<P>(b0, b1, us, kVLd, rb + 16 * k4, h * V + 16 * vv);
          mma_terms<P, P>(e[0], va[vv], b0);
          mma_terms<P, P>(e[1], va[vv], b1);
        }
        uint32_t a[PO][4];
        float2 dc[2];
        float z0[4] = {0.f, 0.f, 0.f, 0.f}, z1[4] = {0.f, 0.f, 0.f, 0.f};  // j < 8, j >= 8
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int n = 2 * k4 + u;
          const float2 li = *reinterpret_cast<const float2*>(li_at + 8 * n);
          const float4 g4 = gt[32 * n];
          const float2 g0 = make_float2(g4.x, g4.y), g1 = make_float2(g4.z, g4.w);
          float2 l0, l1;
          if (k4 == 0) {
            const float lj0 = lj[0], lj1 = lj[8], ej0 = lj[192], ej1 = lj[192 + 8];
            const float2 ei = *reinterpret_cast<const float2*>(li_at + 192 + 8 * n);
            l0 = mul2(make_float2(ex2((li.x - lj0) + (ei.x - ej0)), ex2((li.y - lj0) + (ei.y - ej0))), both(lj[64]));
            l1 = mul2(make_float2(ex2((li.x - lj1) + (ei.x - ej1)), ex2((li.y - lj1) + (ei.y - ej1))), both(lj[64 + 8]));
            const int i = 8 * u + c2;  // i >= j
            l0.x = i >= g ? l0.x : 0.f;
            l0.y = i + 1 >= g ? l0.y : 0.f;
            l1.x = i >= g + 8 ? l1.x : 0.f;
            l1.y = i + 1 >= g + 8 ? l1.y : 0.f;
          } else {
            const float2 s = add2(li, both(between));
            const float2 r = make_float2(ex2(s.x), ex2(s.y));
            l0 = mul2(r, both(end0));
            l1 = mul2(r, both(end1));
          }
          const float2 f0 = mul2(pair(e[u], 0), l0), f1 = mul2(pair(e[u], 1), l1);
          if (F32) {
            set_pair(dsum[n], 0, add2(pair(dsum[n], 0), f0));
            set_pair(dsum[n], 1, add2(pair(dsum[n], 1), f1));
          } else {
            const float4 s = ft[32 * n];
            const float2 s0 = add2(make_float2(s.x, s.y), f0), s1 = add2(make_float2(s.z, s.w), f1);
            ft[32 * n] = make_float4(s0.x, s0.y, s1.x, s1.y);
          }
          const float2 d0 = mul2(f0, g0), d1 = mul2(f1, g1);
          if (k4 == 0) {
            // sum of D over i >= t > j in the block: z = [i >= t] D^T, then row t's sum
            // over j < t; D is 0 for j >= 8 > i.  Row t = 0 of z is D's row sums.
            const uint32_t tri = (c2 >= g ? 0x3f80u : 0u) | (c2 + 1 >= g ? 0x3f800000u : 0u);
            uint32_t x[3];
            split<3>(d0, x);
#pragma unroll
            for (int s = 2; s >= 0; --s) mma_bf16_1688(z0, u ? 0x3f803f80u : tri, u ? tri : 0u, x[s]);
            if (u) {
              split<3>(d1, x);
#pragma unroll
              for (int s = 2; s >= 0; --s) mma_bf16_1688(z1, 0x3f803f80u, tri, x[s]);
            }
          } else {
            ur0 = add2(ur0, d0);
            ur1 = add2(ur1, d1);
            dc[u] = add2(d0, d1);
          }
          uint32_t x0[PO], x1[PO];
          split<PO>(mul2(g0, l0), x0);
          split<PO>(mul2(g1, l1), x1);
#pragma unroll
          for (int s = 0; s < PO; ++s) {
            a[s][2 * u] = x0[s];
            a[s][2 * u + 1] = x1[s];
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
          uint32_t b0[P][2], b1[P][2];
          load_b2_t<P>(b0, b1, us, kVLd, rb + 16 * k4, h * V + 8 * nt);
          mma_terms<PO, P>(dv[nt], a, b0);
          mma_terms<PO, P>(dv[nt + 1], a, b1);
        }
        if (k4 == 0) {
          const bool b0 = lane & 1;
          const float x = (c2 < g ? z0[0] : 0.f) + (c2 + 1 < g ? z0[1] : 0.f);
          const float y = (z0[2] + z0[3]) + ((c2 < g ? z1[2] : 0.f) + (c2 + 1 < g ? z1[3] : 0.f));
          float t = b0 ? y : x;
          t += __shfl_xor_sync(0xffffffffu, b0 ? x : y, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          if (!(lane & 2)) ph[g - c2 + (b0 ? 8 : 0)] = t;
          if (g == 0) {
            float* own = spare(S::k, K, h, rb + c2);
            constexpr int row = ld / 2;  // floats
            own[0] = z0[0];
            own[row] = z0[1];
            own[8 * row] = z1[0];
            own[9 * row] = z1[1];
          }
        } else {  // the column sums: 4 values over the 8 lanes that share lane mod 4
          const bool b4 = lane & 16, b3 = lane & 8;
          float2 s = b4 ? dc[1] : dc[0], o = b4 ? dc[0] : dc[1];
          s.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
          s.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
          float t = b3 ? s.y : s.x;
          t += __shfl_xor_sync(0xffffffffu, b3 ? s.x : s.y, 8);
          t += __shfl_xor_sync(0xffffffffu, t, 4);
          if (!(lane & 4)) ph[16 * k4 + (b4 ? 8 : 0) + (b3 ? 1 : 0)] = t;
        }
      }
      {  // the row sums: 2 values over 4 lanes
        const bool b0 = lane & 1;
        const float u0 = ur0.x + ur0.y, u1 = ur1.x + ur1.y;
        float t = b0 ? u1 : u0;
        t += __shfl_xor_sync(0xffffffffu, b0 ? u0 : u1, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        if (!(lane & 2)) *spare(S::q, K, h, rb + g + (b0 ? 8 : 0)) = t;
      }
      // dv, with w_r (.) u
      const int hv = (hb * HB + h) * V;
#pragma unroll
      for (int nt = 0; nt < NT; nt += 2) {
        if (w_r != nullptr) {
          uint32_t x[P][4];
          load_a<P>(x, us, kVLd, rb, h * V + 8 * nt);
          const E* wr = w_r + static_cast<size_t>(w.head0 + h) * V + 8 * nt + c2;
          const float2 wr0 = load_pair<F32>(wr), wr1 = load_pair<F32>(wr + 8);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint32_t t[P];
#pragma unroll
            for (int s = 0; s < P; ++s) t[s] = x[s][r];
            float(&o)[4] = dv[nt + (r >> 1)];
            set_pair(o, r & 1, fma2(r < 2 ? wr0 : wr1, join<P>(t), pair(o, r & 1)));
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          E* dst = dv_out + ((r & 1) ? dv_8 : 0) + hv + 8 * (nt + (r >> 1));
          if (rb + g + 8 * (r & 1) < rows &&
              in_range(p.status, dst - static_cast<E*>(p.dv), 2, tok_extent * V, CHK_SCAN_OUT))
            store2<F32>(dst, dv[nt + (r >> 1)][2 * (r & 1)], dv[nt + (r >> 1)][2 * (r & 1) + 1]);
        }
      }
    }
    if (!F32) {
      bar_wait(2 * kThreads);  // the other side is done with H
      if (hb + 1 < hb1) fetch_h(hb + 1, tid, kThreads);
    }
    __syncthreads();
    if (hb + 1 < hb1) fetch_rest(hb + 1);
  }
  // by way of the v tile's place (bf16 inputs: and the u tile's), [j][i], to the other side
  static_assert(PO * kChunk * kVLd * 2 <= 2 * S::val, "the terms of the sum of E L");
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    if (2 * rt + n > 7) break;
    const float4 f4 = F32 ? make_float4(dsum[n][0], dsum[n][1], dsum[n][2], dsum[n][3]) : ft[32 * n];
    uint32_t x0[PO], x1[PO];
    split<PO>(make_float2(f4.x, f4.y), x0);
    split<PO>(make_float2(f4.z, f4.w), x1);
#pragma unroll
    for (int s = 0; s < PO; ++s) {
      const uint32_t at = vs + s * kChunk * kVLd * 2 + ((rb + g) * kVLd + rb + 8 * n + c2) * 2;
      ptx::sts_u32(at, x0[s]);
      ptx::sts_u32(at + 8 * kVLd * 2, x1[s]);
    }
  }
  __syncthreads();
}

template <bool F32, int KT, int V>
cudaError_t launch_bwd_kt(const ScanParams& p, cudaStream_t st) {
  constexpr int bytes = BwdSmem<F32, KT, V>::bytes;
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  const cudaError_t e = allow_smem<bwd_kernel<F32, KT, V>>(bytes);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.B) * p.Nq * p.hsplit * p.nc;
  return launch_after(bwd_kernel<F32, KT, V>, dim3(static_cast<unsigned>(grid)), 2 * kThreads, bytes, st, p);
}

}  // namespace
}  // namespace scan
}  // namespace m2rnn

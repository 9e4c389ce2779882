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
// (dl_t: with respect to the natural logarithm of the decay; the last sum
// is the row sums of D from t on less its column sums from t on.)
//
// A CTA takes one chunk of one group and walks over its head blocks: dq and
// dk, and sum over heads of E L, stay in registers, so neither needs a sum
// over CTAs (unless the head blocks are shared out, then their shares are
// added in order).  Warp w holds rows j = 16 w.. of everything indexed by j and
// rows i = 16 w.. of dq; the products within the chunk are formed with j along
// the rows, which leaves G L in the registers as the A operand of dv and the
// sum of E L as that of dk.  States enter with two bf16 terms where a value
// that stays in fp32 depends on them (dl) and with one for dv.
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
  static constexpr int q = 0, k = q + key, v = k + key, u = v + val, h = u + val;
  static constexpr int r = F32 ? h : h + state;  // fp32: R takes H's place
  static constexpr int g = r + state;            // G, column tiles 2w.. of row block w only
  static constexpr int arrays = g + 20 * 512;
  // loc, locj, dts, Pin, Uin, Urow: [HB][64]; Pcol: [4][HB][64]; dw_r: [64]; <R,H>: [4]
  static constexpr int floats = 10 * HB * kChunk + kCols + 4;
  static constexpr int bytes = arrays + floats * 4;
};

// First G tile of row block rt (rt has 8 - 2 rt column tiles).
__device__ __forceinline__ int g_tile(int rt) { return rt * (9 - rt); }

__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// v of 16 values c[id] per lane, summed over the eight lanes that share lane
// mod 4: leaves sums 2 j, 2 j + 1 with j = lane / 4 (bit-reversed into halves,
// quarters, eighths as below) in c[0], c[1]; returns that j.
__device__ __forceinline__ int column_sums(float (&c)[16], int lane) {
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float send = b4 ? c[k] : c[k + 8], keep = b4 ? c[k + 8] : c[k];
    c[k] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float send = b3 ? c[k] : c[k + 4], keep = b3 ? c[k + 4] : c[k];
    c[k] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float send = b2 ? c[k] : c[k + 2], keep = b2 ? c[k + 2] : c[k];
    c[k] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
  }
  return (b4 ? 4 : 0) + (b3 ? 2 : 0) + (b2 ? 1 : 0);
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
__global__ void __launch_bounds__(kThreads, F32 || KT == 16 ? 1 : 2) bwd_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  using S = BwdSmem<F32, KT, V>;
  constexpr int P = S::P, PS = S::PS, PW = Terms<F32>::prob, K = S::K, HB = S::HB, NT = V / 8;
  constexpr int ld = K + 8;
  constexpr int PR = F32 ? PS : 1;  // terms of R in dv
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = ptx::smem_addr(smem);
  const uint32_t qs = base + S::q, ks = base + S::k, vs = base + S::v, us = base + S::u,
                 hs = base + S::h, rs = base + S::r;
  float4* gs = reinterpret_cast<float4*>(smem + S::g);
  float* loc = reinterpret_cast<float*>(smem + S::arrays);
  float* locj = loc + HB * kChunk;
  float* dts = locj + HB * kChunk;
  float* Pin = dts + HB * kChunk;
  float* Uin = Pin + HB * kChunk;
  float* Urow = Uin + HB * kChunk;
  float* Pcol = Urow + HB * kChunk;  // [4][HB][64]
  float* wsum = Pcol + 4 * HB * kChunk;
  float* rh = wsum + kCols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
  const int rt = warp;
  const int c = blockIdx.x % p.nc;
  const int rest = blockIdx.x / p.nc, share = rest % p.hsplit;
  const int group = (rest / p.hsplit) % p.Nq, b = rest / p.hsplit / p.Nq;
  const int t0 = c * kChunk, rows = min(kChunk, p.T - t0);
  const int per = (p.nhb + p.hsplit - 1) / p.hsplit;
  const int hb0 = share * per, hb1 = min(p.nhb, hb0 + per);
  const E* q = static_cast<const E*>(p.q) + b * p.qb + t0 * p.qt + static_cast<size_t>(group) * K;
  const E* k = static_cast<const E*>(p.k) + b * p.kb + t0 * p.kt + static_cast<size_t>(group) * K;
  load_tile<F32>(qs, q, p.qt, rows, K, K, ld, p.status, p.T - t0);
  load_tile<F32>(ks, k, p.kt, rows, K, K, ld, p.status, p.T - t0);
  ptx::cp_async_commit();

  const size_t sd_extent = static_cast<size_t>(p.B) * p.N * p.nc * kChunk;
  const size_t st_extent = state_at(p, PS, p.B, 0, 0);
  const size_t tok_extent = static_cast<size_t>(p.B) * p.T * p.N;  // tokens x heads
  const long long ut = static_cast<long long>(p.N) * V;
  auto fetch_state = [&](uint32_t dst, const __nv_bfloat16* src, int hb) {
    const size_t at = state_at(p, PS, b, group * p.nhb + hb, c);
    if (in_range(p.status, at, PS * kCols * K, st_extent, CHK_SCAN_WS))
      load_linear(dst, src + at, PS * kCols * K * 2);
    ptx::cp_async_commit();
  };
  auto fetch = [&](int hb) {
    const Place w = place_of(p, b, group * p.nhb + hb);
    const E* v = static_cast<const E*>(p.v) + b * p.vb + t0 * p.vt + static_cast<size_t>(w.head0) * V;
    const E* u = static_cast<const E*>(p.dy) + (static_cast<size_t>(b) * p.T + t0) * ut +
                 static_cast<size_t>(w.head0) * V;
    load_tile<F32>(vs, v, p.vt, rows, w.heads * V, kCols, kVLd, p.status, p.T - t0);
    load_tile<F32>(us, u, ut, rows, w.heads * V, kCols, kVLd, p.status, p.T - t0);
    fetch_state(hs, p.Hs, hb);
    if (!F32) fetch_state(rs, p.Rs, hb);
    for (int e = threadIdx.x; e < w.heads * kChunk; e += kThreads) {
      const size_t at = (static_cast<size_t>(b) * p.N + w.head0 + e / kChunk) * p.nc * kChunk + t0 + e % kChunk;
      float2 s = make_float2(0.f, 0.f);
      if (in_range(p.status, at, 1, sd_extent, CHK_SCAN_WS)) s = p.sd[at];
      loc[e] = s.x;
      locj[e] = F32 ? s.x : s.x - log2f(s.y);  // dt = 0: +inf, a weight of 0
      dts[e] = s.y;
    }
  };
  fetch(hb0);
  cp_async_wait<F32 ? 1 : 2>();
  __syncthreads();

  // G with j along the rows, for the tiles with i >= j
  for (int ib = rt; ib < 4; ++ib) {
    float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KT / 2; ++kk) {
      uint32_t a[P][4], b0[P][2], b1[P][2];
      load_a<P>(a, ks, ld, 16 * rt, 16 * kk);
      load_b2<P>(b0, b1, qs, ld, 16 * ib, 16 * kk);
      mma_terms<P, P>(x0, a, b0);
      mma_terms<P, P>(x1, a, b1);
    }
    const int at = (g_tile(rt) + 2 * (ib - rt)) * 32 + lane;
    gs[at] = make_float4(x0[0], x0[1], x0[2], x0[3]);
    gs[at + 32] = make_float4(x1[0], x1[1], x1[2], x1[3]);
  }

  float dq[KT][4], dk[KT][4], dsum[8][4];
#pragma unroll
  for (int nt = 0; nt < KT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) dq[nt][i] = dk[nt][i] = 0.f;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) dsum[nt][i] = 0.f;

  const E* w_r = static_cast<const E*>(p.w_r);
  float* part = p.part + (static_cast<size_t>(b) * p.nc + c) * p.N * (2 + V);
  for (int hb = hb0; hb < hb1; ++hb) {
    const Place w = place_of(p, b, group * p.nhb + hb);
    cp_async_wait<0>();
    __syncthreads();

    // Through a state: out += scale_row (A state^T) for 16 rows, and the rows'
    // products with `with`'s rows (q or k), for one head.
    auto through = [&](uint32_t tile, uint32_t state, uint32_t with, int h, float s0, float s1,
                       float (&out)[KT][4], float* sums) {
      uint32_t a[V / 16][P][4];
#pragma unroll
      for (int vv = 0; vv < V / 16; ++vv) load_a<P>(a[vv], tile, kVLd, 16 * rt, h * V + 16 * vv);
      float d0 = 0.f, d1 = 0.f;
#pragma unroll
      for (int kk = 0; kk < KT / 2; ++kk) {
        float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int vv = 0; vv < V / 16; ++vv) {
          uint32_t b0[PS][2], b1[PS][2];
          state_bt2<PS>(b0, b1, state, K, h * NT + 2 * vv, 2 * kk);
          mma_terms<P, PS>(x0, a[vv], b0);
          mma_terms<P, PS>(x1, a[vv], b1);
        }
        uint32_t m[P][4];
        load_a<P>(m, with, ld, 16 * rt, 16 * kk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // (row g, tile 2kk), (g + 8, 2kk), (g, 2kk + 1), (g + 8, 2kk + 1)
          uint32_t t[P];
#pragma unroll
          for (int s = 0; s < P; ++s) t[s] = m[s][r];
          const float2 y = join<P>(t);
          const float sc = (r & 1) ? s1 : s0;
          const float z0 = sc * (r < 2 ? x0 : x1)[2 * (r & 1)], z1 = sc * (r < 2 ? x0 : x1)[2 * (r & 1) + 1];
          out[2 * kk + (r >> 1)][2 * (r & 1)] += z0;
          out[2 * kk + (r >> 1)][2 * (r & 1) + 1] += z1;
          float& d = (r & 1) ? d1 : d0;
          d = fmaf(y.x, z0, fmaf(y.y, z1, d));
        }
      }
      d0 = quad_sum(d0);
      d1 = quad_sum(d1);
      if ((lane & 3) == 0) {
        sums[h * kChunk + 16 * rt + g] = d0;
        sums[h * kChunk + 16 * rt + g + 8] = d1;
      }
    };

#pragma unroll 1
    for (int h = 0; h < w.heads; ++h) {  // dq through H
      const float* lo = loc + h * kChunk;
      float off = 0.f;
      for (int i4 = 0; i4 < rt; ++i4) off += lo[16 * i4 + 15];
      through(us, hs, qs, h, ex2(off + lo[16 * rt + g]), ex2(off + lo[16 * rt + g + 8]), dq, Pin);
    }
    if (F32) {
      __syncthreads();
      fetch_state(rs, p.Rs, hb);
      cp_async_wait<0>();
      __syncthreads();
    }
    // <R, H> of the warp's 16 columns
    {
      const __nv_bfloat16* hg = p.Hs + state_at(p, PS, b, group * p.nhb + hb, c);
      float s = 0.f;
      if (16 * warp / V < w.heads) {
        for (int e = lane * 8; e < 2 * KT * 64; e += 256) {
          const int at = 2 * warp * KT * 64 + e;
          float x[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.f;
#pragma unroll
          for (int t = PS - 1; t >= 0; --t) {
            const uint4 rr = ptx::lds_u32x4(rs + (t * kCols * K + at) * 2);
            uint4 hh;
            if (F32)
              hh = __ldg(reinterpret_cast<const uint4*>(hg + t * kCols * K + at));
            else
              hh = ptx::lds_u32x4(hs + (t * kCols * K + at) * 2);
            const uint32_t r4[4] = {rr.x, rr.y, rr.z, rr.w}, h4[4] = {hh.x, hh.y, hh.z, hh.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[2 * j] += ptx::bf16x2_lo(r4[j]);
              x[2 * j + 1] += ptx::bf16x2_hi(r4[j]);
              y[2 * j] += ptx::bf16x2_lo(h4[j]);
              y[2 * j + 1] += ptx::bf16x2_hi(h4[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) s = fmaf(x[j], y[j], s);
        }
      }
#pragma unroll
      for (int m = 16; m >= 1; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (lane == 0) rh[warp] = s;
    }

#pragma unroll 1
    for (int h = 0; h < w.heads; ++h) {
      const float* lo = loc + h * kChunk;
      const float* lj = locj + h * kChunk;
      const int r0 = 16 * rt + g, r1 = r0 + 8;
      const float dt0 = dts[h * kChunk + r0], dt1 = dts[h * kChunk + r1];
      const float lj0 = lj[r0], lj1 = lj[r1];
      float w0, w1;  // 2^S(j,end) dt_j
      {
        float later = 0.f;
        for (int i4 = rt + 1; i4 < 4; ++i4) later += lo[16 * i4 + 15];
        w0 = ex2(later + (lo[16 * rt + 15] - lj0));
        w1 = ex2(later + (lo[16 * rt + 15] - lj1));
        if (F32) {
          w0 *= dt0;
          w1 *= dt1;
        }
      }
      through(vs, rs, ks, h, w0, w1, dk, Uin);
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
          uint32_t b0[PR][2], b1[PR][2];
          state_b2<PR>(b0, b1, rs, K, h * NT + nt, kk);
          mma_terms<P, PR>(dv[nt], a, b0);
          mma_terms<P, PR>(dv[nt + 1], a, b1);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        dv[nt][0] *= w0;
        dv[nt][1] *= w0;
        dv[nt][2] *= w1;
        dv[nt][3] *= w1;
      }
      // within the chunk
      uint32_t va[V / 16][P][4];
#pragma unroll
      for (int vv = 0; vv < V / 16; ++vv) load_a<P>(va[vv], vs, kVLd, 16 * rt, h * V + 16 * vv);
      float col[16], ur0 = 0.f, ur1 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) col[i] = 0.f;
      float s0 = -lj0, s1 = -lj1;  // sum of l behind j, up to the start of i's block
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        if (ib < rt) continue;
        if (ib > rt) {
          s0 += lo[16 * ib - 1];
          s1 += lo[16 * ib - 1];
        }
        float e0[4] = {0.f, 0.f, 0.f, 0.f}, e1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int vv = 0; vv < V / 16; ++vv) {
          uint32_t b0[P][2], b1[P][2];
          load_b2<P>(b0, b1, us, kVLd, 16 * ib, h * V + 16 * vv);
          mma_terms<P, P>(e0, va[vv], b0);
          mma_terms<P, P>(e1, va[vv], b1);
        }
        uint32_t a[PW][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int nt = 2 * ib + u;
          const float2 li = *reinterpret_cast<const float2*>(lo + 8 * nt + c2);
          const float4 gg = gs[(g_tile(rt) + 2 * (ib - rt) + u) * 32 + lane];
          float l0 = ex2(s0 + li.x), l1 = ex2(s0 + li.y);
          float l2 = ex2(s1 + li.x), l3 = ex2(s1 + li.y);
          if (F32) {
            l0 *= dt0; l1 *= dt0; l2 *= dt1; l3 *= dt1;
          }
          if (ib == rt) {  // i >= j
            const int i = 8 * u + c2;
            l0 = i >= g ? l0 : 0.f;
            l1 = i + 1 >= g ? l1 : 0.f;
            l2 = i >= g + 8 ? l2 : 0.f;
            l3 = i + 1 >= g + 8 ? l3 : 0.f;
          }
          const float* e = u ? e1 : e0;
          const float f0 = e[0] * l0, f1 = e[1] * l1, f2 = e[2] * l2, f3 = e[3] * l3;
          dsum[nt][0] += f0;
          dsum[nt][1] += f1;
          dsum[nt][2] += f2;
          dsum[nt][3] += f3;
          const float d0 = f0 * gg.x, d1 = f1 * gg.y, d2 = f2 * gg.z, d3 = f3 * gg.w;
          ur0 += d0 + d1;
          ur1 += d2 + d3;
          col[2 * nt] = d0 + d2;
          col[2 * nt + 1] = d1 + d3;
          uint32_t x0[PW], x1[PW];
          split<PW>(gg.x * l0, gg.y * l1, x0);
          split<PW>(gg.z * l2, gg.w * l3, x1);
#pragma unroll
          for (int s = 0; s < PW; ++s) {
            a[s][2 * u] = x0[s];
            a[s][2 * u + 1] = x1[s];
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
          uint32_t b0[P][2], b1[P][2];
          load_b2_t<P>(b0, b1, us, kVLd, 16 * ib, h * V + 8 * nt);
          mma_terms<PW, P>(dv[nt], a, b0);
          mma_terms<PW, P>(dv[nt + 1], a, b1);
        }
      }
      ur0 = quad_sum(ur0);
      ur1 = quad_sum(ur1);
      if ((lane & 3) == 0) {
        Urow[h * kChunk + r0] = ur0;
        Urow[h * kChunk + r1] = ur1;
      }
      const int j8 = column_sums(col, lane);  // this lane: column tile j8
      *reinterpret_cast<float2*>(Pcol + (warp * HB + h) * kChunk + 8 * j8 + c2) = make_float2(col[0], col[1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int r = hh ? r1 : r0;
          float y0 = dv[nt][2 * hh], y1 = dv[nt][2 * hh + 1];
          if (w_r != nullptr) {
            uint32_t x[P];
#pragma unroll
            for (int s = 0; s < P; ++s)
              x[s] = ptx::lds_u32(us + s * kChunk * kVLd * 2 + (r * kVLd + h * V + 8 * nt + c2) * 2);
            const float2 uu = join<P>(x);
            const E* wr = w_r + static_cast<size_t>(w.head0 + h) * V + 8 * nt + c2;
            y0 = fmaf(to_f32(wr[0]), uu.x, y0);
            y1 = fmaf(to_f32(wr[1]), uu.y, y1);
          }
          const size_t at = ((static_cast<size_t>(b) * p.T + t0 + r) * p.N + w.head0 + h) * V + 8 * nt + c2;
          if (r < rows && in_range(p.status, at, 2, tok_extent * V, CHK_SCAN_OUT))
            store2<F32>(static_cast<E*>(p.dv) + at, y0, y1);
        }
    }

    // dw_r: sum over the chunk of u (.) v, half the rows per 64 threads
    float ws = 0.f;
    if (w_r != nullptr) {
      const int col = threadIdx.x & 63, row0 = (threadIdx.x >> 6) * 32;
      for (int r = row0; r < row0 + 32; ++r) {
        const uint32_t at = (r * kVLd + col) * 2;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int s = P - 1; s >= 0; --s) {
          x += __uint_as_float(ptx::lds_u16(vs + s * kChunk * kVLd * 2 + at) << 16);
          y += __uint_as_float(ptx::lds_u16(us + s * kChunk * kVLd * 2 + at) << 16);
        }
        ws = fmaf(x, y, ws);
      }
      if (row0) wsum[col] = ws;
    }
    __syncthreads();
    const size_t part_extent = static_cast<size_t>(p.N) * (2 + V);
    if (w_r != nullptr && threadIdx.x < w.heads * V) {
      const size_t at = 2 * static_cast<size_t>(p.N) + static_cast<size_t>(w.head0) * V + threadIdx.x;
      if (in_range(p.status, at, 1, part_extent, CHK_SCAN_PARAM)) part[at] = ws + wsum[threadIdx.x];
    }
    if (warp < w.heads) {  // the gate: one warp per head, two tokens per lane
      const int h = warp, n = w.head0 + h, t = 2 * lane;
      const float* lo = loc + h * kChunk;
      const float alpha = to_f32(static_cast<const E*>(p.alpha)[n]);
      const float beta = to_f32(static_cast<const E*>(p.beta)[n]);
      float x[2];
      const E* a = static_cast<const E*>(p.a) + b * p.ab + n;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        x[e] = t + e < rows && in_range(p.status, t0 + t + e, 1, p.T, CHK_SCAN_IN)
                   ? to_f32(a[(t0 + t + e) * p.at]) + beta : -INFINITY;
      float fwd[2], bwd[2], uu[2], ui[2];  // Uin; Pin + rows of D - columns of D
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = h * kChunk + t + e;
        ui[e] = Uin[at];
        uu[e] = ui[e] + Urow[at];
        bwd[e] = Pin[at] - Urow[at];
        float pc = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) pc += Pcol[(s * HB + h) * kChunk + t + e];
        bwd[e] += pc;
        fwd[e] = ui[e];
      }
      float inc = fwd[0] + fwd[1], suf = bwd[0] + bwd[1];
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const float up = __shfl_up_sync(0xffffffffu, inc, d);
        const float dn = __shfl_down_sync(0xffffffffu, suf, d);
        if (lane >= d) inc += up;
        if (lane + d < 32) suf += dn;
      }
      float before = __shfl_up_sync(0xffffffffu, inc, 1), behind = __shfl_down_sync(0xffffffffu, suf, 1);
      if (lane == 0) before = 0.f;
      if (lane == 31) behind = 0.f;
      float rhs = 0.f;
#pragma unroll
      for (int s = 0; s < V / 16; ++s) rhs += rh[h * (V / 16) + s];
      const float through_all = ex2((lo[15] + lo[31]) + (lo[47] + lo[63])) * rhs;
      float dl[2];
      dl[0] = through_all + before + (behind + bwd[1] + bwd[0]);
      dl[1] = through_all + (before + fwd[0]) + (behind + bwd[1]);
      float sa = 0.f, sb = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (t + e >= rows) continue;
        const float dt = dts[h * kChunk + t + e];
        const float sg = 1.f / (1.f + expf(-x[e]));
        // sigmoid / softplus -> 1 as both vanish; a token with dt = 0 has no part of U
        const float ratio = dt > 0.f ? sg / dt : 1.f;
        const float da = fmaf(ratio, uu[e], -alpha * sg * dl[e]);
        sa = fmaf(-dt, dl[e], sa);
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
    __syncthreads();
    if (hb + 1 < hb1) fetch(hb + 1);
  }

  // dq and dk within the chunk, from the sum over heads of E L
  uint32_t x[8][2][PW];
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    split<PW>(dsum[nt][0], dsum[nt][1], x[nt][0]);
    split<PW>(dsum[nt][2], dsum[nt][3], x[nt][1]);
#pragma unroll
    for (int s = 0; s < PW; ++s) {  // the v tile's place: [j][i]
      const uint32_t at = vs + s * kChunk * kVLd * 2 + ((16 * rt + g) * kVLd + 8 * nt + c2) * 2;
      ptx::sts_u32(at, x[nt][0][s]);
      ptx::sts_u32(at + 8 * kVLd * 2, x[nt][1][s]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
    if (ib < rt) continue;
    uint32_t a[PW][4];
#pragma unroll
    for (int s = 0; s < PW; ++s) {
      a[s][0] = x[2 * ib][0][s];
      a[s][1] = x[2 * ib][1][s];
      a[s][2] = x[2 * ib + 1][0][s];
      a[s][3] = x[2 * ib + 1][1][s];
    }
#pragma unroll
    for (int nt = 0; nt < KT; nt += 2) {
      uint32_t b0[P][2], b1[P][2];
      load_b2_t<P>(b0, b1, qs, ld, 16 * ib, 8 * nt);
      mma_terms<PW, P>(dk[nt], a, b0);
      mma_terms<PW, P>(dk[nt + 1], a, b1);
    }
  }
  for (int jb = 0; jb <= rt; ++jb) {
    uint32_t a[PW][4];
    load_a_t<PW>(a, vs, kVLd, 16 * jb, 16 * rt);
#pragma unroll
    for (int nt = 0; nt < KT; nt += 2) {
      uint32_t b0[P][2], b1[P][2];
      load_b2_t<P>(b0, b1, ks, ld, 16 * jb, 8 * nt);
      mma_terms<PW, P>(dq[nt], a, b0);
      mma_terms<PW, P>(dq[nt + 1], a, b1);
    }
  }
  const size_t qk_extent = static_cast<size_t>(p.B) * p.T * p.Nq * K;
#pragma unroll
  for (int nt = 0; nt < KT; ++nt)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = 16 * rt + g + 8 * hh;
      const size_t at = ((static_cast<size_t>(b) * p.T + t0 + r) * p.Nq + group) * K + 8 * nt + c2;
      if (r >= rows || !in_range(p.status, at, 2, qk_extent, CHK_SCAN_OUT)) continue;
      if (p.hsplit > 1) {
        float* dst = p.dqk + static_cast<size_t>(share) * 2 * qk_extent + at;
        *reinterpret_cast<float2*>(dst) = make_float2(dq[nt][2 * hh], dq[nt][2 * hh + 1]);
        *reinterpret_cast<float2*>(dst + qk_extent) = make_float2(dk[nt][2 * hh], dk[nt][2 * hh + 1]);
      } else {
        store2<F32>(static_cast<E*>(p.dq) + at, dq[nt][2 * hh], dq[nt][2 * hh + 1]);
        store2<F32>(static_cast<E*>(p.dk) + at, dk[nt][2 * hh], dk[nt][2 * hh + 1]);
      }
    }
}

template <bool F32, int KT, int V>
cudaError_t launch_bwd_kt(const ScanParams& p, cudaStream_t st) {
  constexpr int bytes = BwdSmem<F32, KT, V>::bytes;
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  auto kern = bwd_kernel<F32, KT, V>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.B) * p.Nq * p.hsplit * p.nc;
  kern<<<static_cast<unsigned>(grid), kThreads, bytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace scan
}  // namespace m2rnn

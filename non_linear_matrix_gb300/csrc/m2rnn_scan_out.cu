// m2rnn_scan_out.cu -- the outputs of the selective scan, chunk by chunk, from
// the states before the chunks:
//
//     y_i = 2^S(start,i) H^T q_i + sum_{j<=i} (q_i.k_j) 2^S(j,i) dt_j v_j + w_r (.) v_i
//
// A CTA takes one chunk of one query/key group: q k^T (64 x 64, fp32) is
// formed once, a warp keeping its 16 rows in registers for all heads; then the
// head blocks pass by, each bringing its v tile and state.  For each head
// the weights are made in registers from q k^T, in the layout that the next
// product takes as its A operand.  Between different 16-token blocks the decay
// is a product of a row's and a column's factor, both at most 1 in size for a
// decaying gate (the column's made with the states); only the diagonal blocks
// take a power of two per element.
//
// Bound by latency: each head block waits for its state, converts it and passes
// two barriers, at four CTAs per SM (registers, shared memory).  B=1 T=65536 N=64
// K=64 V=16: 285 us (issue 40 %, shared-memory pipe 50 %, tensor pipe 21 %); B=8 T=4096
// N=32: 79 us.  With one-term weights and states it was 182 and 53, of which
// without the state's fetch 40 remained and without the products within the chunk 48;
// double-buffered tiles (three CTAs) took 63 then, five CTAs (spills) 61.
#include <type_traits>

#include "m2rnn_scan.cuh"

namespace m2rnn {
namespace scan {
namespace {

template <bool F32, int KT, int V>
struct OutSmem {
  static constexpr int P = Terms<F32>::in, PS = Terms<F32>::state, K = 8 * KT, HB = kCols / V;
  static constexpr int key = P * kChunk * (K + 8) * 2, val = P * kChunk * kVLd * 2;
  // the k tile, and after q k^T the rows of y on their way out
  static constexpr int ky = key > kChunk * kVLd * 2 ? key : kChunk * kVLd * 2;
  static constexpr int q = 0, k = key, v = k + ky, h = v + val, gate = h + PS * kCols * K * 2;
  static constexpr int bytes = gate + HB * kGate * 4;
};

// acc (16 rows i x 8 columns) += A (rows i, tokens j of the same 16) times those values
// of v that are infinite or NaN, for j <= i only: what a product with masked
// weights cannot do.  v: shared address of token 0's 8 columns.  Rare, so one token
// at a time.
template <int PA>
__device__ __forceinline__ void add_not_finite(float (&acc)[4], const uint32_t (&a)[PA][4], uint32_t v) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll 1
    for (int jj = 0; jj < 8; ++jj) {
      const int j = 8 * u + jj, from = (lane & 28) | (jj >> 1);
      float w0 = 0.f, w1 = 0.f;  // rows g, g + 8
#pragma unroll
      for (int t = PA - 1; t >= 0; --t) {
        const uint32_t x0 = __shfl_sync(0xffffffffu, a[t][2 * u], from);
        const uint32_t x1 = __shfl_sync(0xffffffffu, a[t][2 * u + 1], from);
        w0 += (jj & 1) ? ptx::bf16x2_hi(x0) : ptx::bf16x2_lo(x0);
        w1 += (jj & 1) ? ptx::bf16x2_hi(x1) : ptx::bf16x2_lo(x1);
      }
      const uint32_t x = ptx::lds_u32(v + (j * kVLd + c2) * 2), bad = not_finite(x);
      const float lo = ptx::bf16x2_lo(x), hi = ptx::bf16x2_hi(x);
      if (bad & 0x8000u) {
        if (j <= g) acc[0] = fmaf(w0, lo, acc[0]);
        if (j <= g + 8) acc[2] = fmaf(w1, lo, acc[2]);
      }
      if (bad & 0x80000000u) {
        if (j <= g) acc[1] = fmaf(w0, hi, acc[1]);
        if (j <= g + 8) acc[3] = fmaf(w1, hi, acc[3]);
      }
    }
}

template <bool F32, int KT, int V>
__global__ void __launch_bounds__(kThreads, F32 ? 1 : (KT == 16 ? 2 : 4)) out_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  using S = OutSmem<F32, KT, V>;
  constexpr int P = S::P, PS = S::PS, PO = Terms<F32>::out, K = S::K, ld = K + 8;
  constexpr int HB = S::HB, NT = V / 8;  // heads per block, column tiles per head
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = ptx::smem_addr(smem), qs = base + S::q, ks = base + S::k, vs = base + S::v,
                 hs = base + S::h, ys = ks;
  const float* gate = reinterpret_cast<const float*>(smem + S::gate);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
  const int rt = row_block(warp);  // the warp's 16 rows
  const int c = blockIdx.x % p.nc;
  const int rest = blockIdx.x / p.nc, part = rest % p.hsplit;
  const int group = (rest / p.hsplit) % p.Nq, b = rest / p.hsplit / p.Nq;
  const int t0 = c * kChunk, rows = min(kChunk, p.T - t0), seg = c / p.cps;
  const int per = (p.nhb + p.hsplit - 1) / p.hsplit;
  const int hb0 = part * per, hb1 = min(p.nhb, hb0 + per);
  const E* q = static_cast<const E*>(p.q) + b * p.qb + t0 * p.qt + static_cast<size_t>(group) * K;
  const E* k = static_cast<const E*>(p.k) + b * p.kb + t0 * p.kt + static_cast<size_t>(group) * K;
  load_tile<F32, K>(threadIdx.x, qs, q, p.qt, rows, K, p.status, p.T - t0);
  load_tile<F32, K>(threadIdx.x, ks, k, p.kt, rows, K, p.status, p.T - t0);
  ptx::cp_async_commit();

  const size_t hl_extent = static_cast<size_t>(p.B) * p.Nq * p.nhb * p.nc * kCols * K;
  auto fetch = [&](int hb) {
    const Place w = place_in(p, HB, b, group, hb);
    const E* v = static_cast<const E*>(p.v) + b * p.vb + t0 * p.vt + static_cast<size_t>(w.head0) * V;
    load_tile<F32, kCols>(threadIdx.x, vs, v, p.vt, rows, w.heads * V, p.status, p.T - t0);
    load_gate(threadIdx.x, base + S::gate, p, w, c);
    ptx::cp_async_commit();
    const StateRef r = state_ref(p, p.Hl, p.Hseg, p.cdec, w, c, seg);
    constexpr int step = kThreads * 8, U = kCols * K >= 2 * step ? 2 : 1;  // rows in flight
    const int n = w.heads * V * K;
#pragma unroll 1
    for (int e0 = threadIdx.x * 8; e0 < n; e0 += U * step) {
      StateRow x[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * step;
        on[u] = e < n && in_range(p.status, r.at + e, 8, hl_extent, CHK_SCAN_WS);
        if (on[u]) x[u] = state_load<K, V>(p, r, e);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on[u]) {
          float2 z[4];
          state_sum(x[u], z);
          put_state_row<PS, K>(hs, e0 + u * step, z);
        }
    }
  };
  await_before();  // (q and k are inputs)
  fetch(hb0);
  cp_async_wait<1>();
  __syncthreads();

  float gm[8][4];  // q k^T: rows 16 rt + g [+8], column tile nt
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) gm[nt][i] = 0.f;
#pragma unroll
  for (int kk = 0; kk < KT / 2; ++kk) {
    uint32_t a[P][4];
    load_a<P>(a, qs, ld, 16 * rt, 16 * kk);
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      if (jb > rt) break;
      uint32_t b0[P][2], b1[P][2];
      load_b2<P>(b0, b1, ks, ld, 16 * jb, 16 * kk);
      mma_terms<P, P>(gm[2 * jb], a, b0);
      mma_terms<P, P>(gm[2 * jb + 1], a, b1);
    }
  }

  const E* w_r = static_cast<const E*>(p.w_r);
  E* y = static_cast<E*>(p.y);
  const size_t y_extent = static_cast<size_t>(p.B) * p.T * p.N * V;
  for (int hb = hb0; hb < hb1; ++hb) {
    const Place w = place_in(p, HB, b, group, hb);
    cp_async_wait<0>();
    __syncthreads();
    if (hb + 1 < hb1) {
      const Place next = place_in(p, HB, b, group, hb + 1);
      state_prefetch(threadIdx.x, state_ref(p, p.Hl, p.Hseg, p.cdec, next, c, seg), next.heads * V * K);
    }
    float acc[8][4];
    // The rows' outputs but for w_r (.) v.  CAREFUL: a value of v that is not finite
    // is kept out of the product with the weights of its own 16 tokens, where a
    // masked weight of 0 would make NaN of it for the tokens before.
    auto form = [&](auto careful) {
      constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
      // from the state: q H
#pragma unroll
      for (int kk = 0; kk < KT / 2; ++kk) {
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
        const float* lo = gate + h * kGate;
        const float* end = lo + 128;
        const float li0 = lo[16 * rt + g], li1 = lo[16 * rt + g + 8];
        const float tot[3] = {lo[15], lo[31], lo[47]};
        {  // decay since the chunk's start
          float off = 0.f;
#pragma unroll
          for (int k4 = 0; k4 < 3; ++k4) off += k4 < rt ? tot[k4] : 0.f;
          const float2 e0 = both(ex2(off + li0)), e1 = both(ex2(off + li1));
#pragma unroll
          for (int nt = h * NT; nt < (h + 1) * NT; ++nt) {
            set_pair(acc[nt], 0, mul2(pair(acc[nt], 0), e0));
            set_pair(acc[nt], 1, mul2(pair(acc[nt], 1), e1));
          }
        }
        // within the chunk; s0, s1: sum of l from the end of j's block to i
        float s0 = li0, s1 = li1;
#pragma unroll
        for (int jj = 3; jj >= 0; --jj) {
          if (jj > rt) continue;
          uint32_t a[PO][4];
          if (jj == rt) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int nt = 2 * jj + u;
              const float2 lj = *reinterpret_cast<const float2*>(lo + 8 * nt + c2);
              const float2 dt = *reinterpret_cast<const float2*>(lo + 64 + 8 * nt + c2);
              const float2 ej = *reinterpret_cast<const float2*>(lo + 192 + 8 * nt + c2);
              const float ei0 = lo[192 + 16 * rt + g], ei1 = lo[192 + 16 * rt + g + 8];
              float2 x0 = mul2(make_float2(ex2((li0 - lj.x) + (ei0 - ej.x)), ex2((li0 - lj.y) + (ei0 - ej.y))), dt);
              float2 x1 = mul2(make_float2(ex2((li1 - lj.x) + (ei1 - ej.x)), ex2((li1 - lj.y) + (ei1 - ej.y))), dt);
              x0 = mul2(pair(gm[nt], 0), x0);
              x1 = mul2(pair(gm[nt], 1), x1);
              const int j = 8 * u + c2;  // j <= i (the product is cut: a later k_j may be NaN)
              x0.x = j <= g ? x0.x : 0.f;
              x0.y = j < g ? x0.y : 0.f;
              x1.x = j <= g + 8 ? x1.x : 0.f;
              x1.y = j < g + 8 ? x1.y : 0.f;
              uint32_t y0[PO], y1[PO];
              split<PO>(x0, y0);
              split<PO>(x1, y1);
#pragma unroll
              for (int t = 0; t < PO; ++t) {
                a[t][2 * u] = y0[t];
                a[t][2 * u + 1] = y1[t];
              }
            }
          } else {
            if (jj + 1 < rt) {
              s0 += tot[jj + 1 < 3 ? jj + 1 : 2];
              s1 += tot[jj + 1 < 3 ? jj + 1 : 2];
            }
            const float2 r0 = both(ex2(s0)), r1 = both(ex2(s1));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int nt = 2 * jj + u;
              const float2 e = *reinterpret_cast<const float2*>(end + 8 * nt + c2);
              uint32_t y0[PO], y1[PO];
              split<PO>(mul2(mul2(pair(gm[nt], 0), e), r0), y0);
              split<PO>(mul2(mul2(pair(gm[nt], 1), e), r1), y1);
#pragma unroll
              for (int t = 0; t < PO; ++t) {
                a[t][2 * u] = y0[t];
                a[t][2 * u + 1] = y1[t];
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; nt += 2) {
            uint32_t b0[P][2], b1[P][2];
            load_b2_t<P>(b0, b1, vs, kVLd, 16 * jj, h * V + 8 * nt);
            if (CAREFUL && jj == rt) {
              add_not_finite<PO>(acc[h * NT + nt], a, vs + (16 * rt * kVLd + h * V + 8 * nt) * 2);
              add_not_finite<PO>(acc[h * NT + nt + 1], a, vs + (16 * rt * kVLd + h * V + 8 * nt + 8) * 2);
#pragma unroll
              for (int t = 0; t < P; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  b0[t][r] = finite_only(b0[t][r]);
                  b1[t][r] = finite_only(b1[t][r]);
                }
            }
            mma_terms<PO, P>(acc[h * NT + nt], a, b0);
            mma_terms<PO, P>(acc[h * NT + nt + 1], a, b1);
          }
        }
      }
    };
    form(std::false_type{});
    {  // rare: once more, with care (a NaN of an earlier token stays one)
      float2 z = make_float2(0.f, 0.f);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) z = fma2(pair(acc[nt], 0), z, mul2(pair(acc[nt], 1), make_float2(0.f, 0.f)));
      if (__any_sync(0xffffffffu, !(z.x + z.y == 0.f))) form(std::true_type{});
    }
    // + w_r (.) v, and out
#pragma unroll
    for (int nt = 0; nt < 8; nt += 2) {
      if (nt >= w.heads * NT) break;
      if (w_r != nullptr) {
        uint32_t x[P][4];
        load_a<P>(x, vs, kVLd, 16 * rt, 8 * nt);
        const E* src = w_r + static_cast<size_t>(w.head0) * V + 8 * nt + c2;
        const float2 wr0 = load_pair<F32>(src), wr1 = load_pair<F32>(src + 8);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t t[P];
#pragma unroll
          for (int s = 0; s < P; ++s) t[s] = x[s][r];
          const float2 wr = r < 2 ? wr0 : wr1;
          set_pair(acc[nt + (r >> 1)], r & 1, fma2(wr, join<P>(t), pair(acc[nt + (r >> 1)], r & 1)));
        }
      }
      if constexpr (F32) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * rt + g + 8 * (r & 1);
          const size_t at = ((static_cast<size_t>(b) * p.T + t0 + row) * p.N + w.head0) * V +
                            8 * (nt + (r >> 1)) + c2;
          if (row < rows && in_range(p.status, at, 2, y_extent, CHK_SCAN_OUT))
            *reinterpret_cast<float2*>(y + at) = pair(acc[nt + (r >> 1)], r & 1);
        }
      } else {
        uint32_t x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float2 o = pair(acc[nt + (r >> 1)], r & 1);
          x[r] = ptx::pack_bf16x2(o.x, o.y);
        }
        stsm4(piece_rc(ys, kVLd, 16 * rt, 8 * nt), x);
      }
    }
    if constexpr (!F32) {
      __syncwarp();  // the warp's own 16 rows, in 16-byte pieces
      const int col = (lane & 7) * 8, r0 = 16 * rt + (lane >> 3);
      size_t at = ((static_cast<size_t>(b) * p.T + t0 + r0) * p.N + w.head0) * V + col;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = r0 + 4 * it;
        if (r < rows && col < w.heads * V && in_range(p.status, at, 8, y_extent, CHK_SCAN_OUT))
          *reinterpret_cast<uint4*>(y + at) = ptx::lds_u32x4(ys + (r * kVLd + col) * 2);
        at += 4 * static_cast<size_t>(p.N) * V;
      }
    }
    __syncthreads();  // v, the state and the gate may be overwritten
    if (hb + 1 < hb1) fetch(hb + 1);
  }
}

template <bool F32, int KT, int V>
cudaError_t run(const ScanParams& p, cudaStream_t st) {
  constexpr int smem = OutSmem<F32, KT, V>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  const cudaError_t e = allow_smem<out_kernel<F32, KT, V>>(smem);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.B) * p.Nq * p.hsplit * p.nc;
  return launch_after(out_kernel<F32, KT, V>, dim3(static_cast<unsigned>(grid)), kThreads, smem, st, p);
}

template <bool F32, int V>
cudaError_t run_k(const ScanParams& p, cudaStream_t st) {
  switch (p.K) {
    case 16: return run<F32, 2, V>(p, st);
    case 32: return run<F32, 4, V>(p, st);
    case 64: return run<F32, 8, V>(p, st);
    default: return run<F32, 16, V>(p, st);
  }
}
template <int V>
cudaError_t run_type(const ScanParams& p, bool f32, cudaStream_t st) {
  return f32 ? run_k<true, V>(p, st) : run_k<false, V>(p, st);
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_out(const ScanParams& p, bool f32, cudaStream_t st) {
  return p.V == 16 ? scan::run_type<16>(p, f32, st) : scan::run_type<32>(p, f32, st);
}

}  // namespace m2rnn

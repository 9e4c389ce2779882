// m2rnn_scan_states.cu -- the states of the selective scan at the chunks'
// borders: forwards (H before each chunk, from k, v and the gate) or in
// reverse (R after each chunk, the gradient that reaches the state from later
// tokens, from q and dy):
//
//     H' = 2^S(start,end) H + sum_j 2^S(j,end) dt_j k_j v_j^T
//     R  = 2^S(start,end) R' + sum_i 2^S(start,i) q_i dy_i^T
//
// A CTA walks along a segment of a sequence with the state of one head block
// (64 value columns x K) in its accumulators, warp w the columns 16 w..; the
// decayed values are the A operand (three bf16 terms, made in registers, so the
// state is good to fp32), the keys the B operand.  Segments run at the same
// time from zero states; join_kernel then carries the states from segment to
// segment.
//
// Bound by the three-term products (42 % of the tensor pipe's cycles), the
// instructions around them (46 % of issue slots) and the states' traffic (54 % of
// DRAM's): B=1 T=65536 N=64 K=64 V=16 takes 101 us.  B=8 T=4096 N=32: 33 us forwards, 28 in reverse; the join
// 5 to 8.  Four CTAs per SM: without that bound on the registers 107 us, with five
// (spills) 151.
#include "m2rnn_scan.cuh"

namespace m2rnn {
namespace scan {
namespace {

template <bool F32, int KT, bool REV>
__global__ void __launch_bounds__(kThreads, F32 ? (KT == 16 ? 2 : 3) : KT == 16 ? 3 : 4) states_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  constexpr int P = Terms<F32>::in, PS = Terms<F32>::state, K = 8 * KT, kLd = K + 8;
  constexpr int kKey = P * kChunk * kLd * 2, kVal = P * kChunk * kVLd * 2;
  extern __shared__ __align__(128) unsigned char smem[];
  float(*weights)[kChunk] = reinterpret_cast<float(*)[kChunk]>(smem);
  const uint32_t key0 = ptx::smem_addr(smem) + 4 * kChunk * 4, val0 = key0 + 2 * kKey;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
  const int seg = blockIdx.x % p.nseg, gbx = blockIdx.x / p.nseg;
  const int gb = gbx % (p.Nq * p.nhb), b = gbx / (p.Nq * p.nhb);
  const Place w = place_of(p, b, gb);
  const int vh = 16 * warp / p.V;  // the warp's head within the block
  const bool on = vh < w.heads;
  const bool leads = on && (16 * warp) % p.V == 0;  // writes what a head has once
  const int n = w.head0 + (on ? vh : 0);
  const int first = seg * p.cps, count = min(p.cps, p.nc - first);
  const E* key = static_cast<const E*>(REV ? p.q : p.k) + b * (REV ? p.qb : p.kb) +
                 static_cast<size_t>(w.group) * K;
  const long long key_t = REV ? p.qt : p.kt;
  const E* val = REV ? static_cast<const E*>(p.dy) +
                           (static_cast<size_t>(b) * p.T * p.N + w.head0) * p.V
                     : static_cast<const E*>(p.v) + b * p.vb + static_cast<size_t>(w.head0) * p.V;
  const long long val_t = REV ? static_cast<long long>(p.N) * p.V : p.vt;
  const float beta = to_f32(static_cast<const E*>(p.beta)[n]);
  // -alpha log2(e) to twice fp32: an error here would be the same for all of a
  // head's tokens, which dalpha (a sum that nearly cancels) shows ten times over
  const float alpha = -to_f32(static_cast<const E*>(p.alpha)[n]);
  const float rate = alpha * kLog2e, rate_lo = fmaf(alpha, kLog2e, -rate) + alpha * kLog2eLo;
  const size_t head = static_cast<size_t>(b) * p.N + n;
  const size_t gate_extent = static_cast<size_t>(p.B) * p.N * p.nc * kGate;

  auto chunk_of = [&](int i) { return REV ? p.nc - 1 - (first + i) : first + i; };
  auto fetch = [&](int i) {  // tiles of the i-th chunk of the segment
    const int t0 = chunk_of(i) * kChunk, rows = min(kChunk, p.T - t0);
    load_tile<F32, K>(threadIdx.x, key0 + (i & 1) * kKey, key + t0 * key_t, key_t, rows, K, p.status, p.T - t0);
    load_tile<F32, kCols>(threadIdx.x, val0 + (i & 1) * kVal, val + t0 * val_t, val_t, rows, w.heads * p.V,
                          p.status, p.T - t0);
    ptx::cp_async_commit();
  };
  float2 ga;  // the lane's two tokens: gate inputs (forward) or block sums (reverse)
  auto fetch_gate = [&](int i) {
    const int c = chunk_of(i), t = c * kChunk + 2 * lane;
    if constexpr (REV) {
      const size_t at = (head * p.nc + c) * kGate + 2 * lane;
      ga = make_float2(0.f, 0.f);
      if (in_range(p.status, at, 2, gate_extent, CHK_SCAN_WS))
        ga = *reinterpret_cast<const float2*>(p.gate + at);
    } else {
      const E* a = static_cast<const E*>(p.a) + b * p.ab + n;
      ga = make_float2(-INFINITY, -INFINITY);
      if (t < p.T && in_range(p.status, t, 1, p.T, CHK_SCAN_IN)) ga.x = to_f32(a[t * p.at]);
      if (t + 1 < p.T && in_range(p.status, t + 1, 1, p.T, CHK_SCAN_IN))
        ga.y = to_f32(a[(t + 1) * p.at]);
    }
  };

  let_next_begin();
  fetch_gate(0);
  fetch(0);
  // state: accumulator nt holds (column 16 warp + g [+8], key row 8 nt + c2, +1)
  float acc[KT][4];
  const float* init = REV ? p.dHT : p.H0;
  const size_t st0 = head * K * p.V, st_extent = static_cast<size_t>(p.B) * p.N * K * p.V;
  const int vcol = (16 * warp) % p.V + g;
#pragma unroll
  for (int nt = 0; nt < KT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[nt][i] = 0.f;
      const size_t at = st0 + static_cast<size_t>(8 * nt + c2 + (i & 1)) * p.V + vcol + (i >> 1) * 8;
      if (on && seg == 0 && init != nullptr && in_range(p.status, at, 1, st_extent, CHK_SCAN_STATE))
        acc[nt][i] = init[at];
    }
  // writes the accumulators as a tile's blocks, whole lines at a time
  auto put = [&](float* base, size_t tiles, size_t tile) {
#pragma unroll
    for (int nt = 0; nt < KT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t at = tile * kCols * K + ((2 * warp + h) * KT + nt) * 64 + 2 * lane;
        if (in_range(p.status, at, 2, tiles * kCols * K, CHK_SCAN_WS))
          *reinterpret_cast<float2*>(base + at) = pair(acc[nt], h);
      }
  };

  const size_t pairs = static_cast<size_t>(p.B) * p.Nq * p.nhb;
  float total = 0.f;  // log2 decay of the segment so far
  for (int i = 0; i < count; ++i) {
    const int c = chunk_of(i);
    // The gate's sums.  Blocks of 16 tokens are 8 lanes; loc: from the block's
    // start up to the lane's tokens, rest: from behind them to its end.
    float2 loc, left, rest = make_float2(0.f, 0.f), dt = make_float2(0.f, 0.f), wt;
    if constexpr (REV) {
      loc = ga;
    } else {
      dt.x = gate_softplus(ga.x + beta);
      dt.y = gate_softplus(ga.y + beta);
      float2 l = make_float2(fmaf(rate, dt.x, rate_lo * dt.x), fmaf(rate, dt.y, rate_lo * dt.y));
      // below 2^-160 a decay is 0 in fp32: the bound keeps sums short
      l.x = l.x < -160.f ? -160.f : l.x;
      l.y = l.y < -160.f ? -160.f : l.y;
      float low, inc = two_sum(l.x, l.y, low), suf = inc;  // inc + low: the sum so far
#pragma unroll
      for (int d = 1; d < 8; d *= 2) {
        const float up = __shfl_up_sync(0xffffffffu, inc, d, 8);
        const float up_low = __shfl_up_sync(0xffffffffu, low, d, 8);
        const float dn = __shfl_down_sync(0xffffffffu, suf, d, 8);
        if ((lane & 7) >= d) {
          float e;
          inc = two_sum(up, inc, e);
          low += up_low + e;
        }
        if ((lane & 7) + d < 8) suf += dn;
      }
      const float before = __shfl_up_sync(0xffffffffu, inc, 1, 8);
      const float before_low = __shfl_up_sync(0xffffffffu, low, 1, 8);
      const float behind = __shfl_down_sync(0xffffffffu, suf, 1, 8);
      loc.y = inc;
      left.y = low;
      loc.x = two_sum((lane & 7) ? before : 0.f, l.x, left.x);
      if (lane & 7) left.x += before_low;
      rest.y = (lane & 7) < 7 ? behind : 0.f;
      rest.x = rest.y + l.y;
    }
    float tot[4], off = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) tot[k] = __shfl_sync(0xffffffffu, loc.y, 8 * k + 7);
    const int blk = lane >> 3;
    if constexpr (REV) {
#pragma unroll
      for (int k = 0; k < 3; ++k) off += k < blk ? tot[k] : 0.f;
      wt = make_float2(ex2(off + loc.x), ex2(off + loc.y));
    } else {
#pragma unroll
      for (int k = 3; k > 0; --k) off += k > blk ? tot[k] : 0.f;
      const float2 end = make_float2(ex2(rest.x) * dt.x, ex2(rest.y) * dt.y);
      wt = make_float2(ex2(off + rest.x) * dt.x, ex2(off + rest.y) * dt.y);
      const size_t at = (head * p.nc + c) * kGate + 2 * lane;
      if (leads && in_range(p.status, at, 194, gate_extent, CHK_SCAN_WS)) {
        *reinterpret_cast<float2*>(p.gate + at) = loc;
        *reinterpret_cast<float2*>(p.gate + at + 64) = dt;
        *reinterpret_cast<float2*>(p.gate + at + 128) = end;
        *reinterpret_cast<float2*>(p.gate + at + 192) = left;
      }
    }
    const float chunk_sum = (tot[0] + tot[1]) + (tot[2] + tot[3]);
    *reinterpret_cast<float2*>(&weights[warp][2 * lane]) = wt;
    const size_t cat = head * p.nc + c;
    if (leads && lane == 0 &&
        in_range(p.status, cat, 1, static_cast<size_t>(p.B) * p.N * p.nc, CHK_SCAN_WS))
      (REV ? p.rdec : p.cdec)[cat] = total;
    total += chunk_sum;
    if (i + 1 < count) fetch_gate(i + 1);
    cp_async_wait<0>();
    __syncthreads();  // tiles of chunk i are there; everyone is done with chunk i - 1
    if (i + 1 < count) fetch(i + 1);
    if (on) {
      put(REV ? p.Rl : p.Hl, pairs * p.nc, static_cast<size_t>(gbx) * p.nc + c);
      const float2 dec = both(ex2(chunk_sum));
      const uint32_t kt = key0 + (i & 1) * kKey, vt = val0 + (i & 1) * kVal;
      constexpr int G = F32 ? 1 : 4;  // steps of 16 tokens at a time (fp32 has more terms to hold)
#pragma unroll
      for (int k0 = 0; k0 < 4; k0 += G) {
        uint32_t a[G][PS][4];  // the decayed values
#pragma unroll
        for (int ks = 0; ks < G; ++ks) {
          const int t = 16 * (k0 + ks);
          uint32_t raw[P][4];
          load_a_t<P>(raw, vt, kVLd, t, 16 * warp);
          const float2 w0 = *reinterpret_cast<const float2*>(&weights[warp][t + c2]);
          const float2 w1 = *reinterpret_cast<const float2*>(&weights[warp][t + 8 + c2]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint32_t x[P], y[PS];
#pragma unroll
            for (int s = 0; s < P; ++s) x[s] = raw[s][r];
            split<PS>(mul2(join<P>(x), r < 2 ? w0 : w1), y);
#pragma unroll
            for (int s = 0; s < PS; ++s) a[ks][s][r] = y[s];
          }
        }
        constexpr int NX = KT >= 4 ? 4 : 2;
        const float2 old = k0 == 0 ? dec : both(1.f);
#pragma unroll
        for (int nt = 0; nt < KT; nt += NX) {
          float x[NX][4];  // what these tokens add
#pragma unroll
          for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
          for (int ks = 0; ks < G; ++ks) {
            uint32_t bb[NX][P][2];
#pragma unroll
            for (int n = 0; n < NX; n += 2)
              load_b2_t<P>(bb[n], bb[n + 1], kt, kLd, 16 * (k0 + ks), 8 * (nt + n));
            mma_terms_n<PS, P, NX>(x, a[ks], bb);
          }
#pragma unroll
          for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              set_pair(acc[nt + n], h, fma2(pair(acc[nt + n], h), old, pair(x[n], h)));
        }
      }
    }
    __syncwarp();  // the warp's weights may be overwritten
  }
  if (!on) return;
  if (p.nseg > 1) {
    put(REV ? p.Rseg : p.Hseg, pairs * p.nseg, static_cast<size_t>(gbx) * p.nseg + seg);
    // the whole segment's decay goes behind its last chunk's
    const size_t at = static_cast<size_t>(p.B) * p.N * p.nc + head * p.nseg + seg;
    if (leads && lane == 0 &&
        in_range(p.status, at, 1, static_cast<size_t>(p.B) * p.N * (p.nc + p.nseg), CHK_SCAN_WS))
      (REV ? p.rdec : p.cdec)[at] = total;
    return;
  }
  float* fin = REV ? p.dH0 : p.HT;
  if (fin == nullptr) return;
#pragma unroll
  for (int nt = 0; nt < KT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t at = st0 + static_cast<size_t>(8 * nt + c2 + (i & 1)) * p.V + vcol + (i >> 1) * 8;
      if (in_range(p.status, at, 1, st_extent, CHK_SCAN_STATE)) fin[at] = acc[nt][i];
    }
}

// Turns each segment's own end state into the sequence's, E_g = E_{g-1} 2^dec_g
// + own_g, and writes the last one as the final state.  A thread takes 4
// neighbouring elements of a tile; grid y runs over the tiles.
__global__ void __launch_bounds__(256) join_kernel(const ScanParams p, float* ends, const float* cdec,
                                                   float* fin, int first_pair) {
  let_next_begin();
  await_before();
  const int per = kCols * p.K, at = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= per) return;
  const int gbx = first_pair + blockIdx.y, groups = p.Nq * p.nhb;
  const int b = gbx / groups;
  const Place w = place_of(p, b, gbx - b * groups);
  const int blk = at / 64, v = (blk / (p.K / 8)) * 8 + (at % 64) / 8, k = (blk % (p.K / 8)) * 8 + at % 8;
  const int vh = v / p.V;
  if (vh >= w.heads) return;
  const size_t head = static_cast<size_t>(b) * p.N + w.head0 + vh;
  float* own = ends + static_cast<size_t>(gbx) * p.nseg * per + at;
  const float* dec = cdec + static_cast<size_t>(p.B) * p.N * p.nc + head * p.nseg;
  const size_t extent = static_cast<size_t>(p.B) * groups * p.nseg * per;
  float4 s = *reinterpret_cast<const float4*>(own);
  constexpr int U = 14;  // loads in flight
  for (int g0 = 1; g0 < p.nseg; g0 += U) {
    float4 x[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u;
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      d[u] = 0.f;
      if (g < p.nseg && in_range(p.status, (static_cast<size_t>(gbx) * p.nseg + g) * per + at, 4, extent,
                                 CHK_SCAN_WS)) {
        x[u] = *reinterpret_cast<const float4*>(own + static_cast<size_t>(g) * per);
        d[u] = dec[g];  // (written by the kernel before: not read-only memory)
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u;
      if (g >= p.nseg) break;
      const float f = ex2(d[u]);
      s = make_float4(fmaf(s.x, f, x[u].x), fmaf(s.y, f, x[u].y), fmaf(s.z, f, x[u].z), fmaf(s.w, f, x[u].w));
      *reinterpret_cast<float4*>(own + static_cast<size_t>(g) * per) = s;
    }
  }
  if (fin == nullptr) return;
  const float r[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const size_t to = (head * p.K + k + i) * p.V + v % p.V;
    if (in_range(p.status, to, 1, static_cast<size_t>(p.B) * p.N * p.K * p.V, CHK_SCAN_STATE)) fin[to] = r[i];
  }
}

template <bool F32, int KT, bool REV>
cudaError_t run(const ScanParams& p, cudaStream_t st) {
  constexpr int P = Terms<F32>::in, K = 8 * KT;
  constexpr int smem = 4 * kChunk * 4 + 2 * P * kChunk * (K + 8 + kVLd) * 2;
  const long long pairs = static_cast<long long>(p.B) * p.Nq * p.nhb;
  const cudaError_t e = allow_smem<states_kernel<F32, KT, REV>>(smem);
  if (e != cudaSuccess) return e;
  states_kernel<F32, KT, REV><<<static_cast<unsigned>(pairs * p.nseg), kThreads, smem, st>>>(p);
  if (p.nseg > 1)
    for (long long y0 = 0; y0 < pairs; y0 += 65535)  // (nseg > 1 means few pairs: one launch)
    {
      const dim3 grid((kCols * K / 4 + 255) / 256, static_cast<unsigned>(pairs - y0 < 65535 ? pairs - y0 : 65535));
      const cudaError_t j = launch_after(join_kernel, grid, 256, 0, st, p, REV ? p.Rseg : p.Hseg,
                                         REV ? p.rdec : p.cdec, REV ? p.dH0 : p.HT, static_cast<int>(y0));
      if (j != cudaSuccess) return j;
    }
  return cudaGetLastError();
}

template <bool F32, bool REV>
cudaError_t run_k(const ScanParams& p, cudaStream_t st) {
  switch (p.K) {
    case 16: return run<F32, 2, REV>(p, st);
    case 32: return run<F32, 4, REV>(p, st);
    case 64: return run<F32, 8, REV>(p, st);
    default: return run<F32, 16, REV>(p, st);
  }
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_states(const ScanParams& p, bool f32, bool reverse, cudaStream_t st) {
  if (f32) return reverse ? scan::run_k<true, true>(p, st) : scan::run_k<true, false>(p, st);
  return reverse ? scan::run_k<false, true>(p, st) : scan::run_k<false, false>(p, st);
}

}  // namespace m2rnn

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
// decayed values are the A operand (two bf16 terms, made in registers), the
// keys the B operand.  The chain is sequential in chunks, so where there
// are fewer (sequence, head block) pairs than the SMs take, a sequence is cut
// into segments: a first launch computes each segment's contribution alone, a
// small one joins them, and this kernel runs again from the joined states,
// writing them.  The second reading of k and v costs 36 of the operator's 74
// bytes per token and head (K = 64, V = 16) and replaces a chain that would
// leave most SMs idle.
#include "m2rnn_scan.cuh"

namespace m2rnn {
namespace scan {
namespace {

template <bool F32, int KT, bool REV, bool WRITE>
__global__ void __launch_bounds__(kThreads) states_kernel(const ScanParams p) {
  using E = typename Elem<F32>::T;
  constexpr int P = Terms<F32>::in, PS = Terms<F32>::state, K = 8 * KT, kLd = K + 8;
  constexpr int kKey = P * kChunk * kLd * 2, kVal = P * kChunk * kVLd * 2;
  extern __shared__ __align__(128) unsigned char smem[];
  float(*weights)[kChunk] = reinterpret_cast<float(*)[kChunk]>(smem);
  const uint32_t key0 = ptx::smem_addr(smem) + 4 * kChunk * 4, val0 = key0 + 2 * kKey;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c2 = (lane & 3) * 2;
  const int nseg = WRITE ? p.nseg : p.nseg - 1;
  const int seg = blockIdx.x % nseg, gbx = blockIdx.x / nseg;
  const int gb = gbx % (p.Nq * p.nhb), b = gbx / (p.Nq * p.nhb);
  const Place w = place_of(p, b, gb);
  const int vh = 16 * warp / p.V;  // the warp's head within the block
  const bool on = vh < w.heads;
  const int n = w.head0 + (on ? vh : 0);
  const int first = seg * p.cps, count = min(p.cps, p.nc - first);
  const E* key = static_cast<const E*>(REV ? p.q : p.k) + b * (REV ? p.qb : p.kb) +
                 static_cast<size_t>(w.group) * K;
  const long long key_t = REV ? p.qt : p.kt;
  const E* val = REV ? static_cast<const E*>(p.dy) +
                           (static_cast<size_t>(b) * p.T * p.N + w.head0) * p.V
                     : static_cast<const E*>(p.v) + b * p.vb + static_cast<size_t>(w.head0) * p.V;
  const long long val_t = REV ? static_cast<long long>(p.N) * p.V : p.vt;
  const float alpha = to_f32(static_cast<const E*>(p.alpha)[n]);
  const float beta = to_f32(static_cast<const E*>(p.beta)[n]);
  const size_t sd_extent = static_cast<size_t>(p.B) * p.N * p.nc * kChunk;

  auto chunk_of = [&](int i) { return REV ? p.nc - 1 - (first + i) : first + i; };
  auto fetch = [&](int i) {  // tiles of the i-th chunk of the segment
    const int t0 = chunk_of(i) * kChunk, rows = min(kChunk, p.T - t0);
    load_tile<F32>(key0 + (i & 1) * kKey, key + t0 * key_t, key_t, rows, K, K, kLd, p.status, p.T - t0);
    load_tile<F32>(val0 + (i & 1) * kVal, val + t0 * val_t, val_t, rows, w.heads * p.V, kCols, kVLd,
                   p.status, p.T - t0);
    ptx::cp_async_commit();
  };
  float ga[2];  // the lane's two tokens' gate inputs (forward)
  float4 gs;    // the same tokens' (block sum, dt) pairs (reverse)
  auto fetch_gate = [&](int i) {
    const int c = chunk_of(i), t = c * kChunk + 2 * lane;
    if constexpr (REV) {
      const size_t at = (static_cast<size_t>(b) * p.N + n) * p.nc * kChunk + t;
      gs = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in_range(p.status, at, 2, sd_extent, CHK_SCAN_WS))
        gs = *reinterpret_cast<const float4*>(p.sd + at);
    } else {
      const E* a = static_cast<const E*>(p.a) + b * p.ab + n;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        ga[u] = t + u < p.T && in_range(p.status, t + u, 1, p.T, CHK_SCAN_IN)
                    ? to_f32(a[(t + u) * p.at]) : -INFINITY;
    }
  };

  fetch_gate(0);
  fetch(0);
  // state: accumulator nt holds (column 16 warp + g [+8], key row 8 nt + c2, +1)
  float acc[KT][4];
  const float* init = REV ? p.dHT : p.H0;
  const size_t st0 = (static_cast<size_t>(b) * p.N + n) * K * p.V;
  const size_t st_extent = static_cast<size_t>(p.B) * p.N * K * p.V;
  const int vcol = (16 * warp) % p.V + g;
  const size_t seg_extent = static_cast<size_t>(p.B) * p.Nq * p.nhb * p.nseg * kCols * K;
  auto seg_at = [&](int s) {
    return ((static_cast<size_t>(b) * p.Nq * p.nhb + gb) * p.nseg + s) * kCols * K +
           static_cast<size_t>(warp) * KT * 128 + lane;
  };
#pragma unroll
  for (int nt = 0; nt < KT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[nt][i] = 0.f;
      if (!on) continue;
      if (seg == 0) {
        const size_t at = st0 + static_cast<size_t>(8 * nt + c2 + (i & 1)) * p.V + vcol + (i >> 1) * 8;
        if (init != nullptr && in_range(p.status, at, 1, st_extent, CHK_SCAN_STATE))
          acc[nt][i] = init[at];
      } else if (WRITE) {
        const size_t at = seg_at(seg - 1) + (nt * 4 + i) * 32;
        if (in_range(p.status, at, 1, seg_extent, CHK_SCAN_WS)) acc[nt][i] = p.segst[at];
      }
    }

  float total = 0.f;  // log2 decay of the segment so far
  for (int i = 0; i < count; ++i) {
    const int c = chunk_of(i);
    // The gate's sums.  Blocks of 16 tokens are 8 lanes; loc: from the block's
    // start up to the lane's tokens, rest: from behind them to its end.
    float wt[2], chunk_sum;
    {
      float l0, l1, dt0 = 0.f, dt1 = 0.f, loc0, loc1;
      if constexpr (REV) {
        loc0 = gs.x;
        loc1 = gs.z;
      } else {
        dt0 = gate_softplus(ga[0] + beta);
        dt1 = gate_softplus(ga[1] + beta);
        // below 2^-160 a decay is 0 in fp32: the bound keeps sums short
        l0 = -alpha * kLog2e * dt0;
        l1 = -alpha * kLog2e * dt1;
        l0 = l0 < -160.f ? -160.f : l0;
        l1 = l1 < -160.f ? -160.f : l1;
        float inc = l0 + l1, suf = inc;
#pragma unroll
        for (int d = 1; d < 8; d *= 2) {
          const float up = __shfl_up_sync(0xffffffffu, inc, d, 8);
          const float dn = __shfl_down_sync(0xffffffffu, suf, d, 8);
          if ((lane & 7) >= d) inc += up;
          if ((lane & 7) + d < 8) suf += dn;
        }
        loc1 = inc;
        const float before = __shfl_up_sync(0xffffffffu, inc, 1, 8);
        loc0 = ((lane & 7) ? before : 0.f) + l0;
        const float behind = __shfl_down_sync(0xffffffffu, suf, 1, 8);
        wt[1] = (lane & 7) < 7 ? behind : 0.f;  // after the second token
        wt[0] = wt[1] + l1;
      }
      float tot[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) tot[k] = __shfl_sync(0xffffffffu, loc1, 8 * k + 7);
      const int blk = lane >> 3;
      float off = 0.f;
      if constexpr (REV) {
#pragma unroll
        for (int k = 0; k < 3; ++k) off += k < blk ? tot[k] : 0.f;
        wt[0] = ex2(off + loc0);
        wt[1] = ex2(off + loc1);
      } else {
#pragma unroll
        for (int k = 3; k > 0; --k) off += k > blk ? tot[k] : 0.f;
        wt[0] = ex2(off + wt[0]) * dt0;
        wt[1] = ex2(off + wt[1]) * dt1;
        const size_t at = (static_cast<size_t>(b) * p.N + n) * p.nc * kChunk + c * kChunk + 2 * lane;
        if (WRITE && on && (16 * warp) % p.V == 0 && in_range(p.status, at, 2, sd_extent, CHK_SCAN_WS))
          *reinterpret_cast<float4*>(p.sd + at) = make_float4(loc0, dt0, loc1, dt1);
      }
      chunk_sum = (tot[0] + tot[1]) + (tot[2] + tot[3]);
      weights[warp][2 * lane] = wt[0];
      weights[warp][2 * lane + 1] = wt[1];
    }
    total += chunk_sum;
    if (i + 1 < count) fetch_gate(i + 1);
    cp_async_wait<0>();
    __syncthreads();  // tiles of chunk i are there; everyone is done with chunk i - 1
    if (i + 1 < count) fetch(i + 1);
    if (on) {
      if (WRITE) {
        __nv_bfloat16* dst = (REV ? p.Rs : p.Hs) + state_at(p, PS, b, gb, c);
        const size_t extent = state_at(p, PS, p.B, 0, 0);
#pragma unroll
        for (int nt = 0; nt < KT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t t[PS];
            split<PS>(acc[nt][2 * h], acc[nt][2 * h + 1], t);
#pragma unroll
            for (int s = 0; s < PS; ++s) {
              const size_t at = static_cast<size_t>(s) * kCols * K + ((2 * warp + h) * KT + nt) * 64 + 2 * lane;
              if (in_range(p.status, (dst - (REV ? p.Rs : p.Hs)) + at, 2, extent, CHK_SCAN_WS))
                *reinterpret_cast<uint32_t*>(dst + at) = t[s];
            }
          }
      }
      const float dec = ex2(chunk_sum);
#pragma unroll
      for (int nt = 0; nt < KT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[nt][j] *= dec;
      const uint32_t kt = key0 + (i & 1) * kKey, vt = val0 + (i & 1) * kVal;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t raw[P][4], a[PS][4];
        load_a_t<P>(raw, vt, kVLd, 16 * ks, 16 * warp);
        const float2 w0 = *reinterpret_cast<const float2*>(&weights[warp][16 * ks + c2]);
        const float2 w1 = *reinterpret_cast<const float2*>(&weights[warp][16 * ks + 8 + c2]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t x[P], t[PS];
#pragma unroll
          for (int s = 0; s < P; ++s) x[s] = raw[s][r];
          const float2 v = join<P>(x);
          const float2 ww = r < 2 ? w0 : w1;
          split<PS>(v.x * ww.x, v.y * ww.y, t);
#pragma unroll
          for (int s = 0; s < PS; ++s) a[s][r] = t[s];
        }
#pragma unroll
        for (int nt = 0; nt < KT; nt += 2) {
          uint32_t b0[P][2], b1[P][2];
          load_b2_t<P>(b0, b1, kt, kLd, 16 * ks, 8 * nt);
          mma_terms<PS, P>(acc[nt], a, b0);
          mma_terms<PS, P>(acc[nt + 1], a, b1);
        }
      }
    }
    __syncwarp();  // the warp's weights may be overwritten
  }
  if (!on) return;
  if (!WRITE) {
#pragma unroll
    for (int nt = 0; nt < KT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t at = seg_at(seg) + (nt * 4 + i) * 32;
        if (in_range(p.status, at, 1, seg_extent, CHK_SCAN_WS)) p.segst[at] = acc[nt][i];
      }
    const size_t at = (static_cast<size_t>(b) * p.N + n) * p.nseg + seg;
    if (lane == 0 && (16 * warp) % p.V == 0 &&
        in_range(p.status, at, 1, static_cast<size_t>(p.B) * p.N * p.nseg, CHK_SCAN_WS))
      p.segdec[at] = total;
    return;
  }
  float* fin = REV ? p.dH0 : p.HT;
  if (seg != p.nseg - 1 || fin == nullptr) return;
#pragma unroll
  for (int nt = 0; nt < KT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t at = st0 + static_cast<size_t>(8 * nt + c2 + (i & 1)) * p.V + vcol + (i >> 1) * 8;
      if (in_range(p.status, at, 1, st_extent, CHK_SCAN_STATE)) fin[at] = acc[nt][i];
    }
}

// Joins the segments: turns each segment's own end state into the sequence's,
// E_g = E_{g-1} 2^dec_g + own_g.  One thread per state element.
__global__ void __launch_bounds__(256) join_kernel(const ScanParams p) {
  const int per = kCols * p.K;
  const long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= static_cast<long long>(p.B) * p.Nq * p.nhb * per) return;
  const long long gbx = e / per;
  const int at = static_cast<int>(e - gbx * per);
  const int gb = static_cast<int>(gbx % (p.Nq * p.nhb)), b = static_cast<int>(gbx / (p.Nq * p.nhb));
  const Place w = place_of(p, b, gb);
  const int vh = 16 * (at / (16 * p.K)) / p.V;
  if (vh >= w.heads) return;
  float* own = p.segst + (gbx * p.nseg) * per + at;
  const float* dec = p.segdec + (static_cast<size_t>(b) * p.N + w.head0 + vh) * p.nseg;
  const size_t extent = static_cast<size_t>(p.B) * p.Nq * p.nhb * p.nseg * per;
  float s = own[0];
  constexpr int U = 8;  // loads in flight
  for (int g0 = 1; g0 < p.nseg - 1; g0 += U) {
    float x[U], d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u;
      x[u] = d[u] = 0.f;
      if (g < p.nseg - 1 && in_range(p.status, (gbx * p.nseg + g) * per + at, 1, extent, CHK_SCAN_WS)) {
        x[u] = own[static_cast<size_t>(g) * per];
        d[u] = dec[g];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u;
      if (g >= p.nseg - 1) break;
      s = fmaf(s, ex2(d[u]), x[u]);
      own[static_cast<size_t>(g) * per] = s;
    }
  }
}

template <bool F32, int KT, bool REV>
cudaError_t run(const ScanParams& p, cudaStream_t st) {
  constexpr int P = Terms<F32>::in, K = 8 * KT;
  constexpr int smem = 4 * kChunk * 4 + 2 * P * kChunk * (K + 8 + kVLd) * 2;
  const long long pairs = static_cast<long long>(p.B) * p.Nq * p.nhb;
  auto own = states_kernel<F32, KT, REV, false>;
  auto write = states_kernel<F32, KT, REV, true>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(own, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(write, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  if (p.nseg > 1) {
    own<<<static_cast<unsigned>(pairs * (p.nseg - 1)), kThreads, smem, st>>>(p);
    if (p.nseg > 2)
      join_kernel<<<static_cast<unsigned>((pairs * kCols * K + 255) / 256), 256, 0, st>>>(p);
  }
  write<<<static_cast<unsigned>(pairs * p.nseg), kThreads, smem, st>>>(p);
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

int scan_state_terms(bool f32) {
  return f32 ? scan::Terms<true>::state : scan::Terms<false>::state;
}

cudaError_t launch_scan_states(const ScanParams& p, bool f32, bool reverse, cudaStream_t st) {
  if (f32) return reverse ? scan::run_k<true, true>(p, st) : scan::run_k<true, false>(p, st);
  return reverse ? scan::run_k<false, true>(p, st) : scan::run_k<false, false>(p, st);
}

}  // namespace m2rnn

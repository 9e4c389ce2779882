// m2rnn_addnorm.cu -- the residual's addition with the RMS norm behind it, its
// gradient, its 8-bit output, and the quantiser of rows.
//
// A row belongs to a group of 1 to 16 warps whose threads hold it in registers
// (vectors of 8 elements, `NV` each): one pass over memory, the mean square between
// load and store.  Bound by HBM: 4 D e bytes per row forward (e the element's size),
// 4 D e backward.
#include "m2rnn_ffn.h"
#include "m2rnn_vec.cuh"

namespace m2rnn {
namespace {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The larger one; NaN if either is.
__device__ __forceinline__ float nan_max(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = nan_max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Two e4m3 codes (round to nearest even, saturating; NaN stays NaN), lo in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 codes of o / scale.  The reciprocal is held to twice fp32 (hi + lo, 2^-47 off; Brisebarre and
// Muller's multiplication by a constant of two parts), so the product, rounded once by the fma,
// is the rounded quotient: quotients of bf16 values do
// fall on the middle between two codes, and the rounded reciprocal alone changed the codes of 1
// in 10^3 of them.  True divisions only where the parts might leave fp32's range.
struct Reciprocal {
  float scale, hi, lo;
};
__device__ __forceinline__ Reciprocal reciprocal_of(float scale) {
  Reciprocal r;
  r.scale = scale;
  r.hi = 1.f / scale;
  r.lo = fmaf(-scale, r.hi, 1.f) * r.hi;
  return r;
}
__device__ __forceinline__ uint2 codes8(const float (&o)[8], const Reciprocal& r) {
  float c[8];
  if (r.scale > 1e-30f && r.scale < 1e30f) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 x = make_float2(o[j], o[j + 1]), q = fma2(x, both(r.hi), mul2(x, both(r.lo)));
      c[j] = q.x;
      c[j + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = r.scale == 0.f ? 0.f : __fdiv_rn(o[j], r.scale);
  }
  return make_uint2(e4m3x2(c[0], c[1]) | (e4m3x2(c[2], c[3]) << 16), e4m3x2(c[4], c[5]) | (e4m3x2(c[6], c[7]) << 16));
}

// Sums (or maxima) over a row's warps, in warp order; a CTA of more than one warp per row
// holds one row.
template <int N, bool MAX>
__device__ __forceinline__ void row_reduce(float (&v)[N], int warps, float* sm) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = MAX ? warp_max(v[i]) : warp_sum(v[i]);
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) sm[warp * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = sm[i];
    for (int w = 1; w < warps; ++w) s = MAX ? nan_max(s, sm[w * N + i]) : s + sm[w * N + i];
    v[i] = s;
  }
  __syncthreads();
}

// Offset of a row, and the elements that the rows span.
__device__ __forceinline__ size_t row_at(const Norm2Params& p, long long row, long long batch, long long token) {
  if (p.T == p.M) return static_cast<size_t>(row) * token;
  const unsigned b = static_cast<unsigned>(row) / static_cast<unsigned>(p.T);
  return static_cast<size_t>(b) * batch + static_cast<size_t>(row - static_cast<long long>(b) * p.T) * token;
}
__device__ __forceinline__ size_t rows_span(const Norm2Params& p, long long batch, long long token) {
  return static_cast<size_t>(p.M / p.T - 1) * batch + static_cast<size_t>(p.T - 1) * token + p.D;
}

// ADD: r = x + res is stored.  Q8: the output as codes and a scale.  us in a loop (floor), bf16, fp32:
// M=65536 D=1024 80.3 (78.9), 157 (158), 8 bits 72.3 (69.0), 126 (128); M=4096 D=16384 81.1 (78.9),
// 175 (158), 8 bits 80.0 (69.0), 159 (128).  Rows just above 4,096 fill little more than half of 8 warps'
// four vectors: M=16384 D=4104 90 (79), 160 (158), 8 bits 116 (69), 186 (128).
template <bool F32, int NV, bool ADD, bool Q8>
__global__ void __launch_bounds__(512) add_norm_kernel(Norm2Params p, int warps, int rows_per_cta) {
  using T = typename Elem<F32>::T;
  __shared__ float sm[32];
  const int group = warps * 32, vecs = p.D / 8;
  const int lane = warps == 1 ? threadIdx.x & 31 : threadIdx.x;
  const long long row = static_cast<long long>(blockIdx.x) * rows_per_cta + (warps == 1 ? threadIdx.x >> 5 : 0);
  if (row >= p.M) return;  // (whole warps; CTAs of several warps per row hold one row)
  const size_t D = p.D, n = static_cast<size_t>(p.M) * D, at = static_cast<size_t>(row) * D;
  const size_t x0 = row_at(p, row, p.xb, p.xt), r0 = ADD ? row_at(p, row, p.rb, p.rt) : 0;
  const T* x = static_cast<const T*>(p.x) + x0;
  const T* res = ADD ? static_cast<const T*>(p.res) + r0 : nullptr;
  const size_t x_ext = rows_span(p, p.xb, p.xt), res_ext = ADD ? rows_span(p, p.rb, p.rt) : 0;
  Raw<F32, 8> xv[NV], rv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + i * group;
    xv[i] = rv[i] = raw_zero<F32, 8>();
    if (v < vecs) {
      if (in_range(p.status, x0 + 8 * v, 8, x_ext, CHK_NORM2_IN))
        xv[i] = raw_load<F32, 8, false>(x + 8 * v);
      if (ADD && in_range(p.status, r0 + 8 * v, 8, res_ext, CHK_NORM2_IN))
        rv[i] = raw_load<F32, 8, false>(res + 8 * v);
    }
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + i * group;
    float o[8];
    raw_unpack<F32, 8>(xv[i], o);
    if constexpr (ADD) {
      float b[8];
      raw_unpack<F32, 8>(rv[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += b[j];
      // rounded as it is stored: the norm acts on the stream that the next layer reads
      xv[i] = raw_pack<F32, 8>(o);
      raw_unpack<F32, 8>(xv[i], o);
      if (v < vecs && in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_OUT))
        raw_store<F32, 8>(static_cast<T*>(p.r) + at + 8 * v, xv[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = fmaf(o[j], o[j], ss[0]);
  }
  row_reduce<1, false>(ss, warps, sm);
  const float rstd = 1.f / sqrtf(ss[0] / static_cast<float>(p.D) + p.eps);
  const auto weights = [&](int v, float (&w)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    if (p.w != nullptr && v < vecs && in_range(p.status, 8 * v, 8, D, CHK_NORM2_PARAM))
      load_vec<F32, 8>(static_cast<const T*>(p.w) + 8 * v, w);
  };
  if constexpr (!Q8) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * group;
      float o[8], w[8];
      raw_unpack<F32, 8>(xv[i], o);
      weights(v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = o[j] * rstd * w[j];
      if (v < vecs && in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_OUT))
        store_vec<F32, 8>(static_cast<T*>(p.y) + at + 8 * v, o);
    }
  } else {
    // rstd leaves the quotient y / scale, which is 448 w r / max|w r|.  From bf16, w r has 16 bits and
    // 448 w r 19, both exact, so the codes are the formula's; through y and the scale, each of them
    // rounded, 1 in 10^4 lay on the other side of a middle that the formula meets.
    float top[1] = {0.f};
    float keep[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * group;
      float w[8];
      raw_unpack<F32, 8>(xv[i], keep[i]);
      weights(v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        keep[i][j] *= w[j];
        if (v < vecs) top[0] = nan_max(top[0], fabsf(keep[i][j]));
      }
    }
    row_reduce<1, true>(top, warps, sm);
    float scale = __fdiv_rn(top[0] * rstd, kE4m3Max);
    const auto put = [&](int v, const float (&o)[8], const Reciprocal& inv) {
      if (v < vecs && in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_OUT))
        *reinterpret_cast<uint2*>(p.q + at + 8 * v) = codes8(o, inv);
    };
    // (the whole row takes the same way)
    if (top[0] > 1e-25f && top[0] < 1e25f && scale > 1e-30f && scale < 1e30f) {
      const Reciprocal inv = reciprocal_of(top[0]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) keep[i][j] *= kE4m3Max;
        put(lane + i * group, keep[i], inv);
      }
    } else {
      // Products or squares may have left fp32's range: the codes of y as it is, from r in memory
      // (a rare row: its registers would be every row's).
      const auto y_of = [&](int v, float (&o)[8]) {
        Raw<F32, 8> r = raw_zero<F32, 8>();
        if (ADD ? in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_OUT) : in_range(p.status, x0 + 8 * v, 8, x_ext, CHK_NORM2_IN))
          r = raw_load<F32, 8, false>((ADD ? static_cast<const T*>(p.r) + at : x) + 8 * v);
        float w[8];
        raw_unpack<F32, 8>(r, o);
        weights(v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = o[j] * rstd * w[j];
      };
      top[0] = 0.f;
#pragma unroll 1
      for (int v = lane; v < vecs; v += group) {
        float o[8];
        y_of(v, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) top[0] = nan_max(top[0], fabsf(o[j]));
      }
      row_reduce<1, true>(top, warps, sm);
      scale = __fdiv_rn(top[0], kE4m3Max);
      const Reciprocal inv = reciprocal_of(scale);
#pragma unroll 1
      for (int v = lane; v < vecs; v += group) {
        float o[8];
        y_of(v, o);
        put(v, o, inv);
      }
    }
    if (lane == 0 && in_range(p.status, row, 1, p.M, CHK_NORM2_OUT)) p.scale[row] = scale;
  }
}

// The quantiser: a CTA per row (four rows where one warp holds a row), whose threads keep NV
// vectors each; what is behind those is read a second time.  Bound by HBM where enough
// is in flight: M=16384 D=5632 bf16 42 us (floor 41), 51 with 256 threads of four vectors.
template <bool F32, int NV>
__global__ void __launch_bounds__(256, F32 ? (NV == 4 ? 4 : NV == 6 ? 3 : 2) : (NV == 8 ? 3 : 4))
    quant_rows_kernel(Norm2Params p, int threads) {
  using T = typename Elem<F32>::T;
  __shared__ float sm[32];
  const int vecs = p.D / 8, step = threads;
  const int lane = threads == 32 ? threadIdx.x & 31 : threadIdx.x;
  const long long row = threads == 32 ? static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.M) return;  // (whole warps)
  const size_t n = static_cast<size_t>(p.M) * p.D, at = static_cast<size_t>(row) * p.D;
  const size_t x0 = row_at(p, row, p.xb, p.xt), x_ext = rows_span(p, p.xb, p.xt);
  const T* x = static_cast<const T*>(p.x) + x0;
  const auto load = [&](int v) {
    return v < vecs && in_range(p.status, x0 + 8 * v, 8, x_ext, CHK_NORM2_IN) ? raw_load<F32, 8>(x + 8 * v)
                                                                              : raw_zero<F32, 8>();
  };
  Raw<F32, 8> keep[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) keep[i] = load(lane + i * step);
  float top[1] = {0.f};
  __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);  // bf16: the largest of packed pairs, exact
  const auto take = [&](const Raw<F32, 8>& r) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) top[0] = nan_max(top[0], fabsf(__uint_as_float(r.w[j])));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = r.w[j] & 0x7FFF7FFFu;
        top2 = __hmax2_nan(top2, reinterpret_cast<const __nv_bfloat162&>(a));
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) take(keep[i]);
  for (int v = lane + NV * step; v < vecs; v += step) take(load(v));
  if constexpr (!F32) top[0] = nan_max(__low2float(top2), __high2float(top2));
  row_reduce<1, true>(top, threads / 32, sm);
  const float scale = __fdiv_rn(top[0], kE4m3Max);
  const Reciprocal inv = reciprocal_of(scale);
  if (lane == 0 && in_range(p.status, row, 1, p.M, CHK_NORM2_OUT)) p.scale[row] = scale;
  const auto put = [&](int v, const Raw<F32, 8>& r) {
    float o[8];
    raw_unpack<F32, 8>(r, o);
    if (v < vecs && in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_OUT))
      *reinterpret_cast<uint2*>(p.q + at + 8 * v) = codes8(o, inv);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) put(lane + i * step, keep[i]);
  for (int v = lane + NV * step; v < vecs; v += step) put(v, load(v));
}

// Backward: with n = r rstd, p = w dy:  dx = dr + rstd (p - n mean(p n)),  dw = sum dy n.
// A CTA holds several groups of warps, each of which walks over rows with its share of dw in
// registers.  A thread copies its vectors of the next S rows into its own places of shared
// memory (asynchronously, so they take no registers while they are in flight: 96 KB to a
// CTA of 256 threads, 48 KB with one vector of bf16, 192 KB to one of 512), and reads them twice,
// for the two sums and for dx.  dw is summed over runs of kRun
// rows, and those apart, so that long sums do not drift; then over groups, then over CTAs
// (sum_parts), always in the same order.  M=32768 D=2048: 88 us, 111 with the next row in
// registers instead.  With dw, in a loop, TB/s of bf16, fp32: D=1024 6.1, 4.0, D=4096 6.0, 4.1.  Above
// 4,096 there is one CTA to an SM, in fp32 with one slot, so that a row's copies and
// arithmetic take turns: D=4104 2.2, 2.6, D=8192 4.2, 3.3, D=16384 5.9, 3.6.
constexpr int kRun = 64;
template <bool F32, int NV>
struct BwdCfg {
  static constexpr int CTA = NV == 4 ? 512 : 256;
  static constexpr int U = F32 ? 2 : 1;  // 16-byte units of a vector
  static constexpr int S = NV == 4 ? (F32 ? 1 : 2) : NV * U == 4 ? 2 : 4;
  static constexpr int RING = S * 3 * NV * U * CTA * 16;
  // the runs' sums of dw (NV = 4, whose CTA is one group: in its part in memory instead)
  static constexpr int SMEM = RING + (NV == 4 ? 0 : CTA * NV * 8 * 4);
};

template <bool F32, int NV>
__global__ void __launch_bounds__(BwdCfg<F32, NV>::CTA, NV == 4 ? 1 : 2) add_norm_bwd_kernel(Norm2Params p, int warps) {
  using T = typename Elem<F32>::T;
  using C = BwdCfg<F32, NV>;
  constexpr int CTA = C::CTA, U = C::U, S = C::S;
  // [S][3][NV][U][CTA] 16-byte units (in the end [groups][D] floats), [NV][8][CTA] floats
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 sums[2][CTA / 32];
  const int group = warps * 32, vecs = p.D / 8, groups = CTA / group;
  const int lane = threadIdx.x % group, mine = threadIdx.x / group;
  let_next_begin();
  const size_t D = p.D, n = static_cast<size_t>(p.M) * D;
  const size_t r_ext = rows_span(p, p.xb, p.xt);
  float dw[NV][8];
  Raw<F32, 8> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + i * group;
    float one[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[i][j] = 0.f;
      one[j] = 1.f;
    }
    w[i] = raw_pack<F32, 8>(one);
    if (p.w != nullptr && v < vecs && in_range(p.status, 8 * v, 8, D, CHK_NORM2_PARAM))
      w[i] = raw_load<F32, 8>(static_cast<const T*>(p.w) + 8 * v);
  }
  const uint32_t base = ptx::smem_addr(ring) + threadIdx.x * 16;
  const auto place = [&](int slot, int which, int i) { return base + ((slot * 3 + which) * NV + i) * U * CTA * 16; };
  const auto fetch = [&](int slot, long long row) {
    const size_t at = static_cast<size_t>(row) * D, r0 = row_at(p, row, p.xb, p.xt);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * group;
      if (v < vecs && row < p.M) {
        const bool r_in = in_range(p.status, r0 + 8 * v, 8, r_ext, CHK_NORM2_IN);
        const bool in = in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_IN);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          constexpr int E = 16 / sizeof(T);
          if (r_in) ptx::cp_async16(place(slot, 0, i) + u * CTA * 16, static_cast<const T*>(p.x) + r0 + 8 * v + u * E);
          if (in) ptx::cp_async16(place(slot, 1, i) + u * CTA * 16, static_cast<const T*>(p.dy) + at + 8 * v + u * E);
          if (in && p.dr != nullptr)
            ptx::cp_async16(place(slot, 2, i) + u * CTA * 16, static_cast<const T*>(p.dr) + at + 8 * v + u * E);
        }
      }
    }
    ptx::cp_async_commit();
  };
  const auto read = [&](int slot, int which, int i, float (&o)[8]) {
    Raw<F32, 8> r = raw_zero<F32, 8>();
    if (lane + i * group < vecs) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint4 q = ptx::lds_u32x4(place(slot, which, i) + u * CTA * 16);
        r.w[4 * u] = q.x;
        r.w[4 * u + 1] = q.y;
        r.w[4 * u + 2] = q.z;
        r.w[4 * u + 3] = q.w;
      }
    }
    raw_unpack<F32, 8>(r, o);
  };
  // Moves a run's sums of dw to those of the runs before (thread by thread).
  float* runs = reinterpret_cast<float*>(ring + C::RING) + threadIdx.x;
  bool first = true;
  const auto end_run = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * group;
      if constexpr (NV == 4) {
        const size_t at = static_cast<size_t>(blockIdx.x) * D + 8 * v;
        if (v < vecs && in_range(p.status, at, 8, static_cast<size_t>(p.nparts) * D, CHK_NORM2_PARAM)) {
          float o[8];
          if (!first) {
            raw_unpack<true, 8>(raw_load<true, 8, false>(p.part + at), o);
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[i][j] += o[j];
          }
          store_vec<true, 8>(p.part + at, dw[i]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float& sum = runs[(i * 8 + j) * CTA];
          sum = first ? dw[i][j] : sum + dw[i][j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    first = false;
  };
  const long long step = static_cast<long long>(gridDim.x) * groups;
  long long row = static_cast<long long>(blockIdx.x) * groups + mine;
#pragma unroll
  for (int k = 0; k < S; ++k) fetch(k, row + k * step);
  int slot = 0, rows = 0;
  for (int turn = 0; row < p.M; row += step, turn ^= 1) {  // (the same count in all warps of a group)
    const size_t at = static_cast<size_t>(row) * D;
    ptx::cp_async_wait<S - 1>();
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[8], dy[8], wf[8];
      read(slot, 0, i, r);
      read(slot, 1, i, dy);
      raw_unpack<F32, 8>(w[i], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = fmaf(r[j], r[j], s[0]);
        s[1] = fmaf(r[j], dy[j] * wf[j], s[1]);
      }
    }
    s[0] = warp_sum(s[0]);
    s[1] = warp_sum(s[1]);
    if (warps > 1) {
      float2* mem = sums[turn] + mine * warps;
      if ((threadIdx.x & 31) == 0) mem[lane >> 5] = make_float2(s[0], s[1]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "r"(group) : "memory");
      s[0] = s[1] = 0.f;
      for (int i = 0; i < warps; ++i) {
        s[0] += mem[i].x;
        s[1] += mem[i].y;
      }
    }
    const float rstd = 1.f / sqrtf(s[0] / static_cast<float>(p.D) + p.eps);
    const float c = s[1] * rstd / static_cast<float>(p.D);  // mean(p n)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * group;
      float r[8], dy[8], wf[8], o[8];
      read(slot, 0, i, r);
      read(slot, 1, i, dy);
      raw_unpack<F32, 8>(w[i], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 0.f;
      if (p.dr != nullptr) read(slot, 2, i, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float nj = r[j] * rstd;
        o[j] += rstd * (wf[j] * dy[j] - nj * c);
        dw[i][j] = fmaf(dy[j], nj, dw[i][j]);
      }
      if (v < vecs && in_range(p.status, at + 8 * v, 8, n, CHK_NORM2_OUT))
        store_vec<F32, 8>(static_cast<T*>(p.dx) + at + 8 * v, o);
    }
    fetch(slot, row + S * step);  // (the thread has read its places)
    slot = slot + 1 == S ? 0 : slot + 1;
    if (++rows % kRun == 0 && p.part != nullptr) end_run();
  }
  ptx::cp_async_wait_all();
  if (p.part == nullptr) return;
  end_run();
  if constexpr (NV == 4) return;
  float* share = reinterpret_cast<float*>(ring);
  __syncthreads();  // (the rows in the ring have been read)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lane + i * group;
    if (v < vecs) {
#pragma unroll
      for (int j = 0; j < 8; ++j) share[mine * p.D + 8 * v + j] = runs[(i * 8 + j) * CTA];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += CTA) {
    float s = 0.f;
    for (int g = 0; g < groups; ++g) s += share[g * p.D + d];
    const size_t at = static_cast<size_t>(blockIdx.x) * D + d;
    if (in_range(p.status, at, 1, static_cast<size_t>(p.nparts) * D, CHK_NORM2_PARAM)) p.part[at] = s;
  }
}

// Vectors per thread and warps per row: the fewest warps (1, 2, 4, 8, 16) whose threads
// hold the row in `most` vectors each (four where 16 warps do not), and then as few vectors as that takes.
struct RowPlan {
  int nv, warps;
};
RowPlan row_plan(int D, int most) {
  const int vecs = D / 8;
  int warps = 1;
  while (warps < 16 && warps * 32 * most < vecs) warps *= 2;
  const int nv = (vecs + warps * 32 - 1) / (warps * 32);
  return {nv <= 1 ? 1 : nv <= 2 ? 2 : 4, warps};
}

template <bool F32, int NV>
cudaError_t launch_nv(const Norm2Params& p, int warps, cudaStream_t st) {
  const int per = warps == 1 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((p.M + per - 1) / per));
  const int threads = warps == 1 ? 128 : 32 * warps;
  const bool add = p.res != nullptr, q8 = p.q != nullptr;
  if (add && q8)
    add_norm_kernel<F32, NV, true, true><<<grid, threads, 0, st>>>(p, warps, per);
  else if (add)
    add_norm_kernel<F32, NV, true, false><<<grid, threads, 0, st>>>(p, warps, per);
  else if (q8)
    add_norm_kernel<F32, NV, false, true><<<grid, threads, 0, st>>>(p, warps, per);
  else
    add_norm_kernel<F32, NV, false, false><<<grid, threads, 0, st>>>(p, warps, per);
  return cudaGetLastError();
}

template <bool F32>
cudaError_t launch_fwd_t(const Norm2Params& p, int sms, cudaStream_t st) {
  // Few rows: one vector per thread, the row's loads all at once.
  const RowPlan r = row_plan(p.D, p.M <= 2 * sms ? 1 : 4);
  return r.nv == 1 ? launch_nv<F32, 1>(p, r.warps, st)
         : r.nv == 2 ? launch_nv<F32, 2>(p, r.warps, st)
                     : launch_nv<F32, 4>(p, r.warps, st);
}

template <bool F32, int NV>
cudaError_t launch_bwd_nv(const Norm2Params& p, int warps, cudaStream_t st) {
  using C = BwdCfg<F32, NV>;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(add_norm_bwd_kernel<F32, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  add_norm_bwd_kernel<F32, NV><<<p.nparts, C::CTA, C::SMEM, st>>>(p, warps);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.part == nullptr) return e;
  const SumOut o = {{p.dw, nullptr, nullptr}, {p.D, 0, 0}};
  return launch_sum_parts(p.part, p.nparts, o, p.status, CHK_NORM2_PARAM, st);
}
// Up to 8 warps of two vectors per thread (the next rows' are in flight beside them); rows of more than
// 4,096 go to 16 warps of four, of which those up to 8,192 leave half of the places empty.
RowPlan bwd_plan(int D) {
  const int vecs = D / 8;
  int warps = 1;
  while (warps < 8 && warps * 64 < vecs) warps *= 2;
  if (warps * 64 < vecs) return {4, 16};
  return {vecs <= warps * 32 ? 1 : 2, warps};
}
template <bool F32>
cudaError_t launch_bwd_t(const Norm2Params& p, cudaStream_t st) {
  const RowPlan r = bwd_plan(p.D);
  return r.nv == 1 ? launch_bwd_nv<F32, 1>(p, r.warps, st)
         : r.nv == 2 ? launch_bwd_nv<F32, 2>(p, r.warps, st)
                     : launch_bwd_nv<F32, 4>(p, r.warps, st);
}

}  // namespace

// CTAs of the backward kernel: two to each of 152 SMs (one of the 512-thread ones), and a
// row for each group at least.
int add_norm_bwd_parts(const m2rnn_norm_shape* s) {
  const RowPlan r = bwd_plan(s->D);
  const int groups = (r.nv == 4 ? 16 : 8) / r.warps;
  const long long rows = static_cast<long long>(s->B) * s->T;
  const long long most = r.nv == 4 ? 152 : 304, need = (rows + groups - 1) / groups;
  return static_cast<int>(need < most ? need : most);
}

cudaError_t launch_add_norm(const Norm2Params& p, bool f32, int sms, cudaStream_t st) {
  return f32 ? launch_fwd_t<true>(p, sms, st) : launch_fwd_t<false>(p, sms, st);
}
cudaError_t launch_add_norm_bwd(const Norm2Params& p, bool f32, cudaStream_t st) {
  return f32 ? launch_bwd_t<true>(p, st) : launch_bwd_t<false>(p, st);
}
template <bool F32>
static cudaError_t launch_quant_t(const Norm2Params& p, cudaStream_t st) {
  // the fewest threads that hold the row in six vectors each (256: as many as it takes)
  const int vecs = p.D / 8;
  int threads = 32;
  while (threads < 256 && threads * 6 < vecs) threads *= 2;
  const int per = threads == 32 ? 4 : 1, cta = threads * per;
  const unsigned grid = static_cast<unsigned>((p.M + per - 1) / per);
  if (vecs <= 4 * threads)
    quant_rows_kernel<F32, 4><<<grid, cta, 0, st>>>(p, threads);
  else if (vecs <= 6 * threads)
    quant_rows_kernel<F32, 6><<<grid, cta, 0, st>>>(p, threads);
  else
    quant_rows_kernel<F32, 8><<<grid, cta, 0, st>>>(p, threads);
  return cudaGetLastError();
}
cudaError_t launch_quant_rows(const Norm2Params& p, bool f32, cudaStream_t st) {
  return f32 ? launch_quant_t<true>(p, st) : launch_quant_t<false>(p, st);
}

}  // namespace m2rnn

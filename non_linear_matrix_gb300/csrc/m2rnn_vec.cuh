// m2rnn_vec.cuh -- vector loads and stores of the block operators' elements
// (bf16 or fp32 in memory, fp32 in registers) and the fixed-order sum over
// CTAs' partial results.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "m2rnn_check.cuh"
#include "ptx.cuh"

namespace m2rnn {

template <bool F32>
struct Elem {
  using T = float;
};
template <>
struct Elem<false> {
  using T = __nv_bfloat16;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Pairs of fp32 values in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// The bf16 value that an fp32 value rounds to, or is cut off to where it would round to infinity.
__device__ __forceinline__ float bf16_term(float v) {
  const float t = __bfloat162float(__float2bfloat16_rn(v));
  return isinf(t) && isfinite(v) ? __uint_as_float(__float_as_uint(v) & 0xffff0000u) : t;
}
// VEC (2, 4 or 8) consecutive elements as they lie in memory: 4, 8 or 16 bytes
// of bf16, 8, 16 or 32 bytes of fp32.
template <bool F32, int VEC>
struct Raw {
  uint32_t w[F32 ? VEC : VEC / 2];
};

template <bool F32, int VEC>
__device__ __forceinline__ Raw<F32, VEC> raw_zero() {
  Raw<F32, VEC> r;
#pragma unroll
  for (uint32_t& x : r.w) x = 0u;
  return r;
}

// CONST: through the read-only path, for memory that nobody writes while the kernel
// is resident (a call's inputs, unless the call may update them in place).
template <bool F32, int VEC, bool CONST = true>
__device__ __forceinline__ Raw<F32, VEC> raw_load(const typename Elem<F32>::T* src) {
  const auto get = [](const auto* p) {
    if constexpr (CONST)
      return __ldg(p);
    else
      return *p;
  };
  Raw<F32, VEC> r;
  if constexpr (sizeof(r.w) == 4) {
    r.w[0] = get(reinterpret_cast<const unsigned int*>(src));
  } else if constexpr (sizeof(r.w) == 8) {
    const uint2 u = get(reinterpret_cast<const uint2*>(src));
    r.w[0] = u.x;
    r.w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r.w) / 16); ++i) {
      const uint4 u = get(reinterpret_cast<const uint4*>(src) + i);
      r.w[4 * i] = u.x;
      r.w[4 * i + 1] = u.y;
      r.w[4 * i + 2] = u.z;
      r.w[4 * i + 3] = u.w;
    }
  }
  return r;
}

template <bool F32, int VEC>
__device__ __forceinline__ void raw_store(typename Elem<F32>::T* dst, const Raw<F32, VEC>& r) {
  if constexpr (sizeof(r.w) == 4) {
    *reinterpret_cast<uint32_t*>(dst) = r.w[0];
  } else if constexpr (sizeof(r.w) == 8) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r.w) / 16); ++i)
      reinterpret_cast<uint4*>(dst)[i] =
          make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
  }
}

template <bool F32, int VEC>
__device__ __forceinline__ void raw_unpack(const Raw<F32, VEC>& r, float (&o)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if constexpr (F32)
      o[i] = __uint_as_float(r.w[i]);
    else
      o[i] = (i & 1) ? ptx::bf16x2_hi(r.w[i / 2]) : ptx::bf16x2_lo(r.w[i / 2]);
  }
}

template <bool F32, int VEC>
__device__ __forceinline__ Raw<F32, VEC> raw_pack(const float (&o)[VEC]) {
  Raw<F32, VEC> r;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.w[i] = ptx::pack_bf16x2(o[2 * i], o[2 * i + 1]);
  }
  return r;
}

// The same as pairs.
template <bool F32, int VEC>
__device__ __forceinline__ void raw_unpack2(const Raw<F32, VEC>& r, float2 (&o)[VEC / 2]) {
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    o[i] = F32 ? make_float2(__uint_as_float(r.w[F32 ? 2 * i : 0]), __uint_as_float(r.w[F32 ? 2 * i + 1 : 0]))
               : make_float2(ptx::bf16x2_lo(r.w[F32 ? 0 : i]), ptx::bf16x2_hi(r.w[F32 ? 0 : i]));
}
template <bool F32, int VEC>
__device__ __forceinline__ Raw<F32, VEC> raw_pack2(const float2 (&o)[VEC / 2]) {
  float t[VEC];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    t[2 * i] = o[i].x;
    t[2 * i + 1] = o[i].y;
  }
  return raw_pack<F32, VEC>(t);
}

template <bool F32, int VEC>
__device__ __forceinline__ void load_vec(const typename Elem<F32>::T* src, float (&o)[VEC]) {
  raw_unpack<F32, VEC>(raw_load<F32, VEC>(src), o);
}

template <bool F32, int VEC>
__device__ __forceinline__ void store_vec(typename Elem<F32>::T* dst, const float (&o)[VEC]) {
  raw_store<F32, VEC>(dst, raw_pack<F32, VEC>(o));
}

// A kernel launched by launch_after may begin while the one before it in the
// stream still runs (once all of that one's CTAs have called let_next_begin or
// ended); await_before returns when it has ended and its writes are seen.  Such a
// kernel calls await_before before it touches anything but the call's inputs.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void await_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         const A&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Sums part[nparts][n0 + n1 + n2] over the parts, always in the same order,
// into up to three outputs (NULL: skipped).  A CTA takes 32 columns, its 32
// warps every 32nd part each; the warps' sums are added in warp order.
struct SumOut {
  float* out[3];
  int n[3];
};

static __global__ void __launch_bounds__(1024)
    sum_parts_kernel(const float* part, int nparts, SumOut o, int* status, int site) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = o.n[0] + o.n[1] + o.n[2];
  const int col = blockIdx.x * 32 + lane;
  float s = 0.f;
  await_before();
  if (col < n) {
#pragma unroll 8
    for (int r = warp; r < nparts; r += 32) {
      const size_t at = static_cast<size_t>(r) * n + col;
      if (in_range(status, at, 1, static_cast<size_t>(nparts) * n, site)) s += part[at];
    }
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= n) return;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) t += acc[i][lane];
  int at = col;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (at < o.n[i]) {
      if (o.out[i] != nullptr) o.out[i][at] = t;
      return;
    }
    at -= o.n[i];
  }
}

static cudaError_t launch_sum_parts(const float* part, int nparts, const SumOut& o, int* status,
                                    int site, cudaStream_t st) {
  const int n = o.n[0] + o.n[1] + o.n[2];
  return launch_after(sum_parts_kernel, dim3((n + 31) / 32), 1024, 0, st, part, nparts, o, status, site);
}

}  // namespace m2rnn

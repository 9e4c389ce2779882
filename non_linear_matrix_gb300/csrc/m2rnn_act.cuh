// m2rnn_act.cuh -- the gated product's activations and their derivatives.
//
// act 0: SiLU g s(g), s(x) = 1 / (1 + e^-x).  act 1: GELU in its tanh form, g s(2 c (g +
// 0.044715 g^3)) with c = (2 / pi)^(1/2), since (1 + tanh x) / 2 = s(2 x).
//
// Scalars: by expf and true divisions, for fp32 results.  Pairs: on the special-function unit
// (2^x and reciprocal, relative errors about 2^-22), for results that are rounded to bf16;
// everything else in packed instructions, because the output warps' instructions are what
// bounds a tile's epilogue.
#pragma once
#include <cuda_runtime.h>

#include "m2rnn_vec.cuh"

namespace m2rnn {

constexpr float kGeluC = 0.7978845608028654f;  // (2 / pi)^(1/2)
constexpr float kLog2e = 1.4426950408889634f;

// ---- exact ---------------------------------------------------------------------

__device__ __forceinline__ float gate_of(float g, int act) {
  const float x = act == 0 ? g : 2.f * kGeluC * (g + 0.044715f * g * g * g);
  return 1.f / (1.f + expf(-x));
}
__device__ __forceinline__ float act_of(float g, int act) { return g * gate_of(g, act); }
// act(g) and its derivative.
__device__ __forceinline__ void act_grad(float g, int act, float& a, float& d) {
  const float s = gate_of(g, act);
  a = g * s;
  const float t = a * (1.f - s);  // 0 where the gate is 0 or 1, whatever g^2 overflows to
  d = s + (act == 0 || t == 0.f ? t : t * (2.f * kGeluC) * (1.f + 3.f * 0.044715f * g * g));
}

// ---- pairs, for bf16 results -----------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 gate2(float2 g, int act) {
  float2 x;  // minus the sigmoid's argument, times log2 e
  if (act == 0) {
    x = mul2(g, both(-kLog2e));
  } else {
    const float2 q = fma2(mul2(g, g), both(0.044715f), both(1.f));
    x = mul2(mul2(g, both(-2.f * kGeluC * kLog2e)), q);
  }
  const float2 e = add2(make_float2(ex2(x.x), ex2(x.y)), both(1.f));
  return make_float2(rcp(e.x), rcp(e.y));
}
__device__ __forceinline__ float2 act2(float2 g, int act) { return mul2(g, gate2(g, act)); }
__device__ __forceinline__ void act_grad2(float2 g, int act, float2& a, float2& d) {
  const float2 s = gate2(g, act);
  a = mul2(g, s);
  const float2 r = fma2(s, both(-1.f), both(1.f));
  if (act == 0) {
    d = fma2(a, r, s);
  } else {
    const float2 t = mul2(a, r);
    const float2 q = fma2(mul2(g, g), both(2.f * kGeluC * 3.f * 0.044715f), both(2.f * kGeluC));
    d = make_float2(t.x == 0.f ? s.x : fmaf(t.x, q.x, s.x), t.y == 0.f ? s.y : fmaf(t.y, q.y, s.y));
  }
}

}  // namespace m2rnn

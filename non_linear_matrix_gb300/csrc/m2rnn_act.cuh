// m2rnn_act.cuh -- the gated product's activations and their derivatives.
// EXACT: by expf, tanhf and true divisions, for fp32 results; otherwise by the
// special-function unit (relative error about 2^-21, far below bf16's half step).
#pragma once
#include <cuda_runtime.h>

namespace m2rnn {

template <bool EXACT>
__device__ __forceinline__ float sigmoid_of(float g) {
  if constexpr (EXACT)
    return 1.f / (1.f + expf(-g));
  else
    return __fdividef(1.f, 1.f + __expf(-g));
}

// 1 + tanh of the GELU's argument, halved: a sigmoid of twice the argument.
template <bool EXACT>
__device__ __forceinline__ float gelu_gate(float g) {
  const float c = 0.7978845608028654f;  // (2 / pi)^(1/2)
  return sigmoid_of<EXACT>(2.f * c * (g + 0.044715f * g * g * g));
}

template <bool EXACT>
__device__ __forceinline__ float act_of(float g, int act) {
  return g * (act == 0 ? sigmoid_of<EXACT>(g) : gelu_gate<EXACT>(g));
}

// act(g) and its derivative.
template <bool EXACT>
__device__ __forceinline__ void act_grad(float g, int act, float& a, float& d) {
  if (act == 0) {
    const float s = sigmoid_of<EXACT>(g);
    a = g * s;
    d = s + a * (1.f - s);
  } else {
    const float s = gelu_gate<EXACT>(g), c = 0.7978845608028654f;
    a = g * s;
    const float t = a * (1.f - s);  // 0 where the gate is 0 or 1, whatever g^2 overflows to
    d = s + (t == 0.f ? 0.f : t * (2.f * c) * (1.f + 3.f * 0.044715f * g * g));
  }
}

}  // namespace m2rnn

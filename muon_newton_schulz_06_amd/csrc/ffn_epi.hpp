// Activations of the gated feed-forward block.
#pragma once

#include <type_traits>

#include "../../include/muon_layers.h"
#include "layers.hpp"

namespace muon {

// e^x and 1/x: correctly rounded library forms for fp32 results, the hardware's
// (relative errors of about 2^-22 over the range that matters, far below
// bf16's 2^-9) for results that are rounded to 16 bits.
template <bool FULL> __device__ __forceinline__ float ffn_exp(float x) {
  return FULL ? expf(x) : __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}
template <bool FULL> __device__ __forceinline__ float ffn_rcp(float x) {
  return FULL ? 1.0f / x : __builtin_amdgcn_rcpf(x);
}

// act(g) and act'(g).
template <int ACT, bool FULL>
__device__ __forceinline__ void ffn_act(float g, float& v, float& d) {
  if constexpr (ACT == MUON_ACT_SILU) {
    const float s = ffn_rcp<FULL>(1.0f + ffn_exp<FULL>(-g));
    v = g * s;
    d = s + v * (1.0f - s);
  } else if constexpr (ACT == MUON_ACT_GELU) {
    const float c = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
    v = g * c;
    d = c + g * 0.39894228040143268f * ffn_exp<FULL>(-0.5f * g * g);
  } else {
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z); s·(1 − s) is 0 long before g²
    // reaches the cap, which keeps 0·∞ out of the derivative
    const float k = 1.59576912160573072f;
    const float s = ffn_rcp<FULL>(1.0f + ffn_exp<FULL>(-k * (g + 0.044715f * g * g * g)));
    v = g * s;
    d = s + v * (1.0f - s) * k * (1.0f + 0.134145f * fminf(g * g, 1e6f));
  }
}

// Runs f with the activation as a compile-time constant.
template <typename F> __device__ __forceinline__ void ffn_with_act(int act, F&& f) {
  if (act == MUON_ACT_SILU) f(std::integral_constant<int, MUON_ACT_SILU>{});
  else if (act == MUON_ACT_GELU) f(std::integral_constant<int, MUON_ACT_GELU>{});
  else f(std::integral_constant<int, MUON_ACT_GELU_TANH>{});
}

}  // namespace muon

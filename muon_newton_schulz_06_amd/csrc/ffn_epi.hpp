// Activations and results of the gated feed-forward block's products.
#pragma once

#include <type_traits>

#include "../../include/muon_layers.h"
#include "layers.hpp"

namespace muon {

// e^x and 1/x: the library's exponential and an IEEE division for fp32 results,
// the hardware's (relative errors of about 2^-22 over the range that matters,
// far below bf16's 2^-9) for results that are rounded to bf16.
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

// ----- results, four columns [j, j + 4) of row i at a time -------------------

// C ← c (+ C); vec: the four elements are one aligned access where they exist.
__device__ __forceinline__ void ffn_store4(void* C, int64_t ldc, int64_t i, int64_t j, int64_t n, bool bf16,
                                           bool accumulate, bool vec, const float (&c)[4]) {
  const int64_t e = i * ldc + j;
  if (bf16) {
    uint16_t* o = (uint16_t*)C + e;
    if (vec && j + 4 <= n) {
      float v[4] = {c[0], c[1], c[2], c[3]};
      if (accumulate) {
        const uint2 u = *(const uint2*)o;
        v[0] += __uint_as_float(u.x << 16);
        v[1] += __uint_as_float(u.x & 0xffff0000u);
        v[2] += __uint_as_float(u.y << 16);
        v[3] += __uint_as_float(u.y & 0xffff0000u);
      }
      *(uint2*)o = make_uint2(l_f32_bf16x2(v[0], v[1]), l_f32_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (j + r < n) o[r] = (uint16_t)l_f32_bf16(c[r] + (accumulate ? l_bf16_f32(o[r]) : 0.f));
    }
  } else {
    float* o = (float*)C + e;
    if (vec && j + 4 <= n) {
      lf32x4 v = {c[0], c[1], c[2], c[3]};
      if (accumulate) v += *(const lf32x4*)o;
      *(lf32x4*)o = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (j + r < n) o[r] = c[r] + (accumulate ? o[r] : 0.f);
    }
  }
}

// One split's sums (half 1: u of FFN_GLU, stored in the second half of a row).
__device__ __forceinline__ void ffn_part4(const FfnProb& P, int split, int64_t i, int64_t j, bool glu, int half,
                                          const float (&c)[4]) {
  const int64_t w = glu ? P.partN / 2 : P.partN;
  if (j < w)  // w is a multiple of 4
    *(lf32x4*)(P.part + ((int64_t)split * P.M + i) * P.partN + half * w + j) = lf32x4{c[0], c[1], c[2], c[3]};
}

// FFN_GLU: h, and with SAVE a = u·act'(g) and b = act(g).  Rows of h and of
// each part of ab have ldh elements, a multiple of 8.
// Of bf16 calls h, and dg and du below, are rounded to bf16: they are operands
// of the next product's MFMA, which takes no wider type at its rate.  That and
// the results' own rounding are 1.65e-3 each (2-norm, against fp64), 2.3e-3
// together; a and b, kept in 24 bits, add nothing to it.
template <typename T, int ACT, bool SAVE>
__device__ __forceinline__ void ffn_glu4(const FfnLaunch& L, const FfnProb& P, int64_t i, int64_t j,
                                         const float (&g)[4], const float (&u)[4]) {
  constexpr bool F32 = LType<T>::kVec == 4;
  float v[4], d[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    ffn_act<ACT, F32>(g[r], v[r], d[r]);
    d[r] *= u[r];
  }
  if constexpr (F32) {
    *(lf32x4*)((float*)P.C + i * P.ldc + j) = lf32x4{v[0] * u[0], v[1] * u[1], v[2] * u[2], v[3] * u[3]};
    if constexpr (SAVE) {
      float* o = (float*)L.ab + i * 2 * L.ldh + j;
      *(lf32x4*)o = lf32x4{d[0], d[1], d[2], d[3]};
      *(lf32x4*)(o + L.ldh) = lf32x4{v[0], v[1], v[2], v[3]};
    }
  } else {
    *(uint2*)((uint16_t*)P.C + i * P.ldc + j) =
        make_uint2(l_f32_bf16x2(v[0] * u[0], v[1] * u[1]), l_f32_bf16x2(v[2] * u[2], v[3] * u[3]));
    if constexpr (SAVE) {
      uint16_t* o = (uint16_t*)L.ab + i * 3 * L.ldh + j;
      *(uint2*)o = make_uint2(l_upper2(d[0], d[1]), l_upper2(d[2], d[3]));
      *(uint2*)(o + L.ldh) = make_uint2(l_upper2(v[0], v[1]), l_upper2(v[2], v[3]));
      *(uint2*)(o + 2 * L.ldh) = make_uint2(l_lower2(d[0], v[0], d[1], v[1]), l_lower2(d[2], v[2], d[3], v[3]));
    }
  }
}

// Runs f(activation, save) with both as compile-time constants.
template <typename F> __device__ __forceinline__ void ffn_with_glu(const FfnLaunch& L, F&& f) {
  ffn_with_act(L.act, [&](auto actc) __attribute__((always_inline)) {
    if (L.ab) f(actc, std::true_type{});
    else f(actc, std::false_type{});
  });
}

// dh times value V (0: a, 1: b) of four columns, as bf16: from the upper halves
// of V and the bytes below of both.
template <int V, typename F> __device__ __forceinline__ uint2 ffn_times24(const F& c, uint2 upper, uint2 lower) {
  return make_uint2(
      l_f32_bf16x2(c[0] * l_join24<V, 0>(upper.x, lower.x), c[1] * l_join24<V, 1>(upper.x, lower.x)),
      l_f32_bf16x2(c[2] * l_join24<V, 0>(upper.y, lower.y), c[3] * l_join24<V, 1>(upper.y, lower.y)));
}

}  // namespace muon

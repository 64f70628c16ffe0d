// Sum of the k splits of a feed-forward product, with the product's epilogue.
//
// The splits' fp32 results lie in the workspace as [split][M][partN]; four
// columns per thread are added up in split order and finished as the
// unsplit product would finish them.  HBM-bound (usually cache-bound: the
// results were just written): 5 µs for one token's five splits of 3584 columns,
// 12 µs for two splits of 2048 × 3584.
#include <hip/hip_runtime.h>

#include "ffn_epi.hpp"

namespace muon {
namespace {

__device__ __forceinline__ void join4(const FfnProb& P, int splits, int64_t i, int64_t c, float (&v)[4]) {
  const float* p = P.part + i * P.partN + c;
  const int64_t step = (int64_t)P.M * P.partN;
  lf32x4 s = *(const lf32x4*)p;
#pragma unroll 4
  for (int k = 1; k < splits; ++k) s += *(const lf32x4*)(p + k * step);
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = s[r];
}

template <typename T, int EPI>
__global__ __launch_bounds__(256) void ffn_join(const FfnLaunch L, int splits) {
  const FfnProb& P = L.prob[blockIdx.y];
  const int64_t width = EPI == FFN_STORE ? P.partN : L.ldh, quads = width / 4;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= P.M * quads) return;
  const int64_t i = e / quads, j = (e - i * quads) * 4;
  float c[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
  if (j < P.N) {
    join4(P, splits, i, j, c);
    if constexpr (EPI == FFN_GLU) join4(P, splits, i, P.partN / 2 + j, u);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (j + r >= P.N) c[r] = u[r] = 0.f;  // results past column N are zeros
  if constexpr (EPI == FFN_GLU) {
    ffn_with_glu(L, [&](auto actc, auto savec) __attribute__((always_inline)) {
      ffn_glu4<T, decltype(actc)::value, decltype(savec)::value>(L, P, i, j, c, u);
    });
  } else if constexpr (EPI == FFN_BACK) {
    if constexpr (LType<T>::kVec == 8) {
      const uint16_t* ab = (const uint16_t*)L.ab + i * 3 * L.ldh + j;
      const uint2 lower = *(const uint2*)(ab + 2 * L.ldh);
      uint16_t* o = (uint16_t*)P.C + i * 2 * L.ldh + j;
      *(uint2*)o = ffn_times24<0>(c, *(const uint2*)ab, lower);
      *(uint2*)(o + L.ldh) = ffn_times24<1>(c, *(const uint2*)(ab + L.ldh), lower);
    } else {
      const float* ab = (const float*)L.ab + i * 2 * L.ldh + j;
      const lf32x4 va = *(const lf32x4*)ab, vb = *(const lf32x4*)(ab + L.ldh);
      float* o = (float*)P.C + i * 2 * L.ldh + j;
      *(lf32x4*)o = lf32x4{c[0] * va[0], c[1] * va[1], c[2] * va[2], c[3] * va[3]};
      *(lf32x4*)(o + L.ldh) = lf32x4{c[0] * vb[0], c[1] * vb[1], c[2] * vb[2], c[3] * vb[3]};
    }
  } else {
    ffn_store4(P.C, P.ldc, i, j, P.N, L.outBf16, L.accumulate, P.vecC, c);
  }
}

template <typename T> void join_launch(int epi, int splits, const FfnLaunch& L, hipStream_t st) {
  int64_t n = 0;
  for (int q = 0; q < L.nprob; ++q) {
    const int64_t m = L.prob[q].M * ((epi == FFN_STORE ? L.prob[q].partN : L.ldh) / 4);
    n = n > m ? n : m;
  }
  const dim3 grid((n + 255) / 256, L.nprob), block(256);
  if (epi == FFN_GLU) hipLaunchKernelGGL((ffn_join<T, FFN_GLU>), grid, block, 0, st, L, splits);
  else if (epi == FFN_BACK) hipLaunchKernelGGL((ffn_join<T, FFN_BACK>), grid, block, 0, st, L, splits);
  else hipLaunchKernelGGL((ffn_join<T, FFN_STORE>), grid, block, 0, st, L, splits);
}

}  // namespace

hipError_t launch_ffn_join(int epi, bool bf16, int splits, const FfnLaunch& L, hipStream_t st) {
  if (bf16) join_launch<Bf16>(epi, splits, L, st);
  else join_launch<float>(epi, splits, L, st);
  return hipGetLastError();
}

}  // namespace muon

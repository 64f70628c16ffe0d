// Products of the gated feed-forward block on fp32 MFMA.
//
// C[i][j] = Σ_k A[i][k]·B[j][k], 128×128 tiles, four waves of 64×64 (2×2
// accumulators of 32×32), k in steps of 16.  The operands are staged through
// registers into k-major LDS panels (rows of 132 floats: the transposing
// writes of a k-contiguous operand, 4 k apart and 16 rows wide, then fall in
// distinct banks), double buffered, one barrier per step.  A 32×32×2 MFMA
// takes 64 cycles for two 4-byte LDS reads shared by two MFMAs each, so the
// loop is bound by the matrix pipe.
#include <hip/hip_runtime.h>

#include "ffn_epi.hpp"

namespace muon {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kT = 128, kKs = 16, kLd = kT + 4;

// Four operand values as fp32: (row, k..k+3) of a k-contiguous operand or
// (row..row+3, k) of a row-contiguous one; zeros outside rows × K.
template <bool ROWC>
__device__ __forceinline__ lf32x4 fetch4(const void* p, int64_t ld, int row, int64_t k, int rows,
                                         int64_t K, bool vec) {
  lf32x4 v = {0.f, 0.f, 0.f, 0.f};
  const int64_t e = ROWC ? k * ld + row : (int64_t)row * ld + k;
  const bool in = row < rows && k < K;
  const int have = !in ? 0 : ROWC ? rows - row : (int)min((int64_t)4, K - k);
  if (have >= 4 && vec) {
    v = *(const lf32x4*)((const float*)p + e);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) v[i] = ((const float*)p)[e + i];
  }
  return v;
}

// Whether 4-element accesses of an operand are aligned.
__device__ __forceinline__ bool aligned4(const void* p, int64_t ld) {
  return ((uintptr_t)p & 15) == 0 && (ld & 3) == 0;
}

template <int EPI, bool AROW, bool BROW>
__global__ __launch_bounds__(256) void ffn_tile32(const FfnLaunch L) {
  __shared__ __attribute__((aligned(16))) float sa[2][kKs * kLd];
  __shared__ __attribute__((aligned(16))) float sb[2][kKs * kLd];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  int q = 0;
  while (q + 1 < L.nprob && (int)blockIdx.x >= L.tiles[q + 1]) ++q;
  const FfnProb& P = L.prob[q];
  // FFN_GLU: a tile is 64 columns of both projections, B rows 32·c .. of
  // w_gate (even 32-row blocks c) and of w_up (odd ones)
  constexpr int TN = EPI == FFN_GLU ? kT / 2 : kT;
  const int tilesM = (P.M + kT - 1) / kT;
  const int t = blockIdx.x - L.tiles[q];
  const int ti = t % tilesM, tj = t / tilesM;
  const int i0 = ti * kT, j0 = tj * TN;

  f32x16 acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  // each thread stages two groups of four values of each operand per step
  auto at_row = [&](bool rowc, int h) { return rowc ? (tid & 31) * 4 : (tid >> 2) + 64 * h; };
  auto at_k = [&](bool rowc, int h) { return rowc ? (tid >> 5) + 8 * h : (tid & 3) * 4; };
  const int steps0 = (P.K[0] + kKs - 1) / kKs, steps1 = (P.K[1] + kKs - 1) / kKs;
  const int steps = steps0 + steps1;
  lf32x4 ra[2], rb[2];
  auto fetch = [&](int s) {
    const int z = s >= steps0;
    const int64_t k0 = (int64_t)(z ? s - steps0 : s) * kKs;
    const int64_t K = P.K[z];
    const bool va = aligned4(P.A[z], P.lda);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ra[h] = fetch4<AROW>(P.A[z], P.lda, i0 + at_row(AROW, h), k0 + at_k(AROW, h), P.M, K, va);
      const int r = at_row(BROW, h);
      if constexpr (EPI == FFN_GLU) {
        const int which = (r >> 5) & 1;
        const int j = j0 + (r >> 6) * 32 + (r & 31);
        rb[h] = fetch4<false>(P.B[which], P.ldb[which], j, k0 + at_k(false, h), P.N, K,
                                 aligned4(P.B[which], P.ldb[which]));
      } else {
        rb[h] = fetch4<BROW>(P.B[z], P.ldb[z], j0 + r, k0 + at_k(BROW, h), P.N, K,
                                aligned4(P.B[z], P.ldb[z]));
      }
    }
  };
  auto put = [&](float* s, bool rowc, int h, const lf32x4& v) {
    const int r = at_row(rowc, h), k = at_k(rowc, h);
    if (rowc) {
      *(lf32x4*)(s + k * kLd + r) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[(k + i) * kLd + r] = v[i];
    }
  };
  if (steps > 0) fetch(0);
  const int lr = lane & 31, lk = lane >> 5;
  for (int s = 0; s < steps; ++s) {
    float* pa = sa[s & 1];
    float* pb = sb[s & 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      put(pa, AROW, h, ra[h]);
      put(pb, BROW, h, rb[h]);
    }
    __syncthreads();
    if (s + 1 < steps) fetch(s + 1);
#pragma unroll
    for (int k = 0; k < kKs; k += 2) {
      float fa[2], fb[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        fa[a] = pa[(k + lk) * kLd + wm * 64 + a * 32 + lr];
        fb[a] = pb[(k + lk) * kLd + wn * 64 + a * 32 + lr];
      }
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[a], fb[b], acc[a][b], 0, 0, 0);
    }
  }

  // acc[a][b][r]: row 8·(r/4) + 4·(lane/32) + r%4, column lane%32
  auto row = [&](int a, int r) { return i0 + wm * 64 + a * 32 + 8 * (r >> 2) + 4 * lk + (r & 3); };
  if constexpr (EPI == FFN_GLU) {
    const int64_t j = j0 + wn * 32 + lr;
    if (j >= L.ldh) return;  // columns N .. ldh − 1 are written as zeros
    ffn_with_act(L.act, [&](auto actc) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t i = row(a, r);
          if (i >= P.M) continue;
          float v, d;
          const float u = acc[a][1][r];
          ffn_act<decltype(actc)::value, true>(acc[a][0][r], v, d);
          ((float*)P.C)[i * P.ldc + j] = v * u;
          if (L.ab) {
            float* ab = (float*)L.ab + i * 2 * L.ldh + j;
            ab[0] = u * d;
            ab[L.ldh] = v;
          }
        }
    });
    return;
  }
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t i = row(a, r);
      if (i >= P.M) continue;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int64_t j = j0 + wn * 64 + b * 32 + lr;
        const float c = acc[a][b][r];
        if constexpr (EPI == FFN_BACK) {
          if (j >= L.ldh) continue;
          const int64_t e = i * 2 * L.ldh + j;
          const float* ab = (const float*)L.ab + e;
          float* o = (float*)P.C + e;
          o[0] = c * ab[0];
          o[L.ldh] = c * ab[L.ldh];
        } else {
          if (j >= P.N) continue;
          const int64_t e = i * P.ldc + j;
          if (L.outBf16) {
            const float old = L.accumulate ? LType<Bf16>::get(P.C, e) : 0.f;
            LType<Bf16>::put(P.C, e, c + old);
          } else {
            const float old = L.accumulate ? LType<float>::get(P.C, e) : 0.f;
            LType<float>::put(P.C, e, c + old);
          }
        }
      }
    }
}

}  // namespace

hipError_t launch_ffn_tile32(int epi, bool aRowContig, bool bRowContig, const FfnLaunch& L,
                             hipStream_t st) {
  const dim3 grid(L.tiles[L.nprob]), block(256);
  if (epi == FFN_GLU) hipLaunchKernelGGL((ffn_tile32<FFN_GLU, false, false>), grid, block, 0, st, L);
  else if (epi == FFN_BACK) hipLaunchKernelGGL((ffn_tile32<FFN_BACK, false, true>), grid, block, 0, st, L);
  else if (aRowContig) hipLaunchKernelGGL((ffn_tile32<FFN_STORE, true, true>), grid, block, 0, st, L);
  else if (bRowContig) hipLaunchKernelGGL((ffn_tile32<FFN_STORE, false, true>), grid, block, 0, st, L);
  else hipLaunchKernelGGL((ffn_tile32<FFN_STORE, false, false>), grid, block, 0, st, L);
  return hipGetLastError();
}

}  // namespace muon

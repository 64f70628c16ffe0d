// Products of the gated feed-forward block on fp32 MFMA.
//
// C[i][j] = Σ_k A[i][k]·B[j][k], tiles of TM×128 (TM 128 or 64), four waves of
// TM/2 × 64 (32×32×2 MFMAs), k in steps of 32.  The operands are staged
// through registers into k-major LDS panels (rows of TM + 4 or 132 floats: the
// transposing writes of a k-contiguous operand then spread over the banks),
// double buffered, one barrier per step, the next step's global loads issued
// before the MFMAs.  A 32×32×2 MFMA takes 64 cycles and its two 4-byte LDS
// reads are shared by two MFMAs each, so a full GPU is bound by the matrix
// pipe; small products are bound by the latency of a step (load, barrier),
// which is what the 64-row tile and the k splits are for.
#include <hip/hip_runtime.h>

#include <cstring>

#include "ffn_epi.hpp"

namespace muon {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTN = 128, kKs = 32;

// Four operand values: (row, k..k+3) of a k-contiguous operand or
// (row..row+3, k) of a row-contiguous one; zeros outside rows × K.  Whole
// groups are one 16-byte load at any 4-byte alignment.
template <bool ROWC>
__device__ __forceinline__ lf32x4 fetch4(const float* p, int64_t ld, int64_t row, int64_t k, int64_t rows,
                                         int64_t K) {
  lf32x4 v = {0.f, 0.f, 0.f, 0.f};
  const int64_t e = ROWC ? k * ld + row : row * ld + k;
  const int64_t have = row >= rows || k >= K ? 0 : ROWC ? rows - row : K - k;
  if (have >= 4) {
    __builtin_memcpy(&v, p + e, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < have) v[i] = p[e + i];
  }
  return v;
}

template <int TM, int EPI, bool AROW, bool BROW>
__global__ __launch_bounds__(256) void ffn_tile32(const FfnLaunch L) {
  constexpr int FA = TM / 64;                         // 32-row blocks of a wave
  constexpr int NA = TM * kKs / 1024, NB = kTN * kKs / 1024;  // groups of four per thread and step
  constexpr int LA = TM + 4, LB = kTN + 4;
  __shared__ __attribute__((aligned(16))) float sa[2][kKs * LA];
  __shared__ __attribute__((aligned(16))) float sb[2][kKs * LB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  int q = 0;
  while (q + 1 < L.nprob && (int)blockIdx.x >= L.tiles[q + 1]) ++q;
  const FfnProb& P = L.prob[q];
  // FFN_GLU: a tile is 64 columns of both projections, B rows 32·c .. of
  // w_gate (even 32-row blocks c) and of w_up (odd ones)
  constexpr int TN = EPI == FFN_GLU ? kTN / 2 : kTN;
  const int tilesM = (P.M + TM - 1) / TM, tilesN = (P.N + TN - 1) / TN;
  int t = blockIdx.x - L.tiles[q];
  const int split = t / (tilesM * tilesN);
  t -= split * (tilesM * tilesN);
  const int ti = t % tilesM, tj = t / tilesM;
  const int64_t i0 = (int64_t)ti * TM, j0 = (int64_t)tj * TN;

  f32x16 acc[FA][2];
#pragma unroll
  for (int a = 0; a < FA; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  // group h of a thread: eight lanes cover 32 k of a row, or T/4 lanes a k-row
  auto at_row = [&](bool rowc, int T, int h) { return rowc ? (tid % (T / 4)) * 4 : (tid >> 3) + 32 * h; };
  auto at_k = [&](bool rowc, int T, int h) { return rowc ? tid / (T / 4) + (1024 / T) * h : (tid & 7) * 4; };
  const int steps0 = (P.K[0] + kKs - 1) / kKs;
  const int all = steps0 + (P.K[1] + kKs - 1) / kKs;
  const int s0 = split * L.splitTiles, s1 = min(all, s0 + L.splitTiles);
  lf32x4 ra[NA], rb[NB];
  auto fetch = [&](int s) {
    const int z = s >= steps0;
    const int64_t k0 = (int64_t)(z ? s - steps0 : s) * kKs;
    const int64_t K = P.K[z];
#pragma unroll
    for (int h = 0; h < NA; ++h)
      ra[h] = fetch4<AROW>((const float*)P.A[z], P.lda, i0 + at_row(AROW, TM, h), k0 + at_k(AROW, TM, h), P.M, K);
#pragma unroll
    for (int h = 0; h < NB; ++h) {
      const int r = at_row(BROW, kTN, h);
      if constexpr (EPI == FFN_GLU) {
        const int which = (r >> 5) & 1;  // the same for the whole group h
        rb[h] = fetch4<false>((const float*)P.B[which], P.ldb[which], j0 + (r >> 6) * 32 + (r & 31),
                              k0 + at_k(false, kTN, h), P.N, K);
      } else {
        rb[h] = fetch4<BROW>((const float*)P.B[z], P.ldb[z], j0 + r, k0 + at_k(BROW, kTN, h), P.N, K);
      }
    }
  };
  auto put = [&](float* s, bool rowc, int T, int ld, int h, const lf32x4& v) {
    const int r = at_row(rowc, T, h), k = at_k(rowc, T, h);
    if (rowc) {
      *(lf32x4*)(s + k * ld + r) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[(k + i) * ld + r] = v[i];
    }
  };
  const int lr = lane & 31, lk = lane >> 5;
  if (s0 < s1) fetch(s0);
  for (int s = s0; s < s1; ++s) {
    float* pa = sa[s & 1];
    float* pb = sb[s & 1];
#pragma unroll
    for (int h = 0; h < NA; ++h) put(pa, AROW, TM, LA, h, ra[h]);
#pragma unroll
    for (int h = 0; h < NB; ++h) put(pb, BROW, kTN, LB, h, rb[h]);
    __syncthreads();
    if (s + 1 < s1) fetch(s + 1);
#pragma unroll
    for (int k = 0; k < kKs; k += 2) {
      float fa[FA], fb[2];
#pragma unroll
      for (int a = 0; a < FA; ++a) fa[a] = pa[(k + lk) * LA + wm * (TM / 2) + a * 32 + lr];
#pragma unroll
      for (int b = 0; b < 2; ++b) fb[b] = pb[(k + lk) * LB + wn * 64 + b * 32 + lr];
#pragma unroll
      for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[a], fb[b], acc[a][b], 0, 0, 0);
    }
  }

  // acc[a][b][r]: row 8·(r/4) + 4·(lane/32) + r%4, column lane%32
  auto row = [&](int a, int r) { return i0 + wm * (TM / 2) + a * 32 + 8 * (r >> 2) + 4 * lk + (r & 3); };
  if constexpr (EPI == FFN_GLU) {
    const int64_t j = j0 + wn * 32 + lr;
    if (j >= L.ldh) return;  // columns N .. ldh − 1 are written as zeros
    ffn_with_act(L.act, [&](auto actc) {
#pragma unroll
      for (int a = 0; a < FA; ++a)
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
  for (int a = 0; a < FA; ++a)
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
          if (L.part) {
            L.part[((int64_t)split * P.M + i) * L.partN + j] = c;
          } else if (L.outBf16) {
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

template <int TM>
void launch_tm(int epi, bool ar, bool br, const FfnLaunch& L, hipStream_t st) {
  const dim3 grid(L.tiles[L.nprob]), block(256);
  if (epi == FFN_GLU) hipLaunchKernelGGL((ffn_tile32<TM, FFN_GLU, false, false>), grid, block, 0, st, L);
  else if (epi == FFN_BACK) hipLaunchKernelGGL((ffn_tile32<TM, FFN_BACK, false, true>), grid, block, 0, st, L);
  else if (ar) hipLaunchKernelGGL((ffn_tile32<TM, FFN_STORE, true, true>), grid, block, 0, st, L);
  else if (br) hipLaunchKernelGGL((ffn_tile32<TM, FFN_STORE, false, true>), grid, block, 0, st, L);
  else hipLaunchKernelGGL((ffn_tile32<TM, FFN_STORE, false, false>), grid, block, 0, st, L);
}

}  // namespace

hipError_t launch_ffn_tile32(int epi, int tileM, bool aRowContig, bool bRowContig, const FfnLaunch& L,
                             hipStream_t st) {
  if (tileM == 128) launch_tm<128>(epi, aRowContig, bRowContig, L, st);
  else launch_tm<64>(epi, aRowContig, bRowContig, L, st);
  return hipGetLastError();
}

}  // namespace muon

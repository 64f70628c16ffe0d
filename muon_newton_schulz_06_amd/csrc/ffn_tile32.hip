// Products of the gated feed-forward block on fp32 MFMA.
//
// C[i][j] = Σ_k A[i][k]·B[j][k], tiles of TM×128 (TM 128 or 64), four waves of
// TM/2 × 64 (32×32×2 MFMAs), k in steps of 32.  The operands are staged
// through registers into k-major LDS panels (rows of TM + 4 or 132 floats: the
// transposing writes of a k-contiguous operand then spread over the banks),
// double buffered, one barrier per step, the global loads two steps ahead.  A
// 32×32×2 MFMA takes 64 cycles and its two 4-byte LDS reads are shared by two
// MFMAs each, so a full GPU is bound by the matrix pipe; small products are
// bound by the latency of a step (load, barrier), which is what the 64-row
// tile and the k splits are for.  1024 tokens, 2048×8192: 107 TFLOP/s (dh 320
// µs), MFMA busy 71%; 501 tokens, 509×1021: 20–41 µs per product.
#include <hip/hip_runtime.h>

#include <cstring>

#include "ffn_epi.hpp"

namespace muon {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTN = 128, kKs = 32;

template <int B, int E, typename F> __device__ __forceinline__ void static_for32(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for32<B + 1, E>(f);
  }
}

// Four operand values: (row, k..k+3) of a k-contiguous operand or
// (row..row+3, k) of a row-contiguous one, one 16-byte load at any 4-byte
// alignment.  Rows past the last one hold anything that lies in the operand
// (their results are not stored).  EDGE: the group may reach over the end of
// the rows or of k; it is loaded from the last place where it fits, without a
// branch, and put right by fix4 when it is used, a step or two later (operands
// with fewer than four values along the group are read one by one).
template <bool ROWC, bool EDGE>
__device__ __forceinline__ lf32x4 fetch4(const float* p, int64_t ld, int row, int k, int rows, int K) {
  lf32x4 v = {0.f, 0.f, 0.f, 0.f};
  if constexpr (!EDGE) {
    const int r = ROWC ? row : min(row, rows - 1);
    __builtin_memcpy(&v, p + (ROWC ? k * ld + r : r * ld + k), 16);
  } else if ((ROWC ? rows : K) < 4) {
    const int have = ROWC ? (k < K ? rows - row : 0) : K - k;
    const int r = ROWC ? row : min(row, rows - 1);
    const float* e = p + (ROWC ? k * ld + r : r * ld + k);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < have) v[i] = e[i];
  } else if constexpr (ROWC) {
    __builtin_memcpy(&v, p + min(k, K - 1) * ld + min(row, rows - 4), 16);
  } else {
    __builtin_memcpy(&v, p + min(row, rows - 1) * ld + min(k, K - 4), 16);
  }
  return v;
}

// An EDGE group's values moved to their places, zeros past the last k.
template <bool ROWC>
__device__ __forceinline__ void fix4(lf32x4& v, int row, int k, int rows, int K) {
  if ((ROWC ? rows : K) < 4) return;  // read one by one
  const int d = ROWC ? row - min(row, rows - 4) : k - min(k, K - 4);
  if (d & 1) {
    v[0] = v[1];
    v[1] = v[2];
    v[2] = v[3];
  }
  if (d & 2) {
    v[0] = v[2];
    v[1] = v[3];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (ROWC ? k : k + i) < K ? v[i] : 0.f;
}

template <int TM, int EPI, bool AROW, bool BROW>
__global__ __launch_bounds__(256, 2) void ffn_tile32(const FfnLaunch L) {
  constexpr int FA = TM / 64;                         // 32-row blocks of a wave
  constexpr int NA = TM * kKs / 1024, NB = kTN * kKs / 1024;  // groups of four per thread and step
  constexpr int LA = TM + 4, LB = kTN + 4;
  __shared__ __attribute__((aligned(16))) float sa[2][kKs * LA];
  __shared__ __attribute__((aligned(16))) float sb[2][kKs * LB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  // Workgroups are dealt round over the eight XCDs; each XCD takes a run of
  // consecutive tiles, so that the row tiles of a column, which read the same B,
  // share an L2 (406 tokens, 580×9088: gated projections 142 -> 130 µs; no
  // difference at 1024 tokens, 2048×8192).
  const int run = gridDim.x >> 3, more = gridDim.x & 7, xcd = blockIdx.x & 7;
  const int wg = xcd * run + min(xcd, more) + (blockIdx.x >> 3);
  int q = 0;
  while (q + 1 < L.nprob && wg >= L.tiles[q + 1]) ++q;
  const FfnProb& P = L.prob[q];
  // FFN_GLU: a tile is 64 columns of both projections, B rows 32·c .. of
  // w_gate (even 32-row blocks c) and of w_up (odd ones)
  constexpr int TN = EPI == FFN_GLU ? kTN / 2 : kTN;
  const int tilesM = (P.M + TM - 1) / TM, tilesN = (P.N + TN - 1) / TN;
  int t = wg - L.tiles[q];
  const int split = t / (tilesM * tilesN);
  t -= split * (tilesM * tilesN);
  const int ti = t % tilesM, tj = t / tilesM;
  const int i0 = ti * TM, j0 = tj * TN;

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
  // copies of the arguments, so that no step reads them again
  const float* const a0 = (const float*)P.A[0];
  const float* const a1 = (const float*)P.A[1];
  const float* const b0 = (const float*)P.B[0];
  const float* const b1 = (const float*)P.B[1];
  const int64_t lda = P.lda, ldb0 = P.ldb[0], ldb1 = P.ldb[1];
  const int M = P.M, N = P.N, K0 = P.K[0], K1 = P.K[1];
  const int steps0 = (K0 + kKs - 1) / kKs;
  const int all = steps0 + (K1 + kKs - 1) / kKs;
  const int s0 = split * L.splitTiles, s1 = min(all, s0 + L.splitTiles);
  lf32x4 ra[2][NA], rb[2][NB];  // of the next two steps
  auto fetch_as = [&](int s, lf32x4 (&fa)[NA], lf32x4 (&fb)[NB], auto edgec) __attribute__((always_inline)) {
    constexpr bool EDGE = decltype(edgec)::value;
    const bool z = s >= steps0;
    const int k0 = (z ? s - steps0 : s) * kKs, K = z ? K1 : K0;
    const float* const a = z ? a1 : a0;
#pragma unroll
    for (int h = 0; h < NA; ++h)
      fa[h] = fetch4<AROW, EDGE>(a, lda, i0 + at_row(AROW, TM, h), k0 + at_k(AROW, TM, h), M, K);
#pragma unroll
    for (int h = 0; h < NB; ++h) {
      const int r = at_row(BROW, kTN, h);
      if constexpr (EPI == FFN_GLU)  // rows 32·h .. of the tile are one matrix's
        fb[h] = fetch4<false, EDGE>(h & 1 ? b1 : b0, h & 1 ? ldb1 : ldb0, j0 + (h >> 1) * 32 + (r & 31),
                                    k0 + at_k(false, kTN, h), N, K);
      else
        fb[h] = fetch4<BROW, EDGE>(z ? b1 : b0, z ? ldb1 : ldb0, j0 + r, k0 + at_k(BROW, kTN, h), N, K);
    }
  };
  const bool inside = (!AROW || i0 + TM <= M) && (!BROW || j0 + TN <= N);
  auto whole = [&](int s) {
    const bool z = s >= steps0;
    return inside && ((z ? s - steps0 : s) + 1) * kKs <= (z ? K1 : K0);
  };
  auto fetch = [&](int s, lf32x4 (&fa)[NA], lf32x4 (&fb)[NB]) __attribute__((always_inline)) {
    if (whole(s)) fetch_as(s, fa, fb, std::false_type{});
    else fetch_as(s, fa, fb, std::true_type{});
  };
  auto fix = [&](int s, lf32x4 (&fa)[NA], lf32x4 (&fb)[NB]) __attribute__((always_inline)) {
    const bool z = s >= steps0;
    const int k0 = (z ? s - steps0 : s) * kKs, K = z ? K1 : K0;
#pragma unroll
    for (int h = 0; h < NA; ++h) fix4<AROW>(fa[h], i0 + at_row(AROW, TM, h), k0 + at_k(AROW, TM, h), M, K);
#pragma unroll
    for (int h = 0; h < NB; ++h) fix4<BROW>(fb[h], j0 + at_row(BROW, kTN, h), k0 + at_k(BROW, kTN, h), N, K);
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
  auto step = [&](int s, auto parity) __attribute__((always_inline)) {
    constexpr int h2 = decltype(parity)::value;
    float* pa = sa[h2];
    float* pb = sb[h2];
    if (!whole(s)) fix(s, ra[h2], rb[h2]);
#pragma unroll
    for (int h = 0; h < NA; ++h) put(pa, AROW, TM, LA, h, ra[h2][h]);
#pragma unroll
    for (int h = 0; h < NB; ++h) put(pb, BROW, kTN, LB, h, rb[h2][h]);
    __syncthreads();
    if (s + 2 < s1) fetch(s + 2, ra[h2], rb[h2]);
    // four pairs of k at a time, the next four's operands read before their
    // MFMAs are issued
    constexpr int G = 4;
    float fa[2][G][FA], fb[2][G][2];
    auto read = [&](int g, float (&xa)[G][FA], float (&xb)[G][2]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int k = (g * G + i) * 2 + lk;
#pragma unroll
        for (int a = 0; a < FA; ++a) xa[i][a] = pa[k * LA + wm * (TM / 2) + a * 32 + lr];
#pragma unroll
        for (int b = 0; b < 2; ++b) xb[i][b] = pb[k * LB + wn * 64 + b * 32 + lr];
      }
    };
    read(0, fa[0], fb[0]);
    const int left = s >= steps0 ? K1 - (s - steps0) * kKs : K0 - s * kKs;
    static_for32<0, kKs / (2 * G)>([&](auto gc) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value;
      // the rest of a last step is zeros (38 tokens, 2944×6681: the weights'
      // gradients 178 -> 158 µs)
      if (g * 2 * G >= left) return;
      if constexpr ((g + 1) * 2 * G < kKs) read(g + 1, fa[(g + 1) & 1], fb[(g + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int a = 0; a < FA; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[g & 1][i][a], fb[g & 1][i][b], acc[a][b], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  if (s0 < s1) fetch(s0, ra[0], rb[0]);
  if (s0 + 1 < s1) fetch(s0 + 1, ra[1], rb[1]);
  for (int s = s0; s < s1; s += 2) {
    step(s, std::integral_constant<int, 0>{});
    if (s + 1 < s1) step(s + 1, std::integral_constant<int, 1>{});
  }

  // acc[a][b][r]: row 8·(r/4) + 4·(lane/32) + r%4, column lane%32
  auto row = [&](int a, int r) { return (int64_t)i0 + wm * (TM / 2) + a * 32 + 8 * (r >> 2) + 4 * lk + (r & 3); };
  if constexpr (EPI == FFN_GLU) {
    const int64_t j = j0 + wn * 32 + lr;
    if (j >= (P.part ? (int64_t)P.N : L.ldh)) return;  // columns N .. ldh − 1 of the results are zeros
    auto each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (row(a, r) < P.M) f(row(a, r), acc[a][0][r], acc[a][1][r]);
    };
    if (P.part) {
      each([&](int64_t i, float g, float u) __attribute__((always_inline)) {
        float* o = P.part + ((int64_t)split * P.M + i) * P.partN + j;
        o[0] = g;
        o[P.partN / 2] = u;
      });
      return;
    }
    const bool real = j < P.N;  // the rows past w_gate's and w_up's last one repeat it
    ffn_with_glu(L, [&](auto actc, auto savec) __attribute__((always_inline)) {
      each([&](int64_t i, float g, float u) __attribute__((always_inline)) {
        float v, d;
        ffn_act<decltype(actc)::value, true>(real ? g : 0.f, v, d);
        u = real ? u : 0.f;
        ((float*)P.C)[i * P.ldc + j] = v * u;
        if constexpr (decltype(savec)::value) {
          float* ab = (float*)L.ab + i * 2 * L.ldh + j;
          ab[0] = u * d;
          ab[L.ldh] = v;
        }
      });
    });
    return;
  }
  // one 32×32 block at a time: what it reads first (one wait), then its stores
  auto block = [&](const f32x16& c, int a, int b, auto read, auto write) __attribute__((always_inline)) {
    const int64_t j = j0 + wn * 64 + b * 32 + lr;
    if (j >= (EPI == FFN_BACK && !P.part ? L.ldh : (int64_t)P.N)) return;
    float u[16], v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      u[r] = v[r] = 0.f;
      if (row(a, r) < P.M) read(row(a, r), j, u[r], v[r]);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (row(a, r) < P.M) write(row(a, r), j, c[r], u[r], v[r]);
  };
  auto blocks = [&](auto read, auto write) __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < FA; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) block(acc[a][b], a, b, read, write);
  };
  auto nothing = [](int64_t, int64_t, float&, float&) {};
  if (P.part) {
    blocks(nothing, [&](int64_t i, int64_t j, float c, float, float) {
      P.part[((int64_t)split * P.M + i) * P.partN + j] = c;
    });
  } else if constexpr (EPI == FFN_BACK) {
    blocks(
        [&](int64_t i, int64_t j, float& u, float& v) {
          const float* ab = (const float*)L.ab + i * 2 * L.ldh + j;
          u = ab[0];
          v = ab[L.ldh];
        },
        [&](int64_t i, int64_t j, float c, float u, float v) {
          float* o = (float*)P.C + i * 2 * L.ldh + j;
          o[0] = j < P.N ? c * u : 0.f;
          o[L.ldh] = j < P.N ? c * v : 0.f;
        });
  } else if (L.outBf16) {
    blocks(
        [&](int64_t i, int64_t j, float& u, float&) {
          if (L.accumulate) u = LType<Bf16>::get(P.C, i * P.ldc + j);
        },
        [&](int64_t i, int64_t j, float c, float u, float) { LType<Bf16>::put(P.C, i * P.ldc + j, c + u); });
  } else {
    blocks(
        [&](int64_t i, int64_t j, float& u, float&) {
          if (L.accumulate) u = ((const float*)P.C)[i * P.ldc + j];
        },
        [&](int64_t i, int64_t j, float c, float u, float) { ((float*)P.C)[i * P.ldc + j] = c + u; });
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

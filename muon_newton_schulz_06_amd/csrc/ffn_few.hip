// Forward products of the gated feed-forward block for few tokens (at most
// 64): every weight is read once, so the reads of the weights bound them.
//
// No operand passes through LDS: a lane reads 16 bytes of a weight row
// straight into the MFMA operand layout (16 rows × four lanes per row), and
// the tokens' values likewise (they stay in the caches).  A workgroup takes 16
// weight rows (of both projections for FFN_GLU); its four waves share the k
// range, interleaved by the 16-byte loads of a whole unrolled step, and are
// added up through LDS in wave order.  Long contractions are also split over
// workgroups, whose results go to the workspace.
// A wave keeps few_deep loads per weight matrix in flight: with about 1200
// workgroups of four waves that is over 20 MB, more than HBM's latency needs.
// One token, 3584×18944 bf16: gated projections 51 µs (5.3 TB/s), down
// projection 29 µs (4.7 TB/s).
#include <hip/hip_runtime.h>

#include "ffn_epi.hpp"

namespace muon {
namespace {

typedef float ff32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 fbf8 __attribute__((ext_vector_type(8)));

template <typename T>
__device__ __forceinline__ ff32x4 few_mfma(lu32x4 w, lu32x4 x, ff32x4 acc) {
  if constexpr (LType<T>::kVec == 8) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(fbf8, w), __builtin_bit_cast(fbf8, x),
                                                   acc, 0, 0, 0);
  } else {
    // k = 4·(lane/16) + i in the i-th product, for both operands
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[i]), __uint_as_float(x[i]), acc, 0, 0, 0);
    return acc;
  }
}

// 16-byte loads per weight matrix and step of a wave: at one token the gated
// projections of 3584×18944 take 52.8, 53.3, 50.1 µs with 2, 4, 8 (5.4 TB/s with
// 8); with more tokens their values take the registers.  Non-temporal loads:
// 55.8 µs.
constexpr int few_deep(int TB) { return TB == 1 ? 8 : 4; }

// TB blocks of 16 tokens.
template <typename T, int TB, int EPI>
__global__ __launch_bounds__(256) void ffn_few(const FfnLaunch L) {
  constexpr int V = LType<T>::kVec, E = 16 / V, KC = 4 * V;  // k of one load per row
  constexpr int kDeep = few_deep(TB);
  constexpr int NM = EPI == FFN_GLU ? 2 : 1;                 // weight matrices
  __shared__ float sums[4][NM * TB][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const FfnProb& P = L.prob[0];
  const int split = blockIdx.y;
  const int64_t j0 = (int64_t)blockIdx.x * 16;
  const int K = P.K[0];
  const int kEnd = min(K, (split + 1) * L.splitTiles * 32);
  const char* w[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m)  // rows past the last one repeat it
    w[m] = (const char*)P.B[m] + min(j0 + lr, (int64_t)P.N - 1) * P.ldb[m] * E;
  const char* x[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) x[b] = (const char*)P.A[0] + min(b * 16 + lr, P.M - 1) * P.lda * E;

  ff32x4 acc[NM][TB];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int b = 0; b < TB; ++b) acc[m][b] = ff32x4{0.f, 0.f, 0.f, 0.f};

  int k = split * L.splitTiles * 32 + wave * (kDeep * KC) + lg * V;
  // whole steps: kDeep chunks of every row, then the other waves' share
  for (; k - lg * V + kDeep * KC <= kEnd; k += 4 * kDeep * KC) {
    lu32x4 cw[NM][kDeep], cx[TB][kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
#pragma unroll
      for (int m = 0; m < NM; ++m) __builtin_memcpy(&cw[m][d], w[m] + (int64_t)(k + d * KC) * E, 16);
#pragma unroll
      for (int b = 0; b < TB; ++b) __builtin_memcpy(&cx[b][d], x[b] + (int64_t)(k + d * KC) * E, 16);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads before the first product
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[m][b] = few_mfma<T>(cw[m][d], cx[b][d], acc[m][b]);
  }
  // the last, partial step of the range: its whole chunks at once, then the
  // chunk that reaches over the end
  const int left = kEnd - (k - lg * V);
  if (left > 0) {
    const int nfull = left / KC;
    lu32x4 cw[NM][kDeep], cx[TB][kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        cw[m][d] = lu32x4{0u, 0u, 0u, 0u};
        if (d < nfull) __builtin_memcpy(&cw[m][d], w[m] + (int64_t)(k + d * KC) * E, 16);
      }
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        cx[b][d] = lu32x4{0u, 0u, 0u, 0u};
        if (d < nfull) __builtin_memcpy(&cx[b][d], x[b] + (int64_t)(k + d * KC) * E, 16);
      }
    }
    const int kt = k + nfull * KC;
    lu32x4 tw[NM], tx[TB];
#pragma unroll
    for (int m = 0; m < NM; ++m) tw[m] = l_load<T, false>(w[m], kt, kEnd);
#pragma unroll
    for (int b = 0; b < TB; ++b) tx[b] = l_load<T, false>(x[b], kt, kEnd);
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[m][b] = few_mfma<T>(cw[m][d], cx[b][d], acc[m][b]);
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int b = 0; b < TB; ++b) acc[m][b] = few_mfma<T>(tw[m], tx[b], acc[m][b]);
  }
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][m * TB + b][r][lane] = acc[m][b][r];
  __syncthreads();

  // acc[m][b][r] is weight row 4·(lane/16) + r, token 16·b + lane%16; wave w
  // finishes the token blocks w, w + 4, ..
  for (int b = wave; b < TB; b += 4) {
    float s[NM][4];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        s[m][r] = ((sums[0][m * TB + b][r][lane] + sums[1][m * TB + b][r][lane]) + sums[2][m * TB + b][r][lane]) +
                  sums[3][m * TB + b][r][lane];
    const int64_t i = b * 16 + lr, j = j0 + 4 * lg;
    if (i >= P.M) continue;
    if (P.part) {
      ffn_part4(P, split, i, j, EPI == FFN_GLU, 0, s[0]);
      if constexpr (EPI == FFN_GLU) ffn_part4(P, split, i, j, true, 1, s[1]);
    } else if constexpr (EPI == FFN_GLU) {
      if (j >= L.ldh) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (j + r >= P.N) s[0][r] = s[1][r] = 0.f;
      ffn_with_glu(L, [&](auto actc, auto savec) __attribute__((always_inline)) {
        ffn_glu4<T, decltype(actc)::value, decltype(savec)::value>(L, P, i, j, s[0], s[1]);
      });
    } else if (j < P.N) {
      ffn_store4(P.C, P.ldc, i, j, P.N, V == 8, false, P.vecC, s[0]);
    }
  }
}

template <typename T, int EPI>
void few_launch(const FfnLaunch& L, int splits, hipStream_t st) {
  const dim3 grid((L.prob[0].N + 15) / 16, splits), block(256);
  const int tb = (L.prob[0].M + 15) / 16;
  if (tb == 1) hipLaunchKernelGGL((ffn_few<T, 1, EPI>), grid, block, 0, st, L);
  else if (tb == 2) hipLaunchKernelGGL((ffn_few<T, 2, EPI>), grid, block, 0, st, L);
  else if (tb == 3) hipLaunchKernelGGL((ffn_few<T, 3, EPI>), grid, block, 0, st, L);
  else hipLaunchKernelGGL((ffn_few<T, 4, EPI>), grid, block, 0, st, L);
}

}  // namespace

hipError_t launch_ffn_few(int epi, bool bf16, int splits, const FfnLaunch& L, hipStream_t st) {
  if (epi == FFN_GLU) {
    if (bf16) few_launch<Bf16, FFN_GLU>(L, splits, st);
    else few_launch<float, FFN_GLU>(L, splits, st);
  } else {
    if (bf16) few_launch<Bf16, FFN_STORE>(L, splits, st);
    else few_launch<float, FFN_STORE>(L, splits, st);
  }
  return hipGetLastError();
}

}  // namespace muon

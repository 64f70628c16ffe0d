// The sums of the backward pass that stretches share, added in the stretches'
// order by the workgroups of the one their block begins in: its part lies in that
// one's second slot, the others in the next ones' first.  One launch for the
// blocks of keys (attn_dkv) and of rows (attn_dq): of few tokens both are bound by
// their chains of dependent reads (333 tokens, fp32: 12.8 + 10.4 µs apart, 15.5
// together).  Of more tokens by reading the parts once (2048 tokens, 14 heads of
// 128: 130 MB in 46 µs).
#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

template <typename T, int DP> __device__ __forceinline__ void join_keys(const AttnGradLaunch& L, int number) {
  constexpr int E = AT<T>::kBytes, kKeys = 8;
  const AttnShape& S = L.s;
  const Stretch W(L.keyRuns, S.combos, number);
  if (W.stop >= W.total) return;
  const int64_t combo = W.stop / W.each;  // of the next stretch's first tile
  const int b = W.find(L.keyRuns, W.stop - combo * W.each);
  const int64_t from = combo * W.each + L.keyRuns.cum[b], to = combo * W.each + L.keyRuns.cum[b + 1];
  if (from >= W.stop || from < W.pos) return;  // not shared, or begun before
  const AttnBlock B = L.keyRuns.list.blocks[b];
  const int64_t batch = combo / S.kv, hk = combo % S.kv;
  constexpr int64_t kSlot = (int64_t)kDkvKeys * 4 * DP;
  for (int i = threadIdx.x; i < kKeys * DP; i += 256) {
    const int key = blockIdx.y * kKeys + i / DP, c0 = i % DP * 4;
    if (B.at + key >= B.n) break;
    const float* p = L.part + (int64_t)key * (4 * DP) + c0;
    lf32x4 s = *(const lf32x4*)(p + (2 * (int64_t)number + 1) * kSlot);
#pragma unroll 4
    for (int64_t w = number + 1; w * W.per < to; ++w) s += *(const lf32x4*)(p + 2 * w * kSlot);
    const int64_t tok = B.tok + B.at + key;
    if (c0 < 2 * DP) {
      const int m = c0 >= DP, c = c0 - m * DP;
      char* o = (char*)L.dk + (batch * L.dks[0] + tok * L.dks[1] + (2 * hk + m) * L.dks[2]) * E;
      for (int j = 0; j < 4; ++j)
        if (c + j < S.dim) LType<T>::put(o, c + j, s[j] * L.scale);
    } else {
      const int c = c0 - 2 * DP;
      char* o = (char*)L.dv + (batch * L.dvs[0] + tok * L.dvs[1] + hk * L.dvs[2]) * E;
      for (int j = 0; j < 4; ++j)
        if (c + j < 2 * S.dim) LType<T>::put(o, c + j, s[j]);
    }
  }
}

template <typename T, int DP> __device__ __forceinline__ void join_rows(const AttnGradLaunch& L, int number) {
  constexpr int E = AT<T>::kBytes, kRows = 8, kLd = 2 * DP + 4, kCols = 2 * DP / 4 + 1;
  const AttnShape& S = L.s;
  const Stretch W(L.rowRuns, S.combos, number);
  if (W.stop >= W.total) return;
  const int64_t combo = W.stop / W.each;  // of the next stretch's first tile
  const int b = W.find(L.rowRuns, W.stop - combo * W.each);
  const int64_t from = combo * W.each + L.rowRuns.cum[b], to = combo * W.each + L.rowRuns.cum[b + 1];
  if (from >= W.stop || from < W.pos) return;  // not shared, or begun before
  const AttnBlock B = L.rowRuns.list.blocks[b];
  const int nq = L.packed ? B.n : (int)S.nq, nk = L.packed ? B.nk : (int)S.nk;
  const int batch = (int)combo / S.kv, hk = (int)combo % S.kv, G = S.group;
  constexpr int64_t kSlot = (int64_t)kDqRows * kLd;
  for (int i = threadIdx.x; i < kRows * kCols; i += 256) {
    const int r = blockIdx.y * kRows + i / kCols, c0 = i % kCols * 4;
    const int row = B.at + r;
    if (row >= nq * G) break;
    const float* p = L.rowPart + r * kLd + c0;
    lf32x4 s = *(const lf32x4*)(p + (2 * (int64_t)number + 1) * kSlot);
#pragma unroll 4
    for (int64_t w = number + 1; w * W.per < to; ++w) s += *(const lf32x4*)(p + 2 * w * kSlot);
    const int t = row / G, head = hk * G + row - t * G;
    const int64_t tok = B.tok + t;
    if (c0 == 2 * DP) {
      const int64_t at = ((int64_t)batch * L.heads + head) * S.nq + tok;
      L.rowLam[at] = L.rec[at].v[3] + s[0];
      continue;
    }
    if (!L.dq) continue;
    const int lim = S.causal ? min(t + nk - nq + 1, nk) : nk;
    const int m = c0 >= DP, c = c0 - m * DP;
    const float f = lim > 1 ? m ? -S.lam[head] * L.scale : L.scale : 0.f;
    char* o = (char*)L.dq + (batch * L.dqs[0] + tok * L.dqs[1] + (2 * head + m) * L.dqs[2]) * E;
    for (int j = 0; j < 4; ++j)
      if (c + j < S.dim) LType<T>::put(o, c + j, lim > 1 ? s[j] * f : 0.f);
  }
}

template <typename T, int DP> __global__ __launch_bounds__(256) void attn_grad_join(const AttnGradLaunch L) {
  const int keys = L.joinKeys ? L.keyRuns.streams : 0;
  if ((int)blockIdx.x < keys) join_keys<T, DP>(L, blockIdx.x);
  else join_rows<T, DP>(L, blockIdx.x - keys);
}

template <typename T, int DP> hipError_t run(const AttnGradLaunch& L, hipStream_t st) {
  const int n = (L.joinKeys ? L.keyRuns.streams : 0) + (L.joinRows ? L.rowRuns.streams : 0);
  static_assert(kDkvKeys == kDqRows, "one grid for both");
  attn_grad_join<T, DP><<<dim3(n, kDqRows / 8), 256, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_grad_join(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st) {
  if (bf16) return dp == 64 ? run<Bf16, 64>(L, st) : run<Bf16, 128>(L, st);
  return dp == 64 ? run<float, 64>(L, st) : run<float, 128>(L, st);
}

}  // namespace muon

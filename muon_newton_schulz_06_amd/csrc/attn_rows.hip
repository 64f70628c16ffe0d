// The row sums of the attention's backward pass, and the sum of λ's gradient.
//
// With O = O_1 − λ·O_2, O_m = P_m·V:  δ_m = Σ_j P_m·dA = dO·O_m.  One pass over dO
// and what the forward pass kept, bound by HBM; 16 lanes share a row.
//
// fp32: δ_1 = dO·O + λ·δ_2 from O and the kept O_2.  bf16: from O_1 and O_2,
// kept as 16-bit whole multiples of a unit of the row, 2^-15 of its largest
// value: rounded to bf16 they would be off by 2^-8 of themselves, and δ with
// them, where a row sees few keys by several times the rounding of the
// dS = P·(dA − δ) that it goes into (of dK of two keys, 40 values a head:
// 6.6·10^-3 instead of 2.5·10^-3).  4 × 4096 tokens, 28 heads of 64 on 4: 94 µs, 4.1
// TB/s, of which 4 for the keys, which are looked through for infinities and NaN.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"
#include "attn_lists.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

// x as the sum of three bf16 (24 bits of it).
__device__ __forceinline__ void split3(float x, uint32_t (&h)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    h[i] = l_f32_bf16(x);
    x -= l_bf16_f32(h[i]);
  }
}

// Whole multiples of a unit.
__device__ __forceinline__ void widen_whole(const lu32x4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (float)(int16_t)v[i];
    f[2 * i + 1] = (float)((int32_t)v[i] >> 16);
  }
}

// Which keys hold an infinity or NaN, for attn_dq: 16 lanes the two maps of a key.
template <typename T> __device__ __forceinline__ void odd_keys(const AttnGradLaunch& L, int block, int blocks) {
  constexpr int V = LType<T>::kVec, E = AT<T>::kBytes;
  const AttnShape& S = L.s;
  const int lane = threadIdx.x & 15, chunks = (S.dim + V - 1) / V;
  const int64_t keys = (int64_t)S.combos * S.nk;
  for (int64_t id = (int64_t)block * (kPrep / 16) + (threadIdx.x >> 4); id < keys; id += (int64_t)blocks * (kPrep / 16)) {
    const int64_t bt = id / S.kv, hk = id - bt * S.kv, b = bt / S.nk, t = bt - b * S.nk;
    const char* k = (const char*)S.k + (b * S.ks[0] + t * S.ks[1] + 2 * hk * S.ks[2]) * E;
    uint32_t top = 0;
    for (int i = lane; i < 2 * chunks; i += 16)
      top = a_top<T>(*(const lu32x4*)(k + (i < chunks ? 0 : S.ks[2] * E) + (i < chunks ? i : i - chunks) * 16), top);
    const uint64_t odd = __ballot(a_odd<T>(top)) >> (threadIdx.x & 48);
    if (lane == 0) L.oddKeys[(b * S.kv + hk) * S.nk + t] = (odd & 0xffff) != 0;
  }
}

// The first workgroups make the lists of the products that follow, which take as
// long (7 µs: scans and searches by one workgroup) as the sums of few rows.
template <typename T, bool VEC>
__global__ __launch_bounds__(kPrep, 8)  // two workgroups a CU
void attn_rows(const AttnGradLaunch L, const AttnPrepLaunch P, int blocks) {
  if ((int)blockIdx.x < P.lists) return attn_lists(P, blockIdx.x);
  if ((int)blockIdx.x >= P.lists + blocks) return odd_keys<T>(L, blockIdx.x - P.lists - blocks, gridDim.x - P.lists - blocks);
  constexpr int V = LType<T>::kVec, E = AT<T>::kBytes;
  const AttnShape& S = L.s;
  const int64_t rows = (int64_t)L.batch * S.nq * L.heads;
  const int64_t each = (int64_t)blocks * (kPrep / 16);
  for (int64_t id = (int64_t)(blockIdx.x - P.lists) * (kPrep / 16) + (threadIdx.x >> 4); id < rows; id += each) {
    const int lane = threadIdx.x & 15;
    const int64_t bt = id / L.heads;
    const int h = (int)(id - bt * L.heads);
    const int64_t b = bt / S.nq, t = bt - b * S.nq;
    const int hk = h / S.group, g = h - hk * S.group;
    const int64_t combo = b * S.kv + hk, row = t * S.group + g, all = S.nq * S.group;
    const char* d = (const char*)L.dout + (b * L.gs[0] + t * L.gs[1] + h * L.gs[2]) * E;
    const char* o = (const char*)L.out + (b * L.os[0] + t * L.os[1] + h * L.os[2]) * E;
    const int64_t at1 = E == 2 ? combo * 2 * all + row : 0, at2 = E == 2 ? at1 + all : combo * all + row;
    const char* o1 = E == 2 ? (const char*)S.kept + at1 * S.pitch * E : o;
    const char* o2 = (const char*)S.kept + at2 * S.pitch * E;
    const int width = 2 * S.dim;
    float s1 = 0.f, s2 = 0.f;
    uint32_t top = 0;
    for (int c = lane * V; c < width; c += 16 * V) {
      // zeros past the width, as in the kept rows
      const lu32x4 cx = *(const lu32x4*)(d + c * E), cz = *(const lu32x4*)(o2 + c * E);
      lu32x4 cy;
      if constexpr (E == 2) cy = *(const lu32x4*)(o1 + c * E);
      else cy = l_load<T, VEC>(o1, c, width);
      __builtin_amdgcn_sched_barrier(0);  // all three on their way
      top = a_top<T>(cx, top);
      float x[V], y[V], z[V];
      l_widen<T>(cx, x);
      if constexpr (E == 2) {
        widen_whole(cy, y);
        widen_whole(cz, z);
      } else {
        l_widen<T>(cy, y);
        l_widen<T>(cz, z);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s1 += x[i] * y[i];
        s2 += x[i] * z[i];
      }
    }
    if (a_odd<T>(top)) s1 = s2 = __builtin_nanf("");  // of an infinity too: attn_dkv takes it out of dO
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
      s1 += __shfl_xor(s1, w, 64);
      s2 += __shfl_xor(s2, w, 64);
    }
    if (lane) continue;
    if constexpr (E == 2) {
      s1 *= S.unit[at1];
      s2 *= S.unit[at2];
    } else {
      s1 += S.lam[h] * s2;
    }
    const float l1 = S.stat[(combo * 2) * all + row], l2 = S.stat[(combo * 2 + 1) * all + row];
    const uint32_t bad = a_bad_row(l1, l2, s1, s2);
    if (l2 == -kNegInf) s1 = s2 = 0.f;  // a row that sees no key, whatever its dO holds
    const int64_t at = (b * L.heads + h) * S.nq + t;
    L.rec[at] = lf4{{l1, l2, s1, s2}};
    if constexpr (E == 2) {
      // −L/c is finite: an infinity would meet zeros in the product
      uint32_t a[3], e[3];
      split3(fmaxf(fminf(-l1 / S.c, 1e30f), -1e30f), a);
      split3(fmaxf(fminf(-l2 / S.c, 1e30f), -1e30f), e);
      if (__builtin_expect(bad, 0)) {
        // a NaN is three finite values whose sum is infinite; and a map without a finite
        // log-sum has P = 0, ∞ or NaN whatever δ, whose NaN would meet zeros too
        if (l1 != l1) a[0] = a[1] = a[2] = 0x7f7fu;
        if (l2 != l2) e[0] = e[1] = e[2] = 0x7f7fu;
        if (bad & 1) s1 = 0.f;
        if (bad & 2) s2 = 0.f;
      }
      // (as values of the product the marks are as good as zeros, and meet zeros)
      L.recL[at] = lu4{{a[0] | a[1] << 16, a[2] | e[0] << 16, e[1] | e[2] << 16, bad}};
      split3(-s1, a);
      split3(-s2, e);
      L.recD[at] = lu4{{a[0] | a[1] << 16, a[2] | e[0] << 16, e[1] | e[2] << 16, 0u}};
    }
  }
}

// dλ of a head: minus the sum of its rows' δ_2, in an order fixed by the sizes.
// A workgroup per head, bound by the latency of its loads: 16 waves with four
// loads in flight each (4x4096 rows: 23 µs with four waves of one load, 5.4 now).
constexpr int kLamThreads = 1024, kLamLoads = 4;
__global__ __launch_bounds__(kLamThreads) void attn_dlam(const AttnGradLaunch L) {
  __shared__ float red[kLamThreads / 64];
  const int h = blockIdx.x;
  float s[kLamLoads] = {};
  for (int b = 0; b < L.batch; ++b) {
    const float* p = L.rowLam + ((int64_t)b * L.heads + h) * L.s.nq;
    for (int64_t t0 = threadIdx.x; t0 < L.s.nq; t0 += kLamThreads * kLamLoads)
#pragma unroll
      for (int i = 0; i < kLamLoads; ++i) {
        const int64_t t = t0 + i * kLamThreads;
        s[i] += t < L.s.nq ? p[t] : 0.f;
      }
  }
  float sum = l_wave_sum((s[0] + s[1]) + (s[2] + s[3]));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  sum = l_wave_sum(threadIdx.x < kLamThreads / 64 ? red[threadIdx.x] : 0.f);
  if (threadIdx.x == 0) L.dlam[h] = -sum;
}

}  // namespace

hipError_t launch_attn_rows(bool bf16, const AttnGradLaunch& L, const AttnPrepLaunch& P, hipStream_t st) {
  auto blocks = [](int64_t n) { return (int)std::min<int64_t>((n + kPrep / 16 - 1) / (kPrep / 16), 1 << 20); };
  const int rows = blocks((int64_t)L.batch * L.s.nq * L.heads);
  const dim3 grid((unsigned)(P.lists + rows + (L.oddKeys ? blocks((int64_t)L.s.combos * L.s.nk) : 0)));
  if (bf16) attn_rows<Bf16, true><<<grid, kPrep, 0, st>>>(L, P, rows);
  else if (L.outVec) attn_rows<float, true><<<grid, kPrep, 0, st>>>(L, P, rows);
  else attn_rows<float, false><<<grid, kPrep, 0, st>>>(L, P, rows);
  return hipGetLastError();
}

hipError_t launch_attn_dlam(const AttnGradLaunch& L, hipStream_t st) {
  attn_dlam<<<dim3(L.heads), kLamThreads, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace muon

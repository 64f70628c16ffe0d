// The row sums of the attention's backward pass, and the sum of λ's gradient.
//
// With O = O_1 − λ·O_2, O_m = P_m·V:  δ_2 = Σ_j P_2·dA = dO·O_2 and
// δ_1 = dO·O_1 = dO·O + λ·δ_2.  One pass over dO, O and the saved O_2, bound by
// HBM; 16 lanes share a row.
#include <hip/hip_runtime.h>

#include "attention.hpp"
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

template <typename T, bool VEC> __global__ __launch_bounds__(256) void attn_rows(const AttnGradLaunch L) {
  constexpr int V = LType<T>::kVec, E = AT<T>::kBytes;
  const AttnShape& S = L.s;
  const int64_t rows = (int64_t)L.batch * S.nq * L.heads;
  const int64_t id = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (id >= rows) return;
  const int lane = threadIdx.x & 15;
  const int64_t bt = id / L.heads;
  const int h = (int)(id - bt * L.heads);
  const int64_t b = bt / S.nq, t = bt - b * S.nq;
  const int hk = h / S.group, g = h - hk * S.group;
  const int64_t combo = b * S.kv + hk, row = t * S.group + g, all = S.nq * S.group;
  const char* d = (const char*)L.dout + (b * L.gs[0] + t * L.gs[1] + h * L.gs[2]) * E;
  const char* o = (const char*)L.out + (b * L.os[0] + t * L.os[1] + h * L.os[2]) * E;
  const char* o2 = (const char*)S.o2 + (combo * all + row) * S.pitch * E;
  const int width = 2 * S.dim;
  float s = 0.f, s2 = 0.f;
  for (int c = lane * V; c < width; c += 16 * V) {
    float x[V], y[V], z[V];
    l_widen<T>(*(const lu32x4*)(d + c * E), x);  // zeros past the width
    l_widen<T>(l_load<T, VEC>(o, c, width), y);
    l_widen<T>(*(const lu32x4*)(o2 + c * E), z);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s += x[i] * y[i];
      s2 += x[i] * z[i];
    }
  }
#pragma unroll
  for (int w = 8; w > 0; w >>= 1) {
    s += __shfl_xor(s, w, 64);
    s2 += __shfl_xor(s2, w, 64);
  }
  if (lane) return;
  const float s1 = s + S.lam[h] * s2;
  const float l1 = S.stat[(combo * 2) * all + row], l2 = S.stat[(combo * 2 + 1) * all + row];
  const int64_t at = (b * L.heads + h) * S.nq + t;
  L.rec[at] = lf4{{l1, l2, s1, s2}};
  if constexpr (E == 2) {
    // −L/c is finite: an infinity would meet zeros in the product
    uint32_t a[3], e[3];
    split3(fmaxf(fminf(-l1 / S.c, 1e30f), -1e30f), a);
    split3(fmaxf(fminf(-l2 / S.c, 1e30f), -1e30f), e);
    L.recL[at] = lu4{{a[0] | a[1] << 16, a[2] | e[0] << 16, e[1] | e[2] << 16, 0u}};
    split3(-s1, a);
    split3(-s2, e);
    L.recD[at] = lu4{{a[0] | a[1] << 16, a[2] | e[0] << 16, e[1] | e[2] << 16, 0u}};
  }
}

// dλ of a head: minus the sum of its rows' δ_2, in an order fixed by the sizes.
__global__ __launch_bounds__(256) void attn_dlam(const AttnGradLaunch L) {
  __shared__ float red[4];
  const int h = blockIdx.x;
  float s = 0.f;
  for (int b = 0; b < L.batch; ++b) {
    const float* p = L.rowLam + ((int64_t)b * L.heads + h) * L.s.nq;
    for (int64_t t = threadIdx.x; t < L.s.nq; t += 256) s += p[t];
  }
  s = l_wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) L.dlam[h] = -(red[0] + red[1] + red[2] + red[3]);
}

}  // namespace

hipError_t launch_attn_rows(bool bf16, const AttnGradLaunch& L, hipStream_t st) {
  const int64_t rows = (int64_t)L.batch * L.s.nq * L.heads;
  const dim3 grid((unsigned)((rows + 15) / 16));
  if (bf16) {
    if (L.outVec) attn_rows<Bf16, true><<<grid, 256, 0, st>>>(L);
    else attn_rows<Bf16, false><<<grid, 256, 0, st>>>(L);
  } else {
    if (L.outVec) attn_rows<float, true><<<grid, 256, 0, st>>>(L);
    else attn_rows<float, false><<<grid, 256, 0, st>>>(L);
  }
  return hipGetLastError();
}

hipError_t launch_attn_dlam(const AttnGradLaunch& L, hipStream_t st) {
  attn_dlam<<<dim3(L.heads), 256, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace muon

// Rotation of queries and keys by their positions.
//
// Pair i of a head (values i and i + R/2, or 2i and 2i + 1) turns by the angle
// θ = position·freq[i]:  (a, b) → scale·(a·cosθ − b·sinθ, a·sinθ + b·cosθ);
// the gradient turns by −θ.
//
// HBM-bound: every value is read and written once.  The angles are the same
// for all heads, so a workgroup takes whole tokens, all heads of q and k: it
// forms cosθ and sinθ of a token's pairs once in LDS and applies them from
// there.  Angles are fp64: a position of 10^6 times a frequency of 1 in fp32
// is off by up to 0.03 rad, and the fp64 product with its reduction to one
// turn is a few instructions per pair and token.  The reduced angle is
// rounded to fp32 (2^-25 of a turn) for the sine and cosine.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"
#include "layers.hpp"

namespace muon {
namespace {

constexpr int kThreads = 256;

// V consecutive elements of T, one access of any alignment.
template <typename T, int V> struct Group {
  static constexpr int kBytes = V * (16 / LType<T>::kVec);
  uint32_t d[(kBytes + 3) / 4];
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (kBytes == 2) {
      uint16_t h;
      __builtin_memcpy(&h, p, 2);
      d[0] = h;
    } else {
      __builtin_memcpy(d, p, kBytes);
    }
  }
  __device__ __forceinline__ void store(char* p) const { __builtin_memcpy(p, d, kBytes); }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (LType<T>::kVec == 4) return __uint_as_float(d[i]);
    else return __uint_as_float(i & 1 ? d[i / 2] & 0xffff0000u : d[i / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (LType<T>::kVec == 4) {
      for (int i = 0; i < V; ++i) d[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
      d[0] = l_f32_bf16(v[0]);
    } else {
      for (int i = 0; i < V / 2; ++i) d[i] = l_f32_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
};

// TB tokens per workgroup: their loads are in flight together.
template <typename T, int V, bool INTER, int TB>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotaryLaunch L) {
  constexpr int E = 16 / LType<T>::kVec;  // bytes of an element
  extern __shared__ float2 cs[];          // [TB][rot / 2] (cosθ, ±sinθ) · scale
  const int half = L.rot / 2, tid = threadIdx.x;
  const int64_t total = L.batch * L.tokens, first = (int64_t)blockIdx.x * TB;
  for (int i = tid; i < TB * half; i += kThreads) {
    const int k = TB == 1 ? 0 : i / half;
    const int64_t at = first + k;
    if (at >= total) break;
    const int64_t b = at / L.tokens, t = at - b * L.tokens;
    double p = (double)(L.start + t);
    if (L.pos) {
      const int64_t e = b * L.posBatch + t;
      p = L.pos64 ? (double)((const int64_t*)L.pos)[e] : (double)((const int32_t*)L.pos)[e];
    }
    double turns = p * L.freqs[i - k * half] * 0.15915494309189533577;  // 1 / 2π
    turns -= rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    cs[i] = float2{c * L.scale, (L.inverse ? -s : s) * L.scale};
  }
  __syncthreads();
  // a head's items: its pairs (V pairs of the half layout, V values of the
  // interleaved one), then groups of V values past them, the last not always whole
  const int turned = INTER ? L.rot / V : half / V;
  const int per = turned + (L.copyRest ? (L.dim - L.rot + V - 1) / V : 0);
  int c = tid % per, h = tid / per;
  const int dc = kThreads % per, dh = kThreads / per;
  for (; h < L.heads; c += dc, h += dh) {
    if (c >= per) {
      c -= per;
      if (++h >= L.heads) break;
    }
    const int z = h >= L.side[0].heads;
    const RotarySide& S = L.side[z];
    const int hh = h - (z ? L.side[0].heads : 0);
    const bool turn = c < turned;
    const int e0 = turn ? c * V : L.rot + (c - turned) * V;
    const bool whole = e0 + V <= L.dim;
    Group<T, V> a[TB], b[TB];
    int64_t out[TB];
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      const int64_t at = first + k;
      if (at >= total) continue;
      const int64_t bb = at / L.tokens, t = at - bb * L.tokens;
      const char* in = (const char*)S.in + (bb * S.in_s[0] + t * S.in_s[1] + hh * S.in_s[2] + e0) * E;
      out[k] = bb * S.out_s[0] + t * S.out_s[1] + hh * S.out_s[2] + e0;
      if (!whole) {
        for (int i = 0; e0 + i < L.dim; ++i) LType<T>::put((char*)S.out + out[k] * E, i, LType<T>::get(in, i));
        continue;
      }
      a[k].load(in);
      if (!INTER && turn) b[k].load(in + half * E);
    }
#pragma unroll
    for (int k = 0; k < TB; ++k) {
      if (first + k >= total || !whole) continue;
      char* o = (char*)S.out + out[k] * E;
      if (turn) {
        const float2* w = cs + k * half + (INTER ? e0 / 2 : e0);
        float x[V], y[V];
        if constexpr (INTER) {
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 r = w[i / 2];
            const float u = a[k].get(i), v = a[k].get(i + 1);
            x[i] = u * r.x - v * r.y;
            x[i + 1] = u * r.y + v * r.x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 r = w[i];
            const float u = a[k].get(i), v = b[k].get(i);
            x[i] = u * r.x - v * r.y;
            y[i] = u * r.y + v * r.x;
          }
          b[k].set(y);
          b[k].store(o + half * E);
        }
        a[k].set(x);
      }
      a[k].store(o);
    }
  }
}

template <typename T, int V, bool INTER> hipError_t run(const RotaryLaunch& L, hipStream_t st) {
  const int64_t total = L.batch * L.tokens;
  // four tokens per workgroup once that leaves two workgroups per CU
  const bool four = total >= 2048;
  const size_t lds = (size_t)(four ? 4 : 1) * (L.rot / 2) * sizeof(float2);
  const dim3 grid((unsigned)(four ? (total + 3) / 4 : total));
  if (four) rotary_kernel<T, V, INTER, 4><<<grid, kThreads, lds, st>>>(L);
  else rotary_kernel<T, V, INTER, 1><<<grid, kThreads, lds, st>>>(L);
  return hipGetLastError();
}

template <typename T> hipError_t by_width(const RotaryLaunch& L, hipStream_t st) {
  if (L.interleaved) {
    if constexpr (LType<T>::kVec == 8)
      if (L.vec == 8) return run<T, 8, true>(L, st);
    return L.vec >= 4 ? run<T, 4, true>(L, st) : run<T, 2, true>(L, st);
  }
  if constexpr (LType<T>::kVec == 8)
    if (L.vec == 8) return run<T, 8, false>(L, st);
  if (L.vec >= 4) return run<T, 4, false>(L, st);
  return L.vec == 2 ? run<T, 2, false>(L, st) : run<T, 1, false>(L, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryLaunch& L, hipStream_t st) {
  return L.bf16 ? by_width<Bf16>(L, st) : by_width<float>(L, st);
}

}  // namespace muon

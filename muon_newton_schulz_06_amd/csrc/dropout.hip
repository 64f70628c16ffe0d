// Dropout with the residual's addition: y = r + x·mult where the element's
// random word is at least the threshold, y = r elsewhere.
//
// The words are those of the counter-based generator Philox4x32-10 (Salmon,
// Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3, SC 2011):
// element i takes word i mod 4 of the block with counter (i / 4, offset) and
// key `seed`.  A block is a function of its counter alone, so the gradient
// makes the same words again and no mask is stored.
//
// HBM-bound if the generator keeps up: a block of four words is twenty
// 32×32→64-bit products and about sixty other operations, shared by four
// elements.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"
#include "layers.hpp"

namespace muon {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void philox(uint64_t index, uint64_t offset, uint32_t k0, uint32_t k1, uint32_t (&w)[4]) {
  uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0;
  w[1] = c1;
  w[2] = c2;
  w[3] = c3;
}

// Kept where the word says so (a selection, not a product: a dropped
// infinity or NaN is dropped), plus the residual in fp32, rounded once.
template <typename T, bool RES>
__device__ __forceinline__ lu32x4 apply(const DropoutLaunch& L, const uint32_t (&w)[LType<T>::kVec], lu32x4 cx, lu32x4 cr) {
  constexpr int V = LType<T>::kVec;
  float x[V], r[V];
  l_widen<T>(cx, x);
  if constexpr (RES) l_widen<T>(cr, r);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float kept = !L.none && w[i] >= L.threshold ? x[i] * L.mult : 0.f;
    x[i] = RES ? kept + r[i] : kept;
  }
  return l_narrow<T>(x);
}

// One row of whole aligned chunks.
template <typename T, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_flat(const DropoutLaunch L) {
  constexpr int V = LType<T>::kVec, U = 4;
  const int64_t n = L.cols / V;
  const uint64_t offset = L.offset + (L.offsetDev ? *L.offsetDev : 0);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads * U) + threadIdx.x; i0 < n;
       i0 += (int64_t)gridDim.x * (kThreads * U)) {
    lu32x4 cx[U], cr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kThreads;
      if (i >= n) break;
      cx[u] = ((const lu32x4*)L.x)[i];
      if constexpr (RES) cr[u] = ((const lu32x4*)L.res)[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kThreads;
      if (i >= n) break;
      uint32_t w[V];
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        uint32_t f[4];
        philox((uint64_t)i * (V / 4) + q, offset, L.key[0], L.key[1], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * q + j] = f[j];
      }
      ((lu32x4*)L.y)[i] = apply<T, RES>(L, w, cx[u], cr[u]);
    }
  }
}

// Rows of any stride, alignment and length: a chunk's elements may begin
// inside a block of four words.
template <typename T, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_rows(const DropoutLaunch L) {
  constexpr int V = LType<T>::kVec, E = 16 / V;
  const int64_t per = (L.cols + V - 1) / V, n = per * L.rows;
  const uint64_t offset = L.offset + (L.offsetDev ? *L.offsetDev : 0);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / per, e = (i - row * per) * V;
    const uint64_t at = (uint64_t)(row * L.cols + e);
    uint32_t f[V + 4];
#pragma unroll
    for (int q = 0; q < V / 4 + 1; ++q) {
      uint32_t g[4] = {0, 0, 0, 0};
      if (q < V / 4 || (at & 3)) philox(at / 4 + q, offset, L.key[0], L.key[1], g);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * q + j] = g[j];
    }
    const int shift = at & 3;
    uint32_t w[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      w[j] = shift == 0 ? f[j] : shift == 1 ? f[j + 1] : shift == 2 ? f[j + 2] : f[j + 3];
    const lu32x4 cx = l_load<T, false>((const char*)L.x + row * L.ldx * E, e, L.cols);
    lu32x4 cr{};
    if constexpr (RES) cr = l_load<T, false>((const char*)L.res + row * L.ldr * E, e, L.cols);
    l_store<T, false>((char*)L.y + row * L.ldy * E, e, L.cols, apply<T, RES>(L, w, cx, cr));
  }
}

template <typename T, bool RES> hipError_t run(const DropoutLaunch& L, hipStream_t st) {
  constexpr int V = LType<T>::kVec;
  if (L.vec) {
    const int64_t n = L.cols / V;
    dropout_flat<T, RES><<<dim3((unsigned)std::min<int64_t>((n + kThreads * 4 - 1) / (kThreads * 4), 1 << 20)), kThreads, 0, st>>>(L);
  } else {
    const int64_t n = (L.cols + V - 1) / V * L.rows;
    dropout_rows<T, RES><<<dim3((unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, 1 << 20)), kThreads, 0, st>>>(L);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutLaunch& L, hipStream_t st) {
  if (L.bf16) return L.res ? run<Bf16, true>(L, st) : run<Bf16, false>(L, st);
  return L.res ? run<float, true>(L, st) : run<float, false>(L, st);
}

}  // namespace muon

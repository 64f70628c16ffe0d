// Root-mean-square norm with the residual's addition, forward and backward.
//
// Forward, per row: s = x + r, rstd = 1/√(mean s² + eps), y = s·rstd·w, one
// pass: the row's chunks stay in registers between the sum of squares and
// the scaling (rows too long for that are read twice).
// Backward, per row: n = s·rstd, c = mean(w·dy·n), dx = rstd·(w·dy − n·c) +
// dsum, also one pass; dw = Σ dy·n is kept per thread for its columns over all
// the rows of a workgroup, written once per workgroup, and the workgroups'
// rows are added in workgroup order by a second kernel (no atomics).
// Both are HBM-bound: 16384 × 3584 bf16 with residual forward 88 µs (5.3 TB/s),
// backward 89 + 5 µs (5.0 TB/s).  Rows of more than 8192 elements are not, in
// the backward pass (see plan_row).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layers.hpp"

namespace muon {
namespace {

// Forward launches have a workgroup per row (or four rows): up to 2^24 of up to
// 1024 threads, where a grid dimension holds less than 2^32 threads, so the
// rows are spread over two dimensions.
constexpr int64_t kRowGrid = int64_t(1) << 21;
dim3 row_grid(int64_t blocks) {
  return dim3(std::min(blocks, kRowGrid), (blocks + kRowGrid - 1) / kRowGrid);  // the last ones may have no row
}
__device__ __forceinline__ int64_t row_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Sum over the WAVES waves that share a row.  `slot` alternates between two
// halves of red from row to row, so one barrier per row is enough.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* red, int slot) {
  v = l_wave_sum(v);
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[slot * WAVES + wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += red[slot * WAVES + w];
  }
  return v;
}

__device__ __forceinline__ float load_w(const void* w, int bf16, int64_t e) {
  return bf16 ? LType<Bf16>::get(w, e) : LType<float>::get(w, e);
}

// V weights from element e on (as many as exist).
template <int V>
__device__ __forceinline__ void load_ws(const void* w, int bf16, int64_t e, int64_t n, float (&f)[V]) {
  if (((uintptr_t)w & 15) == 0 && e + V <= n) {
    if (bf16) {
      if constexpr (V == 8) {
        l_widen<Bf16>(*(const lu32x4*)((const uint16_t*)w + e), f);
      } else {
        const uint2 u = *(const uint2*)((const uint16_t*)w + e);
        f[0] = __uint_as_float(u.x << 16);
        f[1] = __uint_as_float(u.x & 0xffff0000u);
        f[2] = __uint_as_float(u.y << 16);
        f[3] = __uint_as_float(u.y & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < V; h += 4) {
        const lf32x4 u = *(const lf32x4*)((const float*)w + e + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[h + i] = u[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = e + i < n ? load_w(w, bf16, e + i) : 0.f;
  }
}

// WAVES waves per row (1: four rows per workgroup), ITEMS chunks per thread.
template <typename T, bool VEC, int WAVES, int ITEMS>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void norm_fwd(const NormFwdLaunch L) {
  constexpr int V = LType<T>::kVec, E = 16 / V, TPR = 64 * WAVES;
  __shared__ float red[2 * WAVES];
  const int64_t t = WAVES == 1 ? row_block() * 4 + (threadIdx.x >> 6) : row_block();
  if (t >= L.tokens) return;  // whole waves; a shared row's waves leave together
  const int l = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const char* x = (const char*)L.x + t * L.ldx * E;
  const char* r = L.res ? (const char*)L.res + t * L.ldr * E : nullptr;
  float s[ITEMS][V], w[ITEMS][V];
  lu32x4 cx[ITEMS], cr[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t e = (int64_t)(l + i * TPR) * V;
    cx[i] = cr[i] = lu32x4{0u, 0u, 0u, 0u};
    if (e < L.dim) {
      cx[i] = l_load<T, VEC>(x, e, L.dim);
      if (r) cr[i] = l_load<T, VEC>(r, e, L.dim);
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) load_ws<V>(L.w, L.wBf16, (int64_t)(l + i * TPR) * V, L.dim, w[i]);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    float a[V], b[V];
    l_widen<T>(cx[i], a);
    l_widen<T>(cr[i], b);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      s[i][k] = r ? a[k] + b[k] : a[k];
      ss = fmaf(s[i][k], s[i][k], ss);
    }
  }
  ss = row_sum<WAVES>(ss, red, 0);
  const float rstd = 1.0f / sqrtf(ss / (float)L.dim + L.eps);
  if (L.rstd && l == 0) L.rstd[t] = rstd;
  char* y = (char*)L.y + t * L.ldy * E;
  char* sum = L.sum ? (char*)L.sum + t * L.lds * E : nullptr;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t e = (int64_t)(l + i * TPR) * V;
    if (e < L.dim) {
      if (sum) l_store<T, VEC>(sum, e, L.dim, l_narrow<T>(s[i]));
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = s[i][k] * rstd * w[i][k];
      l_store<T, VEC>(y, e, L.dim, l_narrow<T>(o));
    }
  }
}

// Rows of any length: 16 waves per row, the row read again for the output.
template <typename T, bool VEC>
__global__ __launch_bounds__(1024) void norm_fwd_long(const NormFwdLaunch L) {
  constexpr int V = LType<T>::kVec, E = 16 / V;
  __shared__ float red[32];
  const int64_t t = row_block();
  if (t >= L.tokens) return;
  const char* x = (const char*)L.x + t * L.ldx * E;
  const char* r = L.res ? (const char*)L.res + t * L.ldr * E : nullptr;
  auto load = [&](int64_t e, float (&s)[V]) {
    l_widen<T>(l_load<T, VEC>(x, e, L.dim), s);
    if (r) {
      float b[V];
      l_widen<T>(l_load<T, VEC>(r, e, L.dim), b);
#pragma unroll
      for (int k = 0; k < V; ++k) s[k] += b[k];
    }
  };
  float ss = 0.f;
  for (int64_t e = (int64_t)threadIdx.x * V; e < L.dim; e += 1024 * V) {
    float s[V];
    load(e, s);
#pragma unroll
    for (int k = 0; k < V; ++k) ss = fmaf(s[k], s[k], ss);
  }
  ss = row_sum<16>(ss, red, 0);
  const float rstd = 1.0f / sqrtf(ss / (float)L.dim + L.eps);
  if (L.rstd && threadIdx.x == 0) L.rstd[t] = rstd;
  char* y = (char*)L.y + t * L.ldy * E;
  char* sum = L.sum ? (char*)L.sum + t * L.lds * E : nullptr;
  for (int64_t e = (int64_t)threadIdx.x * V; e < L.dim; e += 1024 * V) {
    float s[V], w[V], o[V];
    load(e, s);
    load_ws<V>(L.w, L.wBf16, e, L.dim, w);
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = s[k] * rstd * w[k];
    if (sum) l_store<T, VEC>(sum, e, L.dim, l_narrow<T>(s));
    l_store<T, VEC>(y, e, L.dim, l_narrow<T>(o));
  }
}

// Row groups (one wave, or the workgroup) walk the rows with a stride of all
// groups of the grid; the next row is read while the current one is reduced.
// A thread's columns are the same for every row, so the weights and the
// column sums stay in registers.
template <typename T, bool VEC, int WAVES, int ITEMS>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void norm_bwd(const NormGradLaunch L) {
  constexpr int V = LType<T>::kVec, E = 16 / V, TPR = 64 * WAVES, GROUPS = WAVES == 1 ? 4 : 1;
  __shared__ float red[2 * WAVES];
  extern __shared__ float colsum[];  // WAVES == 1: dim sums of the four waves
  const int g = WAVES == 1 ? threadIdx.x >> 6 : 0;
  const int l = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  struct Row {
    lu32x4 y[ITEMS], s[ITEMS], d[ITEMS];
    float rstd;
  };
  auto load = [&](int64_t t, Row& r) __attribute__((always_inline)) {
    const char* dy = (const char*)L.dy + t * L.ldy * E;
    const char* sr = (const char*)L.s + t * L.lds * E;
    const char* ds = (const char*)L.dsum + t * L.ldd * E;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t e = (int64_t)(l + i * TPR) * V;
      r.y[i] = r.s[i] = r.d[i] = lu32x4{0u, 0u, 0u, 0u};
      if (e < L.dim) {
        r.y[i] = l_load<T, VEC>(dy, e, L.dim);
        r.s[i] = l_load<T, VEC>(sr, e, L.dim);
        if (L.dsum) r.d[i] = l_load<T, VEC>(ds, e, L.dim);
      }
    }
    r.rstd = L.rstd[t];
  };
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t t = (int64_t)blockIdx.x * GROUPS + g;
  Row row;
  if (t < L.tokens) load(t, row);
  float acc[ITEMS][V], w[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    load_ws<V>(L.w, L.wBf16, (int64_t)(l + i * TPR) * V, L.dim, w[i]);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[i][k] = 0.f;
  }
  const float inv = 1.0f / (float)L.dim;
  int slot = 0;
  for (; t < L.tokens; t += step) {
    Row next;
    if (t + step < L.tokens) load(t + step, next);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float a[V], b[V];
      l_widen<T>(row.y[i], a);
      l_widen<T>(row.s[i], b);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float n = b[k] * row.rstd;
        dot = fmaf(w[i][k] * a[k], n, dot);
        acc[i][k] = fmaf(a[k], n, acc[i][k]);
      }
    }
    const float c = row_sum<WAVES>(dot, red, slot) * inv;
    slot ^= 1;
    char* dx = (char*)L.dx + t * L.ldx * E;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t e = (int64_t)(l + i * TPR) * V;
      if (e < L.dim) {
        float a[V], b[V], d[V], o[V];
        l_widen<T>(row.y[i], a);
        l_widen<T>(row.s[i], b);
        l_widen<T>(row.d[i], d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float v = row.rstd * (w[i][k] * a[k] - b[k] * row.rstd * c);
          o[k] = L.dsum ? v + d[k] : v;
        }
        l_store<T, VEC>(dx, e, L.dim, l_narrow<T>(o));
      }
    }
    row = next;
  }
  if (!L.dw) return;
  float* part = L.part + (int64_t)blockIdx.x * L.dim;
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t e = (int64_t)(l + i * TPR) * V;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (e + k < L.dim) part[e + k] = acc[i][k];
    }
  } else {
    // the four waves add their sums in wave order
    for (int w = 0; w < 4; ++w) {
      if (g == w) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int e = (l + i * TPR) * V;
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (e + k < L.dim) colsum[e + k] = w == 0 ? acc[i][k] : colsum[e + k] + acc[i][k];
        }
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < L.dim; e += 256) part[e] = colsum[e];
  }
}

// Rows of any length: 16 waves per row, rows read twice, dweight's partial
// sums kept in the workgroup's row of the workspace.
template <typename T, bool VEC>
__global__ __launch_bounds__(1024) void norm_bwd_long(const NormGradLaunch L) {
  constexpr int V = LType<T>::kVec, E = 16 / V;
  __shared__ float red[32];
  float* part = L.part + (int64_t)blockIdx.x * L.dim;
  if (L.dw)
    for (int64_t e = (int64_t)threadIdx.x * V; e < L.dim; e += 1024 * V)
      for (int k = 0; k < V; ++k)
        if (e + k < L.dim) part[e + k] = 0.f;
  int slot = 0;
  for (int64_t t = blockIdx.x; t < L.tokens; t += gridDim.x) {
    const char* dy = (const char*)L.dy + t * L.ldy * E;
    const char* sr = (const char*)L.s + t * L.lds * E;
    const char* ds = L.dsum ? (const char*)L.dsum + t * L.ldd * E : nullptr;
    char* dx = (char*)L.dx + t * L.ldx * E;
    const float rstd = L.rstd[t];
    float dot = 0.f;
    for (int64_t e = (int64_t)threadIdx.x * V; e < L.dim; e += 1024 * V) {
      float a[V], b[V], w[V];
      l_widen<T>(l_load<T, VEC>(dy, e, L.dim), a);
      l_widen<T>(l_load<T, VEC>(sr, e, L.dim), b);
      load_ws<V>(L.w, L.wBf16, e, L.dim, w);
      for (int k = 0; k < V; ++k) {
        const float n = b[k] * rstd;
        dot = fmaf(w[k] * a[k], n, dot);
        if (L.dw && e + k < L.dim) part[e + k] = fmaf(a[k], n, part[e + k]);
      }
    }
    const float c = row_sum<16>(dot, red, slot) / (float)L.dim;
    slot ^= 1;
    for (int64_t e = (int64_t)threadIdx.x * V; e < L.dim; e += 1024 * V) {
      float a[V], b[V], w[V], o[V];
      l_widen<T>(l_load<T, VEC>(dy, e, L.dim), a);
      l_widen<T>(l_load<T, VEC>(sr, e, L.dim), b);
      load_ws<V>(L.w, L.wBf16, e, L.dim, w);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = rstd * (w[k] * a[k] - b[k] * rstd * c);
      if (ds) {
        float d[V];
        l_widen<T>(l_load<T, VEC>(ds, e, L.dim), d);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] += d[k];
      }
      l_store<T, VEC>(dx, e, L.dim, l_narrow<T>(o));
    }
  }
}

// dweight[e] = Σ over workgroups, in order within each of 16 waves' runs of
// workgroups and then over the waves.
__global__ __launch_bounds__(1024) void norm_dw(const NormGradLaunch L) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t e = (int64_t)blockIdx.x * 64 + lane;
  const int per = (L.blocks + 15) / 16, lo = wave * per, hi = min(L.blocks, lo + per);
  float s = 0.f;
  if (e < L.dim) {
#pragma unroll 8
    for (int b = lo; b < hi; ++b) s += L.part[(int64_t)b * L.dim + e];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && e < L.dim) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += sums[w][lane];
    if (L.wBf16) {
      if (L.accumulate) v += LType<Bf16>::get(L.dw, e);
      LType<Bf16>::put(L.dw, e, v);
    } else {
      if (L.accumulate) v += LType<float>::get(L.dw, e);
      LType<float>::put(L.dw, e, v);
    }
  }
}

struct RowPlan {
  int waves;  // per row; 0: the long-row kernel
  int items;  // chunks per thread
};

// The fewest waves per row that leave a thread at most 16 elements (which
// keeps several workgroups on a CU); rows that 16 waves do not hold so take more
// per thread, up to 8 chunks.  The forward pass keeps its rate there (4096 rows
// with residual: 8192 bf16 47 µs, 5.7 TB/s; 16384 104, 5.2; 32768 209, 5.1).  The
// backward pass does not: a lane of 16 waves has 128 registers, and from two
// chunks of bf16 or four of fp32 on (above 8192 elements) two rows, the weights
// and the column sums spill to scratch memory (4096 rows with dsum: 8192 bf16 64
// µs, 4.2 TB/s; 12288 133, 3.0; 16384 157, 3.4; 32768 926, 1.2; fp32 8192 110,
// 4.9; 16384 439, 2.4; 32768 1764, 1.2).
RowPlan plan_row(int64_t chunks, int V) {
  for (int waves = 1; waves <= 16; waves *= 4)
    for (int items = 1; items <= (waves == 16 ? 8 : 16 / V); items *= 2)
      if (chunks <= (int64_t)64 * waves * items) return {waves, items};
  return {0, 0};
}

// Calls f with the plan's waves and items as compile-time constants.
template <int V, typename F> void with_plan(const RowPlan& p, F&& f) {
  auto items = [&](auto waves) {
    constexpr int W = decltype(waves)::value;
    if (p.items == 1) f(waves, std::integral_constant<int, 1>{});
    else if (p.items == 2) f(waves, std::integral_constant<int, 2>{});
    else if constexpr (W == 16 || V == 4) {
      if (p.items == 4) f(waves, std::integral_constant<int, 4>{});
      else if constexpr (W == 16) f(waves, std::integral_constant<int, 8>{});
    }
  };
  if (p.waves == 1) items(std::integral_constant<int, 1>{});
  else if (p.waves == 4) items(std::integral_constant<int, 4>{});
  else items(std::integral_constant<int, 16>{});
}

template <typename T, bool VEC>
hipError_t fwd_launch(const NormFwdLaunch& L, hipStream_t st) {
  constexpr int V = LType<T>::kVec;
  const RowPlan p = plan_row((L.dim + V - 1) / V, V);
  if (!p.waves) {
    hipLaunchKernelGGL((norm_fwd_long<T, VEC>), row_grid(L.tokens), dim3(1024), 0, st, L);
    return hipGetLastError();
  }
  with_plan<V>(p, [&](auto waves, auto items) {
    constexpr int W = decltype(waves)::value;
    const dim3 grid = row_grid(W == 1 ? (L.tokens + 3) / 4 : L.tokens), block(W == 1 ? 256 : 64 * W);
    hipLaunchKernelGGL((norm_fwd<T, VEC, W, decltype(items)::value>), grid, block, 0, st, L);
  });
  return hipGetLastError();
}

template <typename T, bool VEC>
void bwd_launch(const NormGradLaunch& L, hipStream_t st) {
  constexpr int V = LType<T>::kVec;
  const RowPlan p = plan_row((L.dim + V - 1) / V, V);
  if (!p.waves) {
    hipLaunchKernelGGL((norm_bwd_long<T, VEC>), dim3(L.blocks), dim3(1024), 0, st, L);
    return;
  }
  with_plan<V>(p, [&](auto waves, auto items) {
    constexpr int W = decltype(waves)::value;
    const size_t lds = W == 1 ? (size_t)L.dim * 4 : 0;  // at most 64 lanes × 16 elements: 4 KiB
    hipLaunchKernelGGL((norm_bwd<T, VEC, W, decltype(items)::value>), dim3(L.blocks), dim3(W == 1 ? 256 : 64 * W),
                       lds, st, L);
  });
}

}  // namespace

hipError_t launch_rms_norm(const NormFwdLaunch& L, hipStream_t st) {
  if (L.bf16) return L.vec ? fwd_launch<Bf16, true>(L, st) : fwd_launch<Bf16, false>(L, st);
  return L.vec ? fwd_launch<float, true>(L, st) : fwd_launch<float, false>(L, st);
}

// Measured on 16384×3584 bf16 (µs for 512, 768, 1024, 2048 workgroups): 93, 99,
// 110, 114; fp32: 180, 196, 190, 198.  More workgroups write and add up more
// partial rows of dweight and overlap fewer reads with their own reductions.
int rms_norm_grad_blocks(int64_t tokens) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(512, (tokens + 3) / 4));
}

hipError_t launch_rms_norm_grad(const NormGradLaunch& L, hipStream_t st) {
  if (L.tokens > 0) {
    if (L.bf16) L.vec ? bwd_launch<Bf16, true>(L, st) : bwd_launch<Bf16, false>(L, st);
    else L.vec ? bwd_launch<float, true>(L, st) : bwd_launch<float, false>(L, st);
  }
  if (L.dw) hipLaunchKernelGGL(norm_dw, dim3((L.dim + 63) / 64), dim3(1024), 0, st, L);
  return hipGetLastError();
}

}  // namespace muon

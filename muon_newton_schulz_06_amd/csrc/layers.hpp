// Launch descriptors and device helpers of the layer operators (embedding,
// RMS norm, gated feed-forward block).  Descriptors are passed by value.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// ----- embedding -------------------------------------------------------------
struct EmbedLaunch {
  const void* ids;
  int32_t id64;
  int32_t bf16;
  int64_t tokens, vocab, dim;
  const void* weight;
  int64_t ldw;
  void* out;
  int64_t ldo;
  float scale;
  int32_t vec;  // 16-byte aligned rows of whole 16-byte chunks
};
hipError_t launch_embedding(const EmbedLaunch& L, hipStream_t st);

// Positions per piece of a long run of equal ids: a run's sum is a chain of at
// most two pieces' rows and its whole pieces, and each piece costs an fp32 row.
constexpr int kEmbedPiece = 16;
// Tokens sorted by one workgroup in shared memory.
constexpr int64_t kEmbedSmallSort = 16384;
// Tokens per workgroup and digit bits of the sort in device memory.
constexpr int kEmbedSortBlock = 4096;
constexpr int kEmbedSortBits = 8;

struct EmbedGradLaunch {
  const void* ids;
  int32_t id64;
  int32_t dyBf16, dwBf16, accumulate;
  int64_t tokens, vocab, dim;
  const void* dy;
  int64_t ldy;
  void* dw;
  int64_t ldw;
  float scale;
  int32_t vec;       // dy rows are whole aligned 16-byte chunks
  int32_t vecw;      // so are dweight's
  int64_t zeroRows;  // rows zeroed before the pieces' launch (set by the launcher)
  uint32_t* key[2];  // sorted ids (vocab: none), ping-pong
  uint32_t* idx[2];  // their token positions
  uint32_t* counts;  // digit counts of the device-memory sort
  float* pieces;     // sums of whole pieces of long runs, dim floats each
};
hipError_t launch_embedding_grad(const EmbedGradLaunch& L, hipStream_t st);

// ----- RMS norm --------------------------------------------------------------
struct NormFwdLaunch {
  const void* x;
  const void* res;
  const void* w;
  void* y;
  void* sum;
  float* rstd;
  int64_t ldx, ldr, ldy, lds;
  int64_t tokens, dim;
  float eps;
  int32_t bf16, wBf16, vec;
};
hipError_t launch_rms_norm(const NormFwdLaunch& L, hipStream_t st);

struct NormGradLaunch {
  const void* dy;
  const void* s;
  const void* w;
  const void* dsum;
  const float* rstd;
  void* dx;
  void* dw;
  float* part;  // blocks × dim partial sums of dweight
  int64_t ldy, lds, ldd, ldx;
  int64_t tokens, dim;
  int32_t blocks;
  int32_t bf16, wBf16, vec, accumulate;
};
// Workgroups (and rows of partial sums) of the backward pass.
int rms_norm_grad_blocks(int64_t tokens);
hipError_t launch_rms_norm_grad(const NormGradLaunch& L, hipStream_t st);

// ----- gated feed-forward block ----------------------------------------------
// C = A·Bᵀ over one or two ranges of k.  An operand is k-contiguous (element
// (row, k) at p[row·ld + k]) or row-contiguous (p[k·ld + row]); which one is a
// property of the launch.
enum FfnEpi : int32_t {
  FFN_GLU = 0,    // B holds w_gate and w_up: h = act(g)·u, optional a, b
  FFN_BACK = 1,   // dh → dg = dh·a, du = dh·b
  FFN_STORE = 2,  // C ← acc (+ C)
};

struct FfnProb {
  const void* A[2];  // per k range
  const void* B[2];  // per k range (FFN_GLU: w_gate, w_up over the one range)
  int64_t lda, ldb[2];
  int32_t M, N;
  int32_t K[2];
  // elements of a row-contiguous operand's rows (tile16: a multiple of 8)
  int32_t extA, extB;
  void* C;
  int64_t ldc;
  int32_t vecC;  // four consecutive elements of C are one aligned access
  // where the k splits leave their fp32 sums, [split][M][partN] (null: one
  // split, C is written); partN: N rounded up to 4, for FFN_GLU twice that
  float* part;
  int64_t partN;
};

struct FfnLaunch {
  FfnProb prob[3];
  int32_t tiles[4];  // first tile of each problem, and the total
  int32_t nprob;
  int32_t act;
  int32_t outBf16, accumulate;
  // FFN_GLU: a, b (null: not wanted), C is h; FFN_BACK: reads them, C is dg, du
  // (rows of 2·ldh).  Rows of a, b: fp32 2·ldh values, a then b; bf16 3·ldh
  // 16-bit pieces, the upper halves of a, those of b, the bytes below of both
  void* ab;
  int64_t ldh;  // hidden rounded up to 8: row length of h and of each half
  int32_t splitTiles;  // k-tiles of 32 per split (a multiple of four for bf16 tiles)
};
hipError_t launch_ffn16_glu(int tile, const FfnLaunch& L, hipStream_t st);
hipError_t launch_ffn16_back(int tile, const FfnLaunch& L, hipStream_t st);
hipError_t launch_ffn16_store(int tile, bool aRowContig, bool bRowContig, const FfnLaunch& L,
                              hipStream_t st);

// The few-token forward products (tokens ≤ kFfnFew), any alignment.
constexpr int64_t kFfnFew = 64;
hipError_t launch_ffn_few(int epi, bool bf16, int splits, const FfnLaunch& L, hipStream_t st);

// Sums of the splits' results, with the products' epilogue.
hipError_t launch_ffn_join(int epi, bool bf16, int splits, const FfnLaunch& L, hipStream_t st);

// Aligned, zero-padded copies of a call's bf16 operands.
struct FfnPack {
  const void* src;
  int64_t ld, rows, cols;
  void* dst;
  int64_t ldo;
};
struct FfnPacks {
  FfnPack p[5];
  int32_t n;
};
hipError_t launch_ffn_pack(const FfnPacks& K, hipStream_t st);

hipError_t launch_ffn_tile32(int epi, int tileM, bool aRowContig, bool bRowContig, const FfnLaunch& L,
                             hipStream_t st);

// ----- device helpers --------------------------------------------------------
typedef float lf32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t lu32x4 __attribute__((ext_vector_type(4)));

struct Bf16 {
  uint16_t v;
};

__device__ __forceinline__ float l_bf16_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Round to nearest even (the hardware's conversion; NaN stays NaN): one value,
// and two as the halves of a dword.
typedef __bf16 lbf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t l_f32_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t l_f32_bf16x2(float lo, float hi) {
  const lbf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

template <typename T> struct LType;
template <> struct LType<float> {
  static constexpr int kVec = 4;  // elements of a 16-byte chunk
  static __device__ __forceinline__ float get(const void* p, int64_t e) { return ((const float*)p)[e]; }
  static __device__ __forceinline__ void put(void* p, int64_t e, float v) { ((float*)p)[e] = v; }
};
template <> struct LType<Bf16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(const void* p, int64_t e) {
    return l_bf16_f32(((const uint16_t*)p)[e]);
  }
  static __device__ __forceinline__ void put(void* p, int64_t e, float v) {
    ((uint16_t*)p)[e] = (uint16_t)l_f32_bf16(v);
  }
};

// A raw 16-byte chunk widened to fp32.
template <typename T> __device__ __forceinline__ void l_widen(lu32x4 c, float (&v)[LType<T>::kVec]) {
  if constexpr (LType<T>::kVec == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(c[i] << 16);
      v[2 * i + 1] = __uint_as_float(c[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(c[i]);
  }
}

template <typename T> __device__ __forceinline__ lu32x4 l_narrow(const float (&v)[LType<T>::kVec]) {
  lu32x4 c;
  if constexpr (LType<T>::kVec == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = l_f32_bf16x2(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(v[i]);
  }
  return c;
}

// Elements [e, e + kVec) of a row of n elements as a chunk: one 16-byte access
// when VEC, else one of any alignment where the chunk is whole and one access
// per element that exists at the row's end (others 0).
template <typename T, bool VEC>
__device__ __forceinline__ lu32x4 l_load(const void* row, int64_t e, int64_t n) {
  if constexpr (VEC) {
    return *(const lu32x4*)((const char*)row + e * (16 / LType<T>::kVec));
  } else {
    lu32x4 c = {0u, 0u, 0u, 0u};
    if (e + LType<T>::kVec <= n) {
      __builtin_memcpy(&c, (const char*)row + e * (16 / LType<T>::kVec), 16);
    } else if constexpr (LType<T>::kVec == 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < n) c[i / 2] |= (uint32_t)((const uint16_t*)row)[e + i] << (16 * (i & 1));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < n) c[i] = ((const uint32_t*)row)[e + i];
    }
    return c;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void l_store(void* row, int64_t e, int64_t n, lu32x4 c) {
  if constexpr (VEC) {
    *(lu32x4*)((char*)row + e * (16 / LType<T>::kVec)) = c;
  } else if (e + LType<T>::kVec <= n) {
    __builtin_memcpy((char*)row + e * (16 / LType<T>::kVec), &c, 16);
  } else if constexpr (LType<T>::kVec == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < n) ((uint16_t*)row)[e + i] = (uint16_t)(c[i / 2] >> (16 * (i & 1)));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < n) ((uint32_t*)row)[e + i] = c[i];
  }
}

__device__ __forceinline__ float l_wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The upper 24 bits of an fp32 value (sign, its 8 exponent bits, 15 mantissa
// bits): the whole range of fp32, infinities and NaN (arithmetic makes quiet
// ones, whose mark is the top mantissa bit) included.  Cut off, not rounded:
// the error, below 2^-15 of a normal value, is far below that of the rounding
// to bf16 that follows, and a byte selection is all it takes either way.
// Columns c, c + 1 of two values a, b are kept in three dwords: the upper
// halves of a, those of b, and the bytes below (a, b of c, then of c + 1).
__device__ __forceinline__ uint32_t l_upper2(float v0, float v1) {
  return __builtin_amdgcn_perm(__float_as_uint(v1), __float_as_uint(v0), 0x07060302u);
}
__device__ __forceinline__ uint32_t l_lower2(float a0, float b0, float a1, float b1) {
  return __builtin_amdgcn_perm(__float_as_uint(b0), __float_as_uint(a0), 0x0c0c0501u) |
         __builtin_amdgcn_perm(__float_as_uint(b1), __float_as_uint(a1), 0x05010c0cu);
}
// Value V (0: a, 1: b) of column c + H from its dword of upper halves and the
// dword of lower bytes.
template <int V, int H> __device__ __forceinline__ float l_join24(uint32_t upper, uint32_t lower) {
  return __uint_as_float(
      __builtin_amdgcn_perm(upper, lower, (H ? 0x07060000u : 0x05040000u) | (2 * H + V) << 8 | 0x0cu));
}

}  // namespace muon

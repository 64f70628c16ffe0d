// Tiles of the attention kernels: 32×32 MFMA products whose operands lie in
// LDS rows or come from the result of another product.
//
// Results of a 32×32 product: lane l holds column l % 32, rows
// 8·(i / 4) + 4·(l / 32) + i % 4 in its 16 registers.  An operand gives lane l
// the 16 bytes of row l % 32 that its half l / 32 is due at a step of the
// contraction: 8 bf16 (a step is 16 long) or 4 fp32 (8 long, four products of
// 2).  Which of the step's indexes a half holds is free as long as both
// operands agree, so a result's registers serve as the next product's operand
// as they are, its rows being the contraction: a step takes rows
// 16·s + 4·half + {0…3, 8…11} (bf16) or 8·s + 4·half + {0…3} (fp32).
#pragma once

#include <type_traits>

#include "attention.hpp"
#include "dma.hpp"
#include "layers.hpp"

namespace muon {

typedef float af32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 abf16x8 __attribute__((ext_vector_type(8)));
typedef short as16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) as16x4* a_lds_s4;
typedef __attribute__((address_space(3))) const lu32x4* a_lds_u4;
typedef __attribute__((address_space(3))) const uint32_t* a_lds_u1;

template <typename T> struct AT {
  static constexpr int kBytes = 16 / LType<T>::kVec;
  static constexpr int kStep = 2 * LType<T>::kVec;  // contraction of a step
  static constexpr int kSteps32 = 32 / kStep;       // steps over the rows of a result
};

template <int B, int E, typename F> __device__ __forceinline__ void a_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    a_for<B + 1, E>(f);
  }
}

__device__ __forceinline__ uint32_t a_lds(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

template <typename T> __device__ __forceinline__ af32x16 a_mma(lu32x4 a, lu32x4 b, af32x16 c) {
  if constexpr (AT<T>::kBytes == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(abf16x8, a), __builtin_bit_cast(abf16x8, b), c,
                                                   0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

// sum + the eight bf16 of an operand.
__device__ __forceinline__ float a_operand_sum(const lu32x4& op, float sum) {
  typedef __bf16 Two __attribute__((ext_vector_type(2)));
  const Two one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = op[i];  // (a bit_cast of a vector's element itself takes the vector's first)
    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(Two, two), one, sum, false);
  }
  return sum;
}

// Infinities and NaN in tiles.  0 times one of them is NaN, so where a
// probability of 0 stands for "not seen" they have to stay out of the product.
// The running largest magnitude of chunks (bf16: in either half of the word), and
// whether it is one of them.
template <typename T> __device__ __forceinline__ uint32_t a_top(lu32x4 v, uint32_t top) {
  typedef uint16_t Two __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = v[i] & (AT<T>::kBytes == 2 ? 0x7fff7fffu : 0x7fffffffu);
    if constexpr (AT<T>::kBytes == 2)
      top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(Two, m), __builtin_bit_cast(Two, top)));
    else
      top = max(top, m);
  }
  return top;
}
template <typename T> __device__ __forceinline__ bool a_odd(uint32_t top) {
  return top >= 0x7f800000u || (AT<T>::kBytes == 2 && (top & 0xffffu) >= 0x7f80u);
}
// A chunk with zeros in their place.
template <typename T> __device__ __forceinline__ lu32x4 a_finite(lu32x4 v) {
  lu32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t hi = (v[i] & 0x7f800000u) == 0x7f800000u ? 0u : AT<T>::kBytes == 2 ? 0xffff0000u : 0xffffffffu;
    r[i] = v[i] & (AT<T>::kBytes == 2 ? hi | ((v[i] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) : hi);
  }
  return r;
}
// Operands whose products overflow: ±2^100 where a chunk has an infinity of the
// sign or a NaN; 2^100 at the first n indexes of a lane's part of a step (counted
// over both halves: 4·half is taken off n by the caller).
template <typename T> __device__ __forceinline__ lu32x4 a_odd_of(lu32x4 v, int negative) {
  constexpr bool two = AT<T>::kBytes == 2;
  lu32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = 0;
#pragma unroll
    for (int h = 0; h < (two ? 2 : 1); ++h) {
      const uint32_t x = two && h == 0 ? v[i] << 16 : two ? v[i] & 0xffff0000u : v[i], m = x & 0x7fffffffu;
      const bool odd = m > 0x7f800000u || x == (negative ? 0xff800000u : 0x7f800000u);
      const uint32_t big = odd ? negative ? 0xf1800000u : 0x71800000u : 0u;
      r[i] |= two && h == 0 ? big >> 16 : big;
    }
  }
  return r;
}
template <typename T> __device__ __forceinline__ lu32x4 a_below(int n) {
  lu32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (AT<T>::kBytes == 2) {
      const int first = 8 * (i >> 1) + 2 * (i & 1);
      r[i] = (first < n ? 0x7180u : 0u) | (first + 1 < n ? 0x71800000u : 0u);
    } else {
      r[i] = i < n ? 0x71800000u : 0u;
    }
  }
  return r;
}
// What is not finite of a row's log-sums and δ: bits 0 and 1 the maps' log-sums (that
// of an odd q is not), bit 2 anything.
__device__ __forceinline__ uint32_t a_bad_row(float l1, float l2, float d1, float d2) {
  auto odd = [](float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; };
  const uint32_t l = (odd(l1) ? 1u : 0u) | (odd(l2) ? 2u : 0u);
  return l | (l || odd(d1) || odd(d2) ? 4u : 0u);
}
// Every wave is here, and its LDS accesses are done (loads into LDS may be on their way).
__device__ __forceinline__ void a_meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Step s of a result as an operand.
template <typename T> __device__ __forceinline__ lu32x4 a_operand(const float (&p)[16], int s) {
  lu32x4 r;
  if constexpr (AT<T>::kBytes == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = l_f32_bf16x2(p[8 * s + 2 * i], p[8 * s + 2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(p[4 * s + i]);
  }
  return r;
}

// LDS tiles of rows of RB bytes; 16-byte chunk c of row r lies at c ^ a_swz(r).
// LDS has 64 banks, 256 bytes; 16 lanes of a 16-byte read are served at a time.
// Row reads take the same chunk of 32 rows: sixteen rows that differ in their
// low four bits (whichever of bits 2 to 4 the hardware's groups vary) fall into
// different chunks of 256 bytes.  Column reads take 64 bytes (bf16) of four
// consecutive rows: those differ in which 64 bytes of 256 they fall into.
// (Measured: without bit 3 a row read took 8 cycles, not 4.)
template <int RB> __device__ __forceinline__ int a_swz(int r) {
  if constexpr (RB == 128) return (r >> 1 & 1) << 2 | (r >> 2 & 1) << 1 | (r >> 3 & 1);
  else return (r & 1) << 2 | (r >> 1 & 1) << 3 | (r >> 2 & 1) | (r >> 3 & 1) << 1;
}

// A lane's reads of row operands: rows 32·n + lane % 32, step c.
template <int RB> struct RowReader {
  uint32_t at;
  // offset: bytes added to every tile's address, a multiple of RB
  __device__ __forceinline__ RowReader(int lane, uint32_t offset = 0) {
    const int r = lane & 31;
    at = r * RB + (((lane >> 5) ^ a_swz<RB>(r)) << 4) + offset;
  }
  // tile: LDS address of row 32·n (a multiple of RB); c a constant
  __device__ __forceinline__ lu32x4 get(uint32_t tile, int c) const {
    return *(a_lds_u4)(uintptr_t)((at ^ (c << 5)) + tile);
  }
  __device__ __forceinline__ void put(uint32_t tile, int c, lu32x4 v) const {
    *(__attribute__((address_space(3))) lu32x4*)(uintptr_t)((at ^ (c << 5)) + tile) = v;
  }
};

// A lane's reads of column operands: columns 32·n + lane % 32, the step's rows.
template <typename T, int RB> struct ColReader {
  uint32_t at;
  __device__ __forceinline__ ColReader(int lane) {
    if constexpr (AT<T>::kBytes == 2) {
      // transposing reads: 16 lanes point at four rows of four values each and
      // receive one column each
      const int j = lane & 15, r = 4 * (lane >> 5) + (j >> 2);
      at = r * RB + (((2 * (lane >> 4 & 1) + (j >> 1 & 1)) ^ a_swz<RB>(r)) << 4) + (j & 1) * 8;
    } else {
      // rows 8·s + 4·half + i: i's part of the address follows in get
      const int r = 4 * (lane >> 5);
      at = r * RB + ((((lane & 31) >> 2) ^ a_swz<RB>(r)) << 4) + (lane & 3) * 4;
    }
  }
  // tile: LDS address of the tile's first row; step s of its rows; n a constant
  __device__ __forceinline__ lu32x4 get(uint32_t tile, int s, int n) const {
    if constexpr (AT<T>::kBytes == 2) {
      const uint32_t a = (at ^ (n << 6)) + s * (16 * RB) + tile;
      const uint32_t b = (at ^ (n << 6) ^ (a_swz<RB>(8) << 4)) + (s * 16 + 8) * RB + tile;
      const as16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((a_lds_s4)(uintptr_t)a);
      const as16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((a_lds_s4)(uintptr_t)b);
      return __builtin_bit_cast(lu32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      lu32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *(a_lds_u1)(uintptr_t)((at ^ (n << 7) ^ (a_swz<RB>((s & 1) * 8 + i) << 4)) + (s * 8 + i) * RB + tile);
      return v;
    }
  }
};

// Copies a tile of ROWS rows of RB bytes into LDS with 16-byte buffer loads of
// NW waves; rows past `left` and bytes past `bytes` of a row arrive as zeros.
template <int RB, int ROWS, int NW> struct TileLoader {
  static constexpr int kChunks = RB / 16, kRowsPer = 64 / kChunks, N = ROWS / (kRowsPer * NW);
  static_assert(N * kRowsPer * NW == ROWS, "whole loads");
  uint32_t off[N];
  int row0, wave;
  __device__ __forceinline__ void init(int lane, int w, int64_t ldBytes, int bytes) {
    wave = w;
    row0 = w * N * kRowsPer + lane / kChunks;
#pragma unroll
    for (int p = 0; p < N; ++p) {
      const int r = row0 + p * kRowsPer, c = (lane % kChunks) ^ a_swz<RB>(r);
      off[p] = c * 16 < bytes ? (uint32_t)(r * ldBytes) + c * 16 : kFfnNowhere;
    }
  }
  // a tile of which every row is there
  __device__ __forceinline__ void issue(const char* base, uint32_t dst) const {
    const fi32x4 buf = f_buffer((uint64_t)base);
#pragma unroll
    for (int p = 0; p < N; ++p) f_dma16(__builtin_amdgcn_readfirstlane(dst + (wave * N + p) * 1024), off[p], buf);
  }
  __device__ __forceinline__ void issue(const char* base, int64_t left, uint32_t dst) const {
    const fi32x4 buf = f_buffer((uint64_t)base);
#pragma unroll
    for (int p = 0; p < N; ++p)
      f_dma16(__builtin_amdgcn_readfirstlane(dst + (wave * N + p) * 1024),
              row0 + p * kRowsPer < left ? off[p] : kFfnNowhere, buf);
  }
};

// The tiles of one block that a workgroup runs: begin … end − 1.
struct Piece {
  int combo, tok, n, inside, at;
  int64_t begin, end;
  int64_t slot;  // where its sums go to be joined; −1: the block is its own
};

// A workgroup's stretch of all combos' tiles, in the list's order, or (streams
// = 0) the block of its number.
struct Stretch {
  int64_t each, total, per, pos, stop;  // tiles of a combo, all, of a stretch; this one
  int64_t w;
  int count;
  __device__ __forceinline__ Stretch(const AttnRuns& R, int combos, int64_t number) : w(number) {
    pos = 0;
    stop = 1;
    if (!R.streams) return;
    count = *R.list.count;
    each = R.cum[count];
    total = each * combos;
    per = max((total + R.streams - 1) / R.streams, (int64_t)R.least);
    pos = min(w * per, total);
    stop = min(pos + per, total);
  }
  // the block of a combo's tile
  __device__ __forceinline__ int find(const AttnRuns& R, int64_t tile) const {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (R.cum[mid] <= tile) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
  // at: the row or key the workgroup's block begins at, without a list
  __device__ __forceinline__ bool next(const AttnRuns& R, int combos, int at, Piece& p) {
    if (pos >= stop) return false;
    if (!R.streams) {
      p = Piece{(int)blockIdx.x % combos, 0, 0, 1, at, 0, int64_t(1) << 40, -1};
      if (R.list.blocks) {  // from the last one: in every sequence the rows that see most keys first
        const int id = *R.list.count - 1 - (int)blockIdx.x / combos;
        if (id < 0) return false;
        const AttnBlock B = R.list.blocks[id];
        p.tok = B.tok;
        p.n = B.n;
        p.inside = B.nk > 0;
        p.at = B.at;
      }
      pos = stop;
      return true;
    }
    p.combo = (int)(pos / each);
    const int64_t tile = pos - p.combo * each;
    const int b = find(R, tile);
    const AttnBlock B = R.list.blocks[b];
    p.tok = B.tok;
    p.n = B.n;
    p.inside = B.nk > 0;
    p.at = B.at;
    const int64_t from = R.cum[b], to = R.cum[b + 1], n = min(stop - pos, to - tile);
    p.begin = tile - from;
    p.end = p.begin + n;
    p.slot = n == to - from ? -1 : 2 * w + (p.begin == 0);
    pos += n;
    return true;
  }
};

// Every load into LDS has landed and every wave is here.
__device__ __forceinline__ void a_landed() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The value and its counterpart of the lane 32 further on (or back).
__device__ __forceinline__ float a_half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ uint32_t a_half_max(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(r[0], r[1]);
}
__device__ __forceinline__ float a_half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float a_exp2(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float a_log2(float v) { return __builtin_amdgcn_logf(v); }

constexpr float kNegInf = -__builtin_inff();

typedef uint32_t lu32x2 __attribute__((ext_vector_type(2)));

// Values as 16-bit whole multiples of a unit, their largest magnitude / 32767
// (given as the bits of that magnitude): off by at most one unit.  Rows with an
// infinity or NaN have the unit NaN, rows of zeros (or subnormal values) the unit 0.
struct Whole {
  float unit, inv;  // inv: to [−1, 1]
  __device__ __forceinline__ explicit Whole(uint32_t top) {
    const float f = __uint_as_float(top);
    const bool some = f > 2e-38f, finite = top < 0x7f800000u;
    inv = some && finite ? 1.f / f : 0.f;
    unit = !finite ? __builtin_nanf("") : some ? f / 32767.f : 0.f;
  }
};
__device__ __forceinline__ uint32_t a_pair_whole(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_i16(a, b));
}

// Values of one row and the 32 columns of a result's transpose (lane: row
// l % 32, registers: columns 8·(i / 4) + 4·half + i % 4) as stores of four,
// or, for bf16 with 16-byte stores, of eight columns.
// WHOLE (bf16): of values in [−1, 1] the multiples of 1/32767 instead.
template <typename T, bool WHOLE = false>
__device__ __forceinline__ void a_store_row(char* row, const float (&v)[16], int col0, int width, bool vec, bool valid,
                                            int half) {
  auto pair = [](float a, float b) { return WHOLE ? a_pair_whole(a, b) : l_f32_bf16x2(a, b); };
  if constexpr (AT<T>::kBytes == 2) {
    if (vec) {  // the halves exchange groups of four columns, so that each lane has eight in a row
#pragma unroll
      for (int g = 0; g < 4; g += 2) {
        uint32_t x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const auto s = __builtin_amdgcn_permlane32_swap(pair(v[4 * g + 2 * i], v[4 * g + 2 * i + 1]),
                                                          pair(v[4 * g + 4 + 2 * i], v[4 * g + 5 + 2 * i]), false, false);
          x[i] = s[0];
          y[i] = s[1];
        }
        const int c = col0 + 8 * (g + half);
        if (valid && c < width) *(lu32x4*)(row + c * 2) = lu32x4{x[0], x[1], y[0], y[1]};
      }
      return;
    }
  } else {
    if (vec) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = col0 + 8 * g + 4 * half;
        if (valid && c < width) *(lf32x4*)(row + c * 4) = lf32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = col0 + 8 * (i >> 2) + 4 * half + (i & 3);
    if (valid && c < width) LType<T>::put(row, c, v[i]);
  }
}

}  // namespace muon

// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[t] = scale·W[id_t], up to four 16-byte chunks per lane in flight;
// HBM-bound (16384 × 3584 bf16 from 131072 rows: 35 µs, 6.7 TB/s read and
// written, frequent rows coming from the caches).
//
// Gradient: dW[v] = scale·Σ_{t: id_t = v} dy[t] without float atomics (their
// order, and so the last bits, would change from run to run):
//   1. a stable radix sort of (id, t) by id, while dweight is zeroed;
//   2. pieces: the sorted list is cut every kEmbedPiece positions; a piece
//      that lies wholly inside one run of equal ids is summed to an fp32 row
//      in the workspace, so that no run is summed by one lane group alone;
//   3. one lane group per run: the rows before its first whole piece, the
//      pieces' sums, the rows after the last one, in that order.
// HBM-bound for large vocabularies, whose bytes are mostly zero rows: 16384 ×
// 3584 bf16 tokens into 131072 rows take 65 + 145 + 59 µs (sort, pieces, runs,
// the first two beside 940 MB of zeros), about 4 TB/s; a run is a chain of
// dependent reads, which bounds small calls (4093 × 1023 fp32: 15 + 29 + 22).
// Ids outside [0, vocab) sort to the end as the key `vocab` and are skipped.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layers.hpp"

namespace muon {
namespace {

__device__ __forceinline__ int64_t load_id(const void* ids, int id64, int64_t t) {
  return id64 ? ((const int64_t*)ids)[t] : (int64_t)((const int32_t*)ids)[t];
}

// ----- lookup ----------------------------------------------------------------
// A group of `lanes` lanes (a power of two) serves one token; it takes up to
// four chunks per lane and slice of the row (blockIdx.y).
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void embedding_kernel(const EmbedLaunch L, int lanes, int shift) {
  constexpr int V = LType<T>::kVec;
  const int g = threadIdx.x >> shift, l = threadIdx.x & (lanes - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 >> shift) + g;
  if (t >= L.tokens) return;
  const int64_t id = load_id(L.ids, L.id64, t);
  const bool ok = id >= 0 && id < L.vocab;
  constexpr int E = 16 / V;  // bytes per element
  const char* src = (const char*)L.weight + (ok ? id : 0) * L.ldw * E;
  char* dst = (char*)L.out + t * L.ldo * E;
  const int64_t c0 = (int64_t)blockIdx.y * lanes * 4 + l;
  lu32x4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t e = (c0 + i * lanes) * V;
    if (e < L.dim && ok) v[i] = l_load<T, VEC>(src, e, L.dim);
    else v[i] = lu32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t e = (c0 + i * lanes) * V;
    if (e < L.dim) {
      float f[V];
      l_widen<T>(v[i], f);
      if (ok) {
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] *= L.scale;
      }
      l_store<T, VEC>(dst, e, L.dim, l_narrow<T>(f));
    }
  }
}

// Zeros rows [v0, v1) of dweight by W waves, of which this is wave w: pieces of
// 8 KiB of a contiguous dweight in turn, whatever its rows' alignment, else row
// by row.  Non-temporal stores: with ordinary ones the zeros filled the
// last-level cache and their write-back ran into the sums (sums 76 -> 40 µs,
// sort beside them 67 -> 47 µs for 131072×3584 bf16).
__device__ __forceinline__ void zero_rows(const EmbedGradLaunch& L, int64_t v0, int64_t v1, int64_t w, int64_t W);

// ----- sort ------------------------------------------------------------------
__device__ __forceinline__ uint32_t sort_key(const EmbedGradLaunch& L, int64_t t) {
  const int64_t id = load_id(L.ids, L.id64, t);
  return id >= 0 && id < L.vocab ? (uint32_t)id : (uint32_t)L.vocab;
}

// Lanes of the wave with the same digit, among the active ones of `in`.
template <int BITS>
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t in) {
  uint64_t m = in;
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool bit = (d >> b) & 1u;
    const uint64_t set = __ballot(bit);
    m &= bit ? set : ~set;
  }
  return m;
}

// Orders a wave's shared-memory accesses before it, of all lanes, ahead of
// those after it.  No instruction: the LDS serves a wave in order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One stable counting pass over a workgroup's items, held in registers in
// wave order: wave w's items are consecutive, ITEMS rounds of 64 lanes.
// cnt[digit·WAVES + wave] must be zero on entry and holds the wave's digit
// counts afterwards; rank[i] is the item's rank among its wave's equal digits.
template <int BITS, int ITEMS, int WAVES>
__device__ __forceinline__ void rank_items(const uint32_t (&key)[ITEMS], const bool (&have)[ITEMS],
                                           int sh, uint32_t* cnt, int wave, int lane,
                                           uint32_t (&rank)[ITEMS]) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t d = (key[i] >> sh) & ((1u << BITS) - 1u);
    const uint64_t in = __ballot(have[i]);
    const uint64_t m = same_digit<BITS>(d, in);
    uint32_t* c = cnt + d * WAVES + wave;
    const uint32_t before = have[i] ? *c : 0u;
    rank[i] = before + (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
    // every lane has read; the last lane of each digit stores the new count,
    // which the next round reads
    wave_order();
    if (have[i] && (m >> lane) == 1ull) *c = rank[i] + 1u;
    wave_order();
  }
}

// Exclusive scan of n counts in shared memory by the whole workgroup (n a
// multiple of the thread count).
template <int NT>
__device__ __forceinline__ void scan_counts(uint32_t* cnt, int n, uint32_t* wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = n / NT;
  uint32_t s = 0;
  for (int i = 0; i < per; ++i) s += cnt[tid * per + i];
  uint32_t inc = s;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < wave; ++w) base += wsum[w];
  uint32_t run = base + inc - s;
  for (int i = 0; i < per; ++i) {
    const uint32_t c = cnt[tid * per + i];
    cnt[tid * per + i] = run;
    run += c;
  }
  __syncthreads();
}

// The whole sort of up to kEmbedSmallSort tokens in one workgroup: keys live
// in registers, each pass permutes them through shared memory.  9-bit digits,
// so a vocabulary of up to 2^18 − 1 takes two passes.  The launch's other
// workgroups write zeros of dweight meanwhile (rows of ids that occur are
// written again by the sums: at most tokens · dim elements more).
template <int ITEMS>
__global__ __launch_bounds__(1024) void embed_sort_small(const EmbedGradLaunch L, int passes) {
  constexpr int BITS = 9, WAVES = 16, BINS = 1 << BITS;
  __shared__ uint32_t cnt[BINS * WAVES];
  __shared__ uint32_t skey[ITEMS * 1024];
  __shared__ uint16_t sidx[ITEMS * 1024];
  __shared__ uint32_t wsum[WAVES];
  static_assert(ITEMS * 1024 <= 65536, "token positions are kept in 16 bits");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x > 0) {
    zero_rows(L, 0, L.zeroRows, (int64_t)(blockIdx.x - 1) * 16 + wave, (int64_t)(gridDim.x - 1) * 16);
    return;
  }
  const int n = (int)L.tokens;
  uint32_t key[ITEMS], idx[ITEMS], rank[ITEMS];
  bool have[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int p = wave * (ITEMS * 64) + i * 64 + lane;
    have[i] = p < n;
    key[i] = have[i] ? sort_key(L, p) : 0u;
    idx[i] = p;
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int sh = pass * BITS;
    for (int i = tid; i < BINS * WAVES; i += 1024) cnt[i] = 0u;
    __syncthreads();
    rank_items<BITS, ITEMS, WAVES>(key, have, sh, cnt, wave, lane, rank);
    __syncthreads();
    scan_counts<1024>(cnt, BINS * WAVES, wsum);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (have[i]) {
        const uint32_t to = cnt[((key[i] >> sh) & (BINS - 1u)) * WAVES + wave] + rank[i];
        skey[to] = key[i];
        sidx[to] = (uint16_t)idx[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int p = wave * (ITEMS * 64) + i * 64 + lane;
      if (have[i]) {
        key[i] = skey[p];
        idx[i] = sidx[p];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int p = wave * (ITEMS * 64) + i * 64 + lane;
    if (have[i]) {
      L.key[0][p] = key[i];
      L.idx[0][p] = idx[i];
    }
  }
}

// Sort in device memory, one 8-bit digit per pass: counts per workgroup, one
// scan over (digit, workgroup), stable scatter.
constexpr int kSortItems = kEmbedSortBlock / 256;
constexpr int kSortBins = 1 << kEmbedSortBits;

__device__ __forceinline__ void load_items(const EmbedGradLaunch& L, int pass, uint32_t (&key)[kSortItems],
                                           uint32_t (&idx)[kSortItems], bool (&have)[kSortItems]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t b0 = (int64_t)blockIdx.x * kEmbedSortBlock + wave * (kSortItems * 64) + lane;
  const int from = (pass + 1) & 1;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const int64_t p = b0 + i * 64;
    have[i] = p < L.tokens;
    key[i] = idx[i] = 0u;
    if (have[i]) {
      key[i] = pass == 0 ? sort_key(L, p) : L.key[from][p];
      idx[i] = pass == 0 ? (uint32_t)p : L.idx[from][p];
    }
  }
}

__global__ __launch_bounds__(256) void embed_sort_count(const EmbedGradLaunch L, int pass) {
  __shared__ uint32_t cnt[kSortBins * 4];
  uint32_t key[kSortItems], idx[kSortItems], rank[kSortItems];
  bool have[kSortItems];
  for (int i = threadIdx.x; i < kSortBins * 4; i += 256) cnt[i] = 0u;
  load_items(L, pass, key, idx, have);
  __syncthreads();
  rank_items<kEmbedSortBits, kSortItems, 4>(key, have, pass * kEmbedSortBits, cnt, threadIdx.x >> 6,
                                            threadIdx.x & 63, rank);
  __syncthreads();
  const int d = threadIdx.x;
  L.counts[(int64_t)d * gridDim.x + blockIdx.x] = cnt[4 * d] + cnt[4 * d + 1] + cnt[4 * d + 2] + cnt[4 * d + 3];
}

__global__ __launch_bounds__(1024) void embed_sort_scan(uint32_t* counts, int64_t n) {
  __shared__ uint32_t wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t per = (n + 1023) / 1024, lo = min(n, tid * per), hi = min(n, lo + per);
  uint32_t s = 0;
  for (int64_t i = lo; i < hi; ++i) s += counts[i];
  uint32_t inc = s;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  uint32_t run = inc - s;
  for (int w = 0; w < wave; ++w) run += wsum[w];
  for (int64_t i = lo; i < hi; ++i) {
    const uint32_t c = counts[i];
    counts[i] = run;
    run += c;
  }
}

__global__ __launch_bounds__(256) void embed_sort_scatter(const EmbedGradLaunch L, int pass) {
  __shared__ uint32_t cnt[kSortBins * 4];
  uint32_t key[kSortItems], idx[kSortItems], rank[kSortItems];
  bool have[kSortItems];
  for (int i = threadIdx.x; i < kSortBins * 4; i += 256) cnt[i] = 0u;
  load_items(L, pass, key, idx, have);
  __syncthreads();
  const int sh = pass * kEmbedSortBits, wave = threadIdx.x >> 6;
  rank_items<kEmbedSortBits, kSortItems, 4>(key, have, sh, cnt, wave, threadIdx.x & 63, rank);
  __syncthreads();
  const int d = threadIdx.x;
  uint32_t run = L.counts[(int64_t)d * gridDim.x + blockIdx.x];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t c = cnt[4 * d + w];
    cnt[4 * d + w] = run;
    run += c;
  }
  __syncthreads();
  const int to = pass & 1;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    if (have[i]) {
      const uint32_t p = cnt[((key[i] >> sh) & (kSortBins - 1u)) * 4 + wave] + rank[i];
      L.key[to][p] = key[i];
      L.idx[to][p] = idx[i];
    }
  }
}

// ----- segmented sums --------------------------------------------------------
// A lane group adds the rows idx[p0 .. p0 + n) of dy at its columns, in order;
// the indices are read by the group's lanes at once and eight rows are in
// flight.  The group's lanes are active together.
template <typename T, bool VEC>
__device__ __forceinline__ void add_rows(const EmbedGradLaunch& L, const uint32_t* idx, int64_t p0, int n,
                                         int64_t e, int l, int lanes, float (&acc)[LType<T>::kVec]) {
  constexpr int V = LType<T>::kVec, E = 16 / V;
  const int first = (threadIdx.x & 63) - l;  // the group's first lane in the wave
  const bool in = e < L.dim;
  for (int base = 0; base < n; base += lanes) {
    const int cnt = min(lanes, n - base);
    const int mine = l < cnt ? (int)idx[p0 + base + l] : 0;
    int j = 0;
    auto batch = [&](auto nc) __attribute__((always_inline)) {
      constexpr int N = decltype(nc)::value;
      for (; j + N <= cnt; j += N) {
        lu32x4 c[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int64_t t = (uint32_t)__shfl(mine, first + j + i, 64);
          c[i] = lu32x4{0u, 0u, 0u, 0u};
          if (in) c[i] = l_load<T, VEC>((const char*)L.dy + t * L.ldy * E, e, L.dim);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float f[V];
          l_widen<T>(c[i], f);
#pragma unroll
          for (int k = 0; k < V; ++k) acc[k] += f[k];
        }
      }
    };
    batch(std::integral_constant<int, 8>{});
    batch(std::integral_constant<int, 2>{});
    batch(std::integral_constant<int, 1>{});
  }
}

// Sums of whole pieces inside one run.  One lane group per (piece, slice); the
// workgroups from sumBlocks on write the zeros the sort's launch left.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void embed_pieces(const EmbedGradLaunch L, const uint32_t* key,
                                                    const uint32_t* idx, int lanes, int shift, int slices,
                                                    int sumBlocks) {
  constexpr int V = LType<T>::kVec;
  if ((int)blockIdx.x >= sumBlocks) {
    zero_rows(L, L.zeroRows, L.vocab, (int64_t)(blockIdx.x - sumBlocks) * 4 + (threadIdx.x >> 6),
              (int64_t)(gridDim.x - sumBlocks) * 4);
    return;
  }
  const int g = threadIdx.x >> shift, l = threadIdx.x & (lanes - 1);
  const int64_t c = (int64_t)(blockIdx.x / slices) * (256 >> shift) + g;
  const int64_t p0 = c * kEmbedPiece;
  if (p0 + kEmbedPiece > L.tokens) return;
  const uint32_t k = key[p0];
  if (k != key[p0 + kEmbedPiece - 1] || k >= (uint32_t)L.vocab) return;
  const int64_t e = ((int64_t)(blockIdx.x % slices) * lanes + l) * V;
  float acc[V] = {};
  add_rows<T, VEC>(L, idx, p0, kEmbedPiece, e, l, lanes, acc);
  float* out = L.pieces + c * L.dim + e;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e + i < L.dim) out[i] = acc[i];
}

// Stores V values of a dweight row (adding to it when accumulating).
template <typename TW, bool VECW, int V>
__device__ __forceinline__ void put_dw(const EmbedGradLaunch& L, int64_t v, int64_t e, const float (&f)[V]) {
  constexpr int VW = LType<TW>::kVec, EW = 16 / VW;
  char* row = (char*)L.dw + v * L.ldw * EW;
  if constexpr (V % VW == 0) {
#pragma unroll
    for (int h = 0; h < V; h += VW) {
      if (e + h >= L.dim) break;  // whole chunks of dy's type may be two of dweight's
      float o[VW];
      if (L.accumulate) l_widen<TW>(l_load<TW, VECW>(row, e + h, L.dim), o);
      else {
#pragma unroll
        for (int i = 0; i < VW; ++i) o[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) o[i] = fmaf(L.scale, f[h + i], o[i]);
      l_store<TW, VECW>(row, e + h, L.dim, l_narrow<TW>(o));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e + i < L.dim) {
        const float old = L.accumulate ? LType<TW>::get(row, e + i) : 0.f;
        LType<TW>::put(row, e + i, fmaf(L.scale, f[i], old));
      }
  }
}

// Number of leading positions p, p + step, .. < limit whose key is k, looked
// at by the group's lanes at once.
__device__ __forceinline__ int run_length(const uint32_t* key, int64_t p, int64_t limit, uint32_t k, int l,
                                          int lanes, int step) {
  const int first = (threadIdx.x & 63) - l;
  int n = 0;
  for (;;) {
    const int64_t at = p + (int64_t)(n + l) * step;
    const uint64_t same = __ballot(at < limit && key[at] == k) >> first;
    const uint64_t miss = lanes == 64 ? ~same : ~same & ((1ull << lanes) - 1ull);
    if (miss) return n + (__ffsll((unsigned long long)miss) - 1);
    n += lanes;
  }
}

// One lane group per sorted position and slice: sums the run that starts
// there.
template <typename T, bool VEC, typename TW, bool VECW>
__global__ __launch_bounds__(256) void embed_rows(const EmbedGradLaunch L, const uint32_t* key,
                                                  const uint32_t* idx, int lanes, int shift) {
  constexpr int V = LType<T>::kVec;
  const int g = threadIdx.x >> shift, l = threadIdx.x & (lanes - 1);
  const int64_t s = (int64_t)blockIdx.x * (256 >> shift) + g;
  if (s >= L.tokens) return;
  const uint32_t k = key[s];
  if (k >= (uint32_t)L.vocab || (s > 0 && key[s - 1] == k)) return;
  const int64_t e = ((int64_t)blockIdx.y * lanes + l) * V;
  float acc[V] = {};
  // rows up to the first piece boundary, whole pieces, the rest
  const int64_t b = min((s + kEmbedPiece - 1) / kEmbedPiece * kEmbedPiece, L.tokens);
  const int head = run_length(key, s, b, k, l, lanes, 1);
  add_rows<T, VEC>(L, idx, s, head, e, l, lanes, acc);
  int64_t p = s + head;
  if (p == b) {
    // a piece is whole if its last key is k too
    const int whole = run_length(key, p + kEmbedPiece - 1, L.tokens, k, l, lanes, kEmbedPiece);
    const float* pc = L.pieces + (p / kEmbedPiece) * L.dim + e;
    if (e < L.dim) {
#pragma unroll 8
      for (int j = 0; j < whole; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (VEC || e + i < L.dim) acc[i] += pc[j * L.dim + i];
      }
    }
    p += (int64_t)whole * kEmbedPiece;
    const int tail = run_length(key, p, L.tokens, k, l, lanes, 1);
    add_rows<T, VEC>(L, idx, p, tail, e, l, lanes, acc);
  }
  if (e < L.dim) put_dw<TW, VECW, V>(L, k, e, acc);
}

__device__ __forceinline__ void zero_rows(const EmbedGradLaunch& L, int64_t v0, int64_t v1, int64_t w, int64_t W) {
  const int esz = L.dwBf16 ? 2 : 4, lane = threadIdx.x & 63;
  auto zero = [lane](char* p, int64_t n, int64_t w, int64_t W) {
    constexpr int64_t kPiece = 8192;
    const lu32x4 z = {0u, 0u, 0u, 0u};
    const int64_t head = min(n, (int64_t)(-(uintptr_t)p & 15)), body = (n - head) & ~(int64_t)15;
    for (int64_t c = w * kPiece; c < body; c += W * kPiece) {
      const int64_t end = min(c + kPiece, body);
      for (int64_t e = c + lane * 16; e < end; e += 1024) __builtin_nontemporal_store(z, (lu32x4*)(p + head + e));
    }
    if (w == 0) {  // less than 16 bytes at either end
      if (lane * 2 < head) *(uint16_t*)(p + lane * 2) = 0;
      if (head + body + lane * 2 < n) *(uint16_t*)(p + head + body + lane * 2) = 0;
    }
  };
  if (L.ldw == L.dim) {
    zero((char*)L.dw + v0 * L.ldw * esz, (v1 - v0) * L.dim * esz, w, W);
  } else {
    for (int64_t v = v0 + w; v < v1; v += W) zero((char*)L.dw + v * L.ldw * esz, L.dim * esz, 0, 1);
  }
}

__global__ __launch_bounds__(256) void embed_zero(const EmbedGradLaunch L) {
  zero_rows(L, 0, L.zeroRows, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), (int64_t)gridDim.x * 4);
}

// Lanes of a group: the chunks of a row, at most a wave's.
int group_shift(int64_t chunks) {
  int s = 3;
  while (s < 6 && (1 << s) < chunks) ++s;
  return s;
}

template <typename T, bool VEC, typename TW, bool VECW>
hipError_t rows_launch(const EmbedGradLaunch& L, hipStream_t st) {
  constexpr int V = LType<T>::kVec;
  const int64_t chunks = (L.dim + V - 1) / V;
  const int sh = group_shift(chunks), lanes = 1 << sh, per = 256 >> sh;
  const int64_t slices = (chunks + lanes - 1) / lanes;
  const int64_t np = L.tokens / kEmbedPiece;
  // the device-memory sort ends in the buffer its last pass wrote
  const uint32_t *key = L.key[0], *idx = L.idx[0];
  const int64_t sums = (np + per - 1) / per * slices;
  const int64_t zeros = L.zeroRows < L.vocab ? std::min<int64_t>(1024, L.vocab - L.zeroRows) : 0;
  if (sums + zeros > 0)
    hipLaunchKernelGGL((embed_pieces<T, VEC>), dim3(sums + zeros), dim3(256), 0, st, L, key, idx, lanes, sh,
                       (int)slices, (int)sums);
  if (L.tokens > 0)
    hipLaunchKernelGGL((embed_rows<T, VEC, TW, VECW>), dim3((L.tokens + per - 1) / per, slices), dim3(256), 0,
                       st, L, key, idx, lanes, sh);
  return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t rows_dw(const EmbedGradLaunch& L, hipStream_t st) {
  if (L.dwBf16)
    return L.vecw ? rows_launch<T, VEC, Bf16, true>(L, st) : rows_launch<T, VEC, Bf16, false>(L, st);
  return L.vecw ? rows_launch<T, VEC, float, true>(L, st) : rows_launch<T, VEC, float, false>(L, st);
}

}  // namespace

hipError_t launch_embedding(const EmbedLaunch& L, hipStream_t st) {
  const int V = L.bf16 ? 8 : 4;
  const int64_t chunks = (L.dim + V - 1) / V;
  const int sh = group_shift(chunks), lanes = 1 << sh, per = 256 >> sh;
  const dim3 grid((L.tokens + per - 1) / per, (chunks + 4 * lanes - 1) / (4 * lanes));
  if (L.bf16) {
    if (L.vec) hipLaunchKernelGGL((embedding_kernel<Bf16, true>), grid, dim3(256), 0, st, L, lanes, sh);
    else hipLaunchKernelGGL((embedding_kernel<Bf16, false>), grid, dim3(256), 0, st, L, lanes, sh);
  } else {
    if (L.vec) hipLaunchKernelGGL((embedding_kernel<float, true>), grid, dim3(256), 0, st, L, lanes, sh);
    else hipLaunchKernelGGL((embedding_kernel<float, false>), grid, dim3(256), 0, st, L, lanes, sh);
  }
  return hipGetLastError();
}

hipError_t launch_embedding_grad(const EmbedGradLaunch& L0, hipStream_t st) {
  EmbedGradLaunch L = L0;
  int bits = 1;  // of the largest key, vocab
  while ((L.vocab >> bits) != 0) ++bits;
  // Zeros: what HBM takes while the one-workgroup sort runs (7, 14 or 44 µs
  // for its three sizes) is written beside it,
  // the rest beside the pieces' sums; all at once where there is no such sort.
  const bool small = L.tokens > 0 && L.tokens <= kEmbedSmallSort;
  const int64_t row = L.dim * (L.dwBf16 ? 2 : 4);
  const int64_t hidden = L.tokens <= 1024 ? 35 << 20 : L.tokens <= 4096 ? 70 << 20 : 240 << 20;
  if (L.accumulate) L.zeroRows = L.vocab;  // nothing to write
  else L.zeroRows = small ? std::min(L.vocab, hidden / row + 1) : L.vocab;
  const int64_t zero = L.accumulate ? 0 : std::min<int64_t>(256, (L.zeroRows * row + 65535) / 65536);
  if (!small && zero > 0) hipLaunchKernelGGL(embed_zero, dim3(zero * 4), dim3(256), 0, st, L);
  if (small) {
    const int passes = (bits + 8) / 9;
    const dim3 grid(1 + zero), block(1024);
    if (L.tokens <= 1024) hipLaunchKernelGGL(embed_sort_small<1>, grid, block, 0, st, L, passes);
    else if (L.tokens <= 4096) hipLaunchKernelGGL(embed_sort_small<4>, grid, block, 0, st, L, passes);
    else hipLaunchKernelGGL(embed_sort_small<16>, grid, block, 0, st, L, passes);
  } else if (L.tokens > 0) {
    const int passes = (bits + kEmbedSortBits - 1) / kEmbedSortBits;
    const int blocks = (int)((L.tokens + kEmbedSortBlock - 1) / kEmbedSortBlock);
    for (int p = 0; p < passes; ++p) {
      hipLaunchKernelGGL(embed_sort_count, dim3(blocks), dim3(256), 0, st, L, p);
      hipLaunchKernelGGL(embed_sort_scan, dim3(1), dim3(1024), 0, st, L.counts, (int64_t)blocks * kSortBins);
      hipLaunchKernelGGL(embed_sort_scatter, dim3(blocks), dim3(256), 0, st, L, p);
    }
    if ((passes & 1) == 0) {  // pass p writes buffer p & 1: the last one ended in buffer 1
      std::swap(L.key[0], L.key[1]);
      std::swap(L.idx[0], L.idx[1]);
    }
  }
  if (L.dyBf16) return L.vec ? rows_dw<Bf16, true>(L, st) : rows_dw<Bf16, false>(L, st);
  return L.vec ? rows_dw<float, true>(L, st) : rows_dw<float, false>(L, st);
}

}  // namespace muon

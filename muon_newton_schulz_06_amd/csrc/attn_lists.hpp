// The block lists of the attention's passes.
#pragma once

#include "attention.hpp"

namespace muon {

// Inclusive scan over the workgroup; f combines.
template <typename F> __device__ __forceinline__ int64_t a_scan(int64_t v, int64_t* red, F f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(v, o, 64);
    if (lane >= o) v = f(v, u);
  }
  if (lane == 63) red[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v = f(v, red[w]);
  __syncthreads();
  return v;
}

// Block list number `list` of a batch, by one workgroup.  The spans are the rows
// before the first offset, each sequence, and the rows after the last one; the
// first and last of these have no keys.  Offsets are cut to [0, tokens] and
// one below its predecessor is raised to it, so whatever they hold, every row
// belongs to exactly one span.
constexpr int kPrep = 1024;  // threads
__device__ __forceinline__ void attn_lists(const AttnPrepLaunch& L, int list) {
  __shared__ int64_t red[kPrep / 64];
  __shared__ int begin[kPrep], size[kPrep], first[kPrep];  // a chunk of spans: tokens, blocks before
  const auto& D = L.list[list];
  const int tid = threadIdx.x, spans = L.offsets ? L.sequences + 2 : 1;
  auto larger = [](int64_t a, int64_t b) { return a > b ? a : b; };
  auto sum = [](int64_t a, int64_t b) { return a + b; };
  const int64_t tokens = D.tokens;
  int64_t edge = 0;  // where the chunk's first span begins
  int done = 0;      // blocks of the chunks before
  for (int s0 = 0; s0 < spans; s0 += kPrep) {
    const int s = s0 + tid;
    int64_t end = tokens;  // of span s
    if (L.offsets && s <= L.sequences) end = min(max((int64_t)L.offsets[s], (int64_t)0), tokens);
    end = a_scan(larger(end, edge), red, larger);
    size[tid] = (int)end;  // for the neighbour
    __syncthreads();
    const int64_t start = tid ? size[tid - 1] : edge;
    edge = size[kPrep - 1];
    __syncthreads();
    const int64_t n = s < spans ? end - start : 0;
    const int blocks = (int)((n * D.units + D.per - 1) / D.per);
    const int upto = (int)a_scan(blocks, red, sum);
    begin[tid] = (int)start;
    size[tid] = (int)n;
    first[tid] = upto - blocks;
    __syncthreads();
    const int total = first[kPrep - 1] + (int)((size[kPrep - 1] * (int64_t)D.units + D.per - 1) / D.per);
    for (int b = tid; b < total; b += kPrep) {
      int lo = 0, hi = kPrep - 1;  // the last span whose blocks begin at or before b
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= b) lo = mid;
        else hi = mid - 1;
      }
      const bool inside = !L.offsets || (s0 + lo > 0 && s0 + lo <= L.sequences);
      D.blocks[done + b] = AttnBlock{begin[lo], size[lo], inside ? size[lo] : 0, (b - first[lo]) * D.per};
    }
    done += total;
    __syncthreads();
  }
  if (tid == 0) *D.count = done;
  if (!D.cum) return;
  int64_t before = 0;
  for (int b0 = 0; b0 < done; b0 += kPrep) {
    int64_t n = 0;
    if (b0 + tid < done) {
      const AttnBlock B = D.blocks[b0 + tid];
      const int64_t nq = L.offsets ? B.n : L.queries, nk = L.offsets ? B.nk : L.keys;
      if (D.units == 1 && D.tile == 0) {
        const int64_t first = L.causal ? max(B.at - (B.n - nq), (int64_t)0) & ~(int64_t)31 : 0;
        n = B.nk > 0 && nq > first ? (nq - first + 31) / 32 * L.group : 1;
      } else {
        const int64_t last = min((int64_t)B.at + D.per, nq * D.units) - 1;
        const int64_t see = L.causal ? min(max(last / D.units + nk - nq + 1, (int64_t)0), nk) : nk;
        n = max((see + D.tile - 1) / D.tile, (int64_t)1);
      }
    }
    const int64_t upto = a_scan(n, red, sum);
    if (b0 + tid < done) D.cum[b0 + tid] = before + upto - n;
    if (tid == kPrep - 1) red[0] = upto;
    __syncthreads();
    before += red[0];
    __syncthreads();
  }
  if (tid == 0) D.cum[done] = before;
}

}  // namespace muon

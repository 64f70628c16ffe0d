// What precedes the attention products: the block lists, and aligned copies
// of tensors that the 16-byte loads into LDS cannot read.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"
#include "attn_lists.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

__global__ __launch_bounds__(kPrep) void attn_prep(const AttnPrepLaunch L) { attn_lists(L, blockIdx.x); }

// One workgroup per 256 chunks of a tensor's copy; the pitch's end holds zeros.
template <typename T> __global__ __launch_bounds__(256) void attn_copy(const AttnCopies K) {
  constexpr int V = LType<T>::kVec, E = AT<T>::kBytes;
  const AttnCopy& C = K.c[blockIdx.y];
  const int per = C.pitch / V;
  const int64_t n = C.batch * C.tokens * C.heads * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    int64_t r = i / per;
    const int e = (int)(i - r * per) * V;
    const int h = (int)(r % C.heads);
    r /= C.heads;
    const int64_t b = r / C.tokens, t = r - b * C.tokens;
    const char* src = (const char*)C.src + (b * C.s[0] + t * C.s[1] + h * C.s[2]) * E;
    ((lu32x4*)C.dst)[i] = l_load<T, false>(src, e, C.dim);
  }
}

}  // namespace

// Before a forward pass; before a backward pass the lists are made beside the
// row sums (attn_rows.hip).
hipError_t launch_attn_prep(const AttnPrepLaunch& L, hipStream_t st) {
  attn_prep<<<dim3(L.lists), kPrep, 0, st>>>(L);
  return hipGetLastError();
}

hipError_t launch_attn_copy(bool bf16, const AttnCopies& K, hipStream_t st) {
  int64_t most = 1;
  for (int i = 0; i < K.n; ++i)
    most = std::max(most, K.c[i].batch * K.c[i].tokens * K.c[i].heads * K.c[i].pitch / (bf16 ? 8 : 4));
  const dim3 grid((unsigned)std::min<int64_t>((most + 255) / 256, 1 << 16), K.n);
  if (bf16) attn_copy<Bf16><<<grid, 256, 0, st>>>(K);
  else attn_copy<float><<<grid, 256, 0, st>>>(K);
  return hipGetLastError();
}

}  // namespace muon

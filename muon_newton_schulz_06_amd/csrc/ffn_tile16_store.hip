// bf16 feed-forward products with a plain result: the down projection, the
// gradient of the input, the gradients of the weights; the aligned copy of an
// operand.
#include "ffn_tile16.hpp"

namespace muon {
namespace {

// rows × cols of any stride and alignment → rows of ldo (a multiple of 8),
// zeros beyond cols; one operand per blockIdx.y.
__global__ __launch_bounds__(256) void ffn_pack(const FfnPacks L) {
  const FfnPack& K = L.p[blockIdx.y];
  const int64_t chunks = K.ldo / 8;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < K.rows * chunks; e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / chunks, c = (e - r * chunks) * 8;
    const lu32x4 v = l_load<Bf16, false>((const uint16_t*)K.src + r * K.ld, c, K.cols);
    *(lu32x4*)((uint16_t*)K.dst + r * K.ldo + c) = v;
  }
}

}  // namespace

hipError_t launch_ffn16_store(int tile, bool aRowContig, bool bRowContig, const FfnLaunch& L,
                              hipStream_t st) {
  if (aRowContig) ffn16_launch<FFN_STORE, true, true>(tile, L, st);
  else if (bRowContig) ffn16_launch<FFN_STORE, false, true>(tile, L, st);
  else ffn16_launch<FFN_STORE, false, false>(tile, L, st);
  return hipGetLastError();
}

hipError_t launch_ffn_pack(const FfnPacks& K, hipStream_t st) {
  int64_t blocks = 1;
  for (int i = 0; i < K.n; ++i) {
    const int64_t b = (K.p[i].rows * (K.p[i].ldo / 8) + 255) / 256;
    blocks = b > blocks ? b : blocks;
  }
  hipLaunchKernelGGL(ffn_pack, dim3(blocks < 16384 ? blocks : 16384, K.n), dim3(256), 0, st, K);
  return hipGetLastError();
}

}  // namespace muon

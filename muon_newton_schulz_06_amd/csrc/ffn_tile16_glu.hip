// bf16 feed-forward products: the gated projections, the product with the
// down projection's weights in the backward pass.
#include "ffn_tile16.hpp"

namespace muon {

hipError_t launch_ffn16_glu(int tile, const FfnLaunch& L, hipStream_t st) {
  const dim3 grid(L.tiles[L.nprob]);
  if (tile == 256) hipLaunchKernelGGL((ffn_tile16<256, FFN_GLU, false, false>), grid, dim3(512), 0, st, L);
  else hipLaunchKernelGGL((ffn_tile16<128, FFN_GLU, false, false>), grid, dim3(256), 0, st, L);
  return hipGetLastError();
}

hipError_t launch_ffn16_back(int tile, const FfnLaunch& L, hipStream_t st) {
  const dim3 grid(L.tiles[L.nprob]);
  if (tile == 256) hipLaunchKernelGGL((ffn_tile16<256, FFN_BACK, false, true>), grid, dim3(512), 0, st, L);
  else hipLaunchKernelGGL((ffn_tile16<128, FFN_BACK, false, true>), grid, dim3(256), 0, st, L);
  return hipGetLastError();
}

}  // namespace muon

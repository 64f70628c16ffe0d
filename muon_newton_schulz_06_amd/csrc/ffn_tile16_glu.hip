// bf16 feed-forward products: the gated projections, the product with the
// down projection's weights in the backward pass.
#include "ffn_tile16.hpp"

namespace muon {

hipError_t launch_ffn16_glu(int tile, const FfnLaunch& L, hipStream_t st) {
  ffn16_launch<FFN_GLU, false, false>(tile, L, st);
  return hipGetLastError();
}

hipError_t launch_ffn16_back(int tile, const FfnLaunch& L, hipStream_t st) {
  ffn16_launch<FFN_BACK, false, true>(tile, L, st);
  return hipGetLastError();
}

}  // namespace muon

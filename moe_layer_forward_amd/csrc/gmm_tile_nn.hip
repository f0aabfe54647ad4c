// Tile kernel of the grouped products, bf16 gradient for the rows (gmm_tile.h).
#include "gmm_tile.h"

namespace moe {
hipError_t launch_gmm_tile_nn(const GmmArgs& a, int waves, bool once, hipStream_t s) {
  return gmm_launch_rows<GmmForm::kNN, GmmBf16>(a, waves, once, s);
}
}  // namespace moe

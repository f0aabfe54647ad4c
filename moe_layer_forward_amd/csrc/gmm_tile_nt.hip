// Tile kernel of the grouped products, bf16 forward (gmm_tile.h).
#include "gmm_tile.h"

namespace moe {
hipError_t launch_gmm_tile_nt(const GmmArgs& a, int waves, bool once, hipStream_t s) {
  return gmm_launch_rows<GmmForm::kNT, GmmBf16>(a, waves, once, s);
}
}  // namespace moe

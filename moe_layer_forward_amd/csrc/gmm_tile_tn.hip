// Tile kernel of the grouped products, bf16 gradient for the weights (gmm_tile.h).
#include "gmm_tile.h"

namespace moe {
int64_t gmm_tile_items(const GmmArgs& a) {
  const int64_t slabs = ((a.form == GmmForm::kNT ? a.N : a.K) + kGmmTile - 1) / kGmmTile;
  return slabs * (a.form == GmmForm::kTN ? (int64_t)a.G * ((a.N + kGmmTile - 1) / kGmmTile)
                                         : gmm_max_tiles(a.max_rows, a.G, kGmmTile));
}

hipError_t launch_gmm_tile_tn(const GmmArgs& a, hipStream_t s) {
  const int p_tiles = (a.N + kGmmTile - 1) / kGmmTile, slabs = (a.K + kGmmTile - 1) / kGmmTile;
  const int64_t tiles = (int64_t)a.G * p_tiles, items = tiles * slabs;
  const int chunk = gmm_weight_chunk(items);
  const dim3 grid((unsigned)(gmm_weight_grid(items) * a.split)), block(kGmmThreads);
  if (a.row_index)
    gmm_weights_kernel<GmmBf16, true><<<grid, block, 0, s>>>(a, tiles, slabs, p_tiles, chunk);
  else
    gmm_weights_kernel<GmmBf16, false><<<grid, block, 0, s>>>(a, tiles, slabs, p_tiles, chunk);
  return hipGetLastError();
}
}  // namespace moe

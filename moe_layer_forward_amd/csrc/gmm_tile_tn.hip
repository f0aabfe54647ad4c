// Tile kernel of the grouped products, bf16 gradient for the weights (gmm_tile.h).
#include "gmm_tile.h"

namespace moe {
namespace {

template <int W>
hipError_t launch_weights(const GmmArgs& a, hipStream_t s) {
  constexpr int kTile = GmmShape<W>::kTile;
  const int p_tiles = (a.N + kTile - 1) / kTile, slabs = (a.K + kTile - 1) / kTile;
  const int64_t tiles = gmm_max_sums(a) * p_tiles, items = tiles * slabs;
  const int chunk = gmm_weight_chunk(items);
  const dim3 grid = gmm_grid(gmm_weight_grid(items)), block(64 * W);
  if (a.row_index)
    gmm_weights_kernel<GmmBf16, W, true><<<grid, block, 0, s>>>(a, tiles, slabs, p_tiles, chunk);
  else
    gmm_weights_kernel<GmmBf16, W, false><<<grid, block, 0, s>>>(a, tiles, slabs, p_tiles, chunk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gmm_tile_tn(const GmmArgs& a, int waves, hipStream_t s) {
  return waves == 8 ? launch_weights<8>(a, s) : launch_weights<4>(a, s);
}

int64_t gmm_tile_items(const GmmArgs& a, int waves) {
  const int64_t tile = 32 * waves, slabs = ((a.form == GmmForm::kNT ? a.N : a.K) + tile - 1) / tile;
  return slabs * (a.form == GmmForm::kTN ? (int64_t)a.G * ((a.N + tile - 1) / tile)
                                         : gmm_max_tiles(a.max_rows, a.G, (int)tile));
}

}  // namespace moe

// How the output tiles of row groups become work items, and which work-group takes which.
#pragma once
#include "gmm_core.h"

namespace moe {

constexpr int kGmmSuper = 4;  // row tiles that run side by side on one XCD

// Work items are tiles x slabs, numbered so that kGmmSuper tiles run slab by slab, side by side: 32
// work-groups of an XCD then share kGmmSuper tiles' rows and 8 slabs in its L2.
__device__ __forceinline__ void gmm_unnumber(int64_t item, int64_t tiles, int slabs, int64_t& tile, int& slab) {
  const int64_t sup = item / ((int64_t)kGmmSuper * slabs), first = sup * kGmmSuper;
  const int rem = (int)(item - first * slabs);
  const int n = tiles - first < kGmmSuper ? (int)(tiles - first) : kGmmSuper;
  tile = first + rem % n;
  slab = rem / n;
}

// The hardware deals work-group b to XCD b % 8.  The items of the full tiles are cut into one contiguous range per
// XCD, and after them those of the partial tiles: every XCD gets the same share of both (to within one
// item), and the short items come last, where they fill the chip's last round.  False for padding.
__device__ __forceinline__ bool gmm_row_item(int64_t b, const GmmTiles& t, int slabs, int& tile, int& slab) {
  const int64_t xcd = b % kXcds;
  int64_t local = b / kXcds, nf = (int64_t)t.full * slabs, np = (int64_t)t.partial * slabs, tt;
  const int64_t per_f = (nf + kXcds - 1) / kXcds, per_p = (np + kXcds - 1) / kXcds;
  if (local < per_f) {
    const int64_t item = xcd * per_f + local;
    if (item >= nf) return false;
    gmm_unnumber(item, t.full, slabs, tt, slab);
    tile = (int)tt;
    return true;
  }
  local -= per_f;
  const int64_t item = xcd * per_p + local;
  if (local >= per_p || item >= np) return false;
  gmm_unnumber(item, t.partial, slabs, tt, slab);
  tile = t.full + (int)tt;
  return true;
}

// Work-groups that cover the items of any grouping of max_rows rows.
inline int64_t gmm_row_grid(int64_t max_rows, int G, int slabs, int tile) {
  const int64_t full = max_rows / tile, partial = max_rows < G ? max_rows : G;
  const auto per = [&](int64_t tiles) { return (tiles * slabs + kXcds - 1) / kXcds; };
  return (per(full) + per(partial)) * kXcds;
}

}  // namespace moe

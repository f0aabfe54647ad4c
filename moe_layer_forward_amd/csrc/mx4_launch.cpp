// Which kernel a microscaled 4-bit product runs on.
#include <algorithm>

#include "mx4.h"

namespace moe {
namespace {

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }

// Waves of the tile kernel's work-groups: 8 (256 x 256 tiles, one work-group to a CU) move half the bytes per product
// through LDS, 4 (128 x 128, two to a CU) pad less and fill the chip with fewer tiles (rules as in gmm_launch.cpp; 8192 x
// 18432 x 7168: 565 us with 8, 690 with 4; 64 x 18432 x 7168: 25 with 8, 17 with 4).  Groups that mostly fit one row tile
// of 128 (343 groups of 96 rows, 2624 x 384: 137 us with 8, 126 with 4; 91 of 103, 712 x 4992: 72 and 64; 177 of 142, 1160 x
// 2528: 117 and 161).
int tile_waves(const Mx4Args& a) {
  if (padded(a.N, 256) * 100 > padded(a.N, 128) * 115) return 4;
  if (a.G > 1 && a.max_rows <= (int64_t)a.G * 112) return 4;
  const int64_t items = mx4_tile_grid(a, 8);
  return items >= 512 || (items >= 160 && a.K >= 12 * 256) ? 8 : 4;
}

// Whether the scales are packed before the 256 x 256 tiles.  The product gains a tenth of its time (about 4 POP/s), the
// packing takes 4 us and two passes over the scales at 2.5 TB/s: 8192 rows, 18432 x 7168: 565 -> 512 us; 3 groups of 16384
// rows, 4096 x 7168: 290 -> 262; 4096 x 4096 x 4096: 40.5 and 40.7; 48 groups of 8192 rows, 2048 x 7168: 133 -> 138.
bool pack_scales(const Mx4Args& a) {
  const double product = 2.0 * (double)a.max_rows * a.N * a.K / 4e15, bytes = 2.0 * (double)mx4_packed_bytes(a);
  return 0.1 * product > 4e-6 + bytes / 2.5e12;
}

}  // namespace

// Groups of up to 12 rows on average: the ring, one pass over the weights (340 groups of 12 rows, 1264 x 928: 62 us, tiles
// 71; 120 of 9, 1736 x 4480: 106 and 117; with 15 rows: 358 groups, 960 x 3008: 178 and 135), where it has 800 items, three
// for every two of its work-groups (31 groups, 31 rows, 3904 x 1344: 17.7 and 17.0; 19 groups of 12 rows, 2176 x 3520, 561
// items: 30 and 19).  Few items of long sums: the stream kernel, whose waves share a sum (24 groups of 2 rows, 896 x 5632:
// 19 us on the ring, 15 on tiles, 13.5).  Otherwise tiles.
// One group of up to 64 rows: the stream kernel, with 32-column items where 16-column ones would read the rows of x too
// often and enough of them remain (32 rows, 7168 x 18432: 32 us with 16, 24 with 32; 4096 x 14336: 13.5 and 17.3); from 33
// rows on tiles where 128 columns still make 72 of them (64 rows, 18432 x 7168: 38 us, 24 on tiles; 7168 x 18432: 34 and
// 48).
Mx4Plan mx4_plan(const Mx4Args& a, void* workspace) {
  Mx4Plan p{a, Mx4Kernel::kTile, {1, 1}, 0, "matmul_mx4_stream"};
  if (a.G > 1) {
    const int64_t items = mx4_ring_items(a);
    if (a.max_rows <= (int64_t)a.G * 12 && items >= 800 && items <= (int64_t)1 << 30) {
      p.kernel = Mx4Kernel::kRing;
      p.name = "matmul_mx4_ring";
    } else if (a.max_rows <= (int64_t)a.G * 12 && items < 256 && a.K >= 2048) {
      p.kernel = Mx4Kernel::kStream;
    }
  } else if (a.max_rows <= 32 || (a.max_rows <= 64 && a.N < 72 * 128)) {
    p.kernel = Mx4Kernel::kStream;
    p.stream.p_blocks = (int)std::max<int64_t>(1, (a.max_rows + 15) / 16);
    p.stream.q_blocks = a.max_rows > 8 && a.N >= 5120 ? 2 : 1;
  }
  if (p.kernel == Mx4Kernel::kTile) {
    p.tile_waves = tile_waves(a);
    p.name = p.tile_waves == 8 ? "matmul_mx4_tile256" : "matmul_mx4_tile128";
    p.pack = p.tile_waves == 8 && pack_scales(a);
    p.args.packed = p.pack ? static_cast<uint8_t*>(workspace) : nullptr;
  }
  return p;
}

size_t mx4_workspace(const Mx4Args& a) {
  const Mx4Plan p = mx4_plan(a, nullptr);
  return p.pack ? mx4_packed_bytes(a) : 0;
}

bool mx4_grid_ok(const Mx4Args& a) {
  const Mx4Plan p = mx4_plan(a, nullptr);
  const int64_t items = p.kernel == Mx4Kernel::kTile   ? mx4_tile_grid(a, p.tile_waves)
                        : p.kernel == Mx4Kernel::kRing ? mx4_ring_items(a)
                                                       : mx4_stream_grid(a, p.stream);
  return items <= (int64_t(1) << 31);
}

hipError_t launch_mx4(const Mx4Plan& p, hipStream_t s) {
  if (p.kernel == Mx4Kernel::kTile) return launch_mx4_tile(p.args, p.tile_waves, s);
  if (p.kernel == Mx4Kernel::kRing) return launch_mx4_ring(p.args, s);
  return launch_mx4_stream(p.args, p.stream, s);
}

}  // namespace moe

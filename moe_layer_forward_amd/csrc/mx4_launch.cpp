// Which kernel a microscaled 4-bit product runs on.
#include <algorithm>

#include "mx4.h"

namespace moe {
namespace {

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }

// Waves of the tile kernel's work-groups: 8 (256 x 256 tiles, one work-group to a CU) move half the bytes per product
// through LDS, 4 (128 x 128, two to a CU) pad less and fill the chip with fewer tiles (rules as in gmm_launch.cpp; 8192 x
// 18432 x 7168: 565 us with 8, 690 with 4; 64 x 18432 x 7168: 25 with 8, 17 with 4).
int tile_waves(const Mx4Args& a) {
  if (padded(a.N, 256) * 100 > padded(a.N, 128) * 115) return 4;
  const int64_t items = mx4_tile_grid(a, 8);
  return items >= 512 || (items >= 160 && a.K >= 12 * 256) ? 8 : 4;
}

// Whether the tile kernel's scales are packed first.  The product gains a tenth of its time (about 4 POP/s), the packing
// takes 4 us and two passes over the scales at 2.5 TB/s: 8192 rows, 18432 x 7168: 565 -> 512 us; 3 groups of 16384 rows,
// 4096 x 7168: 290 -> 262; 4096 x 4096 x 4096: 40.5 and 40.7; 48 groups of 8192 rows, 2048 x 7168: 133 -> 138.
bool pack_scales(const Mx4Args& a, int waves) {
  const double product = 2.0 * (double)a.max_rows * a.N * a.K / 4e15, bytes = 2.0 * (double)mx4_packed_bytes(a, waves);
  return 0.1 * product > 4e-6 + bytes / 2.5e12;
}

}  // namespace

Mx4Plan mx4_plan(const Mx4Args& a, void* workspace) {
  Mx4Plan p{a, Mx4Kernel::kStream, {4, 1, 8}, 8, "matmul_mx4_stream"};
  const int64_t mean = a.max_rows / a.G;
  if (a.max_rows > (int64_t)a.G * 64) {
    p.kernel = Mx4Kernel::kTile;
    p.tile_waves = tile_waves(a);
  } else if (a.G == 1) {
    p.stream.p_blocks = (int)std::max<int64_t>(1, (a.max_rows + 15) / 16);
    if (p.stream.p_blocks >= 3 && a.N >= 160 * 64) {
      p.kernel = Mx4Kernel::kTile;
      p.tile_waves = 4;
    }
  } else if (mean > 24) {
    p.kernel = Mx4Kernel::kTile;
    p.tile_waves = 4;
  } else {
    p.kernel = Mx4Kernel::kRing;
    p.stream = mean > 8 ? Mx4Stream{2, 1, 2} : Mx4Stream{1, 2, 2};
    p.name = "matmul_mx4_ring";
  }
  if (p.kernel == Mx4Kernel::kTile) {
    p.name = p.tile_waves == 8 ? "matmul_mx4_tile256" : "matmul_mx4_tile128";
    p.pack = pack_scales(a, p.tile_waves);
    p.args.packed = p.pack ? static_cast<uint8_t*>(workspace) : nullptr;
  }
  return p;
}

size_t mx4_workspace(const Mx4Args& a) {
  const Mx4Plan p = mx4_plan(a, nullptr);
  return p.pack ? mx4_packed_bytes(a, p.tile_waves) : 0;
}

bool mx4_grid_ok(const Mx4Args& a) {
  const Mx4Plan p = mx4_plan(a, nullptr);
  const int64_t items = p.kernel == Mx4Kernel::kTile   ? mx4_tile_grid(a, p.tile_waves)
                        : p.kernel == Mx4Kernel::kRing ? mx4_ring_items(a, p.stream.p_blocks, p.stream.q_blocks)
                                                       : mx4_stream_grid(a, p.stream);
  return items <= (int64_t(1) << 31);
}

hipError_t launch_mx4(const Mx4Plan& p, hipStream_t s) {
  if (p.kernel == Mx4Kernel::kTile) return launch_mx4_tile(p.args, p.tile_waves, s);
  if (p.kernel == Mx4Kernel::kRing) return launch_mx4_ring(p.args, p.stream.p_blocks, p.stream.q_blocks, p.stream.waves, s);
  return launch_mx4_stream(p.args, p.stream, s);
}

}  // namespace moe

// Which kernel a microscaled 4-bit product runs on.
#include <algorithm>
#include <cmath>

#include "mx4.h"

namespace moe {
namespace {

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }

// Waves of the tile kernel's work-groups: 8 (256 x 256 tiles, one work-group to a CU) move half the bytes per product
// through LDS, 4 (128 x 128, two to a CU) pad less, and their rounds are shorter.
//   * 4 where 256 columns would mostly pad, and for groups that mostly fit one row tile of 128 (343 groups of 96
//     rows, 2624 x 384: 131 us with 4, 144 with 8; 48 of 64, 2048 x 7168: 73 and 81).
//   * Otherwise by the rounds over the chip's 256 CUs.  A work-group of 8 takes 1.7 us a step and 5 around them, its
//     last row tile from half of that; two of 4 on a CU 1.25 a step and 3, one 0.6 of that.  8's rounds are whole
//     ones while there are few.  Within 4% of the better of the two on 193 of 200 sizes drawn.  1024 rows, 18432 x
//     7168, 288 tiles of 256: 85 us with 4, 104 with 8; 8192 rows: 690 and 500; 8 groups of 512 rows, 2048 x 7168: 39
//     and 52; 177 of 142, 1160 x 2528: 194 and 118.
int tile_waves(const Mx4Args& a) {
  const double rows = (double)a.max_rows / a.G, steps = (a.K + 255) / 256;
  if (rows <= 0 || padded(a.N, 256) * 100 > padded(a.N, 128) * 115 || (a.G > 1 && rows <= 112)) return 4;
  const double full = std::floor(rows / 256), part = rows - 256 * full, tiles = part > 0 ? full + 1 : full;
  const double each = (full + (part > 0 ? 0.5 + part / 512 : 0)) / tiles;
  double r8 = a.G * tiles * (padded(a.N, 256) / 256) / 256;
  r8 = r8 <= 3 ? std::ceil(r8) : r8 + 0.5;
  const double r4 = a.G * std::ceil(rows / 128) * (padded(a.N, 128) / 128) / 512 + 0.15;
  const double t4 = r4 <= 0.65 ? 0.6 : std::max(1.0, r4);  // one to a CU
  return t4 * (1.25 * steps + 3) < r8 * each * (1.7 * steps + 5) ? 4 : 8;
}

// Whether the scales are packed before the 256 x 256 tiles.  The product gains a tenth of its time (about 4 POP/s),
// the packing takes 4 us and two passes over the scales at 2.5 TB/s: 8192 rows, 18432 x 7168: 565 -> 512 us; 3 groups
// of 16384 rows, 4096 x 7168: 290 -> 262; 4096 x 4096 x 4096: 40.5 and 40.7; 48 groups of 8192 rows, 2048 x 7168: 133
// -> 138.
bool pack_scales(const Mx4Args& a) {
  const double product = 2.0 * (double)a.max_rows * a.N * a.K / 4e15, bytes = 2.0 * (double)mx4_packed_bytes(a);
  return 0.1 * product > 4e-6 + bytes / 2.5e12;
}

// Whether the tiles read the weights past the caches: more than the last level holds, 256 MB, and few row tiles read
// each (64 groups of 32 rows, 2048 x 7168, 470 MB: 97 -> 85 us; of 128: 118 -> 102; of 256: 158 -> 147; 48 of 200:
// 125 -> 115; 4 of 512, 18432 x 7168: 181 -> 177; of 2048: 526 -> 534).  Smaller weights may still be there from a
// call before (one group of 64 rows, 18432 x 7168, 66 MB: 16.5 -> 20.1, and 22.4 -> 21.5 where they are not).
bool stream_weights(const Mx4Args& a) {
  return (int64_t)a.G * a.N * (a.K / 2) > 256000000 && a.max_rows <= (int64_t)a.G * 512;
}

}  // namespace

// Groups of few rows: the ring, one pass over the weights, up to 12 rows on average (340 groups of 12 rows, 1264 x
// 928: 59 us, tiles 74; 384 of 8, 7168 x 2048: 511 and 585; 120 of 9, 1736 x 4480: 106 and 107; with 15 rows: 358
// groups, 960 x 3008: 178 and 135), of long sums up to 6 (384 of 4, 2048 x 7168: 443 and 440; of 12: 494 and 461),
// where it has 800 items, three for every two of its work-groups (31 groups, 31 rows, 3904 x 1344: 17.7 and 17.0; 19
// groups of 12 rows, 2176 x 3520, 561 items: 29 and 21).  Long sums and at most 128 tiles: the stream kernel, whose
// waves share a sum (8 groups of 4 rows, 2048 x 7168: 14.7, tiles 17.4; 24 of 8, 896 x 5632, 168 tiles: 19.7 and
// 15.7).  Otherwise tiles.
// One group: the stream kernel up to 8 rows (18432 x 7168: 16.3 us, tiles 15.0 with the weights in the cache, 18.7
// and 20.0 without; one row 13.9 and 15.0), or 2 where 128 columns make tiles for 0.7 of the CUs or more, in whole
// rounds (4 rows, 28672 x 4096, 224 tiles: 13.9 and 11.4, 14.9 and 13.9; 65536 x 4096, 512: 29.2 and 24.1, 31.8 and
// 27.2; one row 25.9 and 24.1, 28672 x 4096 13.3 and 13.8); up to 16 unless 128 columns make 128 tiles (16 rows,
// 18432 x 7168: 18.0 and 15.1; 12288 x 5120: 10.0 and 11.3); up to 64 unless they make 72 (32 rows, 18432 x 7168:
// 23.6 and 15.3; 9216 x 4096: 11.7 and 9.4; 8192 x 8192: 12.2 and 16.1; 64 rows, 7168 x 18432: 31 and 33), with
// 32-column items where 16-column ones would read the rows of x too often and enough of them remain (32 rows, 7168 x
// 18432: 30 us with 16, 21.4 with 32; 8 rows: 17.5 and 15.7, one: 14.5 and 14.9; 32 rows, 4096 x 14336: 13.4 and
// 17.0).
Mx4Plan mx4_plan(const Mx4Args& a, void* workspace) {
  Mx4Plan p{a, Mx4Kernel::kTile, {1, 1}, 0, "matmul_mx4_stream"};
  const int64_t rows = a.max_rows, columns = padded(a.N, 128) / 128;
  if (a.G > 1) {
    const int64_t items = mx4_ring_items(a);
    if (rows <= (int64_t)a.G * (a.K < 6144 ? 12 : 6) && items >= 800 && items <= (int64_t)1 << 30) {
      p.kernel = Mx4Kernel::kRing;
      p.name = "matmul_mx4_ring";
    } else if (rows <= (int64_t)a.G * 12 && a.G * columns <= 128 && a.K >= 2048) {
      p.kernel = Mx4Kernel::kStream;
    }
  } else if (const bool fill = columns * 10 >= padded(columns, 256) * 7;
             rows <= (fill ? 2 : 8) || (rows <= 16 && columns < 128) || (rows <= 64 && columns < 72)) {
    p.kernel = Mx4Kernel::kStream;
    p.stream.p_blocks = (int)std::max<int64_t>(1, (rows + 15) / 16);
    p.stream.q_blocks = rows > 4 && a.N >= 5120 ? 2 : 1;
  }
  if (p.kernel == Mx4Kernel::kTile) {
    p.tile_waves = tile_waves(a);
    p.name = p.tile_waves == 8 ? "matmul_mx4_tile256" : "matmul_mx4_tile128";
    p.pack = p.tile_waves == 8 && pack_scales(a);
    p.stream_w = !p.pack && stream_weights(a);
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
  if (p.kernel == Mx4Kernel::kTile) return launch_mx4_tile(p.args, p.tile_waves, p.stream_w, s);
  if (p.kernel == Mx4Kernel::kRing) return launch_mx4_ring(p.args, s);
  return launch_mx4_stream(p.args, p.stream, s);
}

}  // namespace moe

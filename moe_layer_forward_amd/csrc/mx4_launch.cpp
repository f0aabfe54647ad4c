// Which kernel a microscaled 4-bit product runs on.
#include <cstdlib>
#include <cstdio>
#include <algorithm>
#include "mx4.h"

namespace moe {
namespace {

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }

int tile_waves(const Mx4Args& a) {
  if (padded(a.N, 256) * 100 > padded(a.N, 128) * 115) return 4;
  const int64_t items = mx4_tile_grid(a, 8);
  return items >= 512 || (items >= 160 && a.K >= 12 * 256) ? 8 : 4;
}

}  // namespace

Mx4Plan mx4_plan(const Mx4Args& a, void*) {
  Mx4Plan p{a, Mx4Kernel::kStream, {4, 1, 8}, 8, "matmul_mx4_stream"};
  if (a.max_rows > (int64_t)a.G * 64) {
    p.kernel = Mx4Kernel::kTile;
    p.tile_waves = tile_waves(a);
    p.name = p.tile_waves == 8 ? "matmul_mx4_tile256" : "matmul_mx4_tile128";
    return p;
  }
  const int64_t mean = a.max_rows / a.G;
  if (a.G == 1) {
    p.stream.p_blocks = (int)std::max<int64_t>(1, (a.max_rows + 15) / 16);
    if (p.stream.p_blocks >= 3 && a.N >= 160 * 64) {
      p.kernel = Mx4Kernel::kTile;
      p.tile_waves = 4;
      p.name = "matmul_mx4_tile128";
    }
  } else if (mean > 24) {
    p.kernel = Mx4Kernel::kTile;
    p.tile_waves = 4;
    p.name = "matmul_mx4_tile128";
  } else {
    p.kernel = Mx4Kernel::kRing;
    p.stream = mean > 8 ? Mx4Stream{2, 1, 2} : Mx4Stream{1, 2, 2};
    p.name = "matmul_mx4_ring";
  }
  int t=0;
  if (const char* e = getenv("MXC")) sscanf(e, "%d/%d/%d/%d", &t, &p.stream.p_blocks, &p.stream.q_blocks, &p.stream.waves);
  if (t==1) p.kernel=Mx4Kernel::kRing;
  if (t>1) {p.kernel=Mx4Kernel::kTile;p.tile_waves=t;}
  return p;
}

size_t mx4_workspace(const Mx4Args&) { return 0; }

bool mx4_grid_ok(const Mx4Args& a) {
  const Mx4Plan p = mx4_plan(a, nullptr);
  const int64_t items = p.kernel == Mx4Kernel::kTile ? mx4_tile_grid(a, p.tile_waves)
                        : p.kernel == Mx4Kernel::kRing ? mx4_ring_items(a, p.stream.p_blocks, p.stream.q_blocks) : mx4_stream_grid(a, p.stream);
  return items <= (int64_t(1) << 31);
}

hipError_t launch_mx4(const Mx4Plan& p, hipStream_t s) {
  if (p.kernel == Mx4Kernel::kTile) return launch_mx4_tile(p.args, p.tile_waves, s);
  if (p.kernel == Mx4Kernel::kRing) return launch_mx4_ring(p.args, p.stream.p_blocks, p.stream.q_blocks, p.stream.waves, s);
  return launch_mx4_stream(p.args, p.stream, s);
}

}  // namespace moe

// Which kernel a microscaled 4-bit product runs on.
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
  Mx4Plan p{a, 0, 4, "matmul_mx4_stream64"};
  if (a.max_rows <= (int64_t)a.G * 12) {
    p.p_blocks = 1;
    p.name = "matmul_mx4_stream16";
  } else if (a.max_rows > (int64_t)a.G * 64) {
    p.waves = tile_waves(a);
    p.name = p.waves == 8 ? "matmul_mx4_tile256" : "matmul_mx4_tile128";
  }
  return p;
}

size_t mx4_workspace(const Mx4Args&) { return 0; }

bool mx4_grid_ok(const Mx4Args& a) {
  const Mx4Plan p = mx4_plan(a, nullptr);
  return (p.waves ? mx4_tile_grid(a, p.waves) : mx4_stream_grid(a, p.p_blocks)) <= (int64_t(1) << 31);
}

hipError_t launch_mx4(const Mx4Plan& p, hipStream_t s) {
  return p.waves ? launch_mx4_tile(p.args, p.waves, s) : launch_mx4_stream(p.args, p.p_blocks, s);
}

}  // namespace moe

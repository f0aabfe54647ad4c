// Which kernel a microscaled 4-bit product runs on.
#include "mx4.h"

namespace moe {

Mx4Plan mx4_plan(const Mx4Args& a, void*) {
  Mx4Plan p{a, 4, "matmul_mx4_stream64"};
  if (a.max_rows <= (int64_t)a.G * 12) {
    p.p_blocks = 1;
    p.name = "matmul_mx4_stream16";
  }
  return p;
}

size_t mx4_workspace(const Mx4Args&) { return 0; }

bool mx4_grid_ok(const Mx4Args& a) { return mx4_stream_grid(a, mx4_plan(a, nullptr).p_blocks) <= (int64_t(1) << 31); }

hipError_t launch_mx4(const Mx4Plan& p, hipStream_t s) { return launch_mx4_stream(p.args, p.p_blocks, s); }

}  // namespace moe

// Which kernel a grouped product runs on.
#include "kernels.h"

namespace moe {
namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The tile kernels move 16-byte pieces: operand rows start on 16 bytes and are multiples of 16 bytes long.
bool tile_ok(const GmmArgs& a) {
  if (a.type == GmmType::kF32) return false;
  const int e = a.type == GmmType::kI8 ? 1 : 2;
  if ((int64_t)a.K * e % 16) return false;
  if (a.form != GmmForm::kNT && (int64_t)a.N * e % 16) return false;
  return (a.form == GmmForm::kNN || aligned16(a.x)) && (a.form == GmmForm::kNT || aligned16(a.dy)) &&
         (a.form == GmmForm::kTN || aligned16(a.w));
}

}  // namespace

// Work-groups of 512 threads or fewer, a dealt grid at most twice the tiles.
bool gmm_grid_ok(const GmmArgs& a) { return 2 * 512 * gmm_any_grid(a) < (int64_t(1) << 32); }

size_t gmm_workspace(const GmmArgs&) { return 0; }

hipError_t launch_gmm(const GmmArgs& a, void*, hipStream_t s) {
  if (!tile_ok(a)) return launch_gmm_any(a, s);
  if (a.form == GmmForm::kNN) return launch_gmm_tile_nn(a, s);
  if (a.form == GmmForm::kTN) return launch_gmm_tile_tn(a, s);
  return a.type == GmmType::kI8 ? launch_gmm_tile_i8(a, s) : launch_gmm_tile_nt(a, s);
}

}  // namespace moe

// Which kernel a grouped product runs on, and into how many ranges its contraction is cut.
#include <algorithm>

#include "gmm.h"

namespace moe {
namespace {

constexpr int64_t kCus = 256;

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int elem_bytes(const GmmArgs& a) { return a.type == GmmType::kI8 ? 1 : a.type == GmmType::kBf16 ? 2 : 4; }

// The tile kernels move 16-byte pieces: operand rows are multiples of 16 bytes long ...
bool tile_sizes(const GmmArgs& a) {
  if (a.type == GmmType::kF32) return false;
  const int e = elem_bytes(a);
  return (int64_t)a.K * e % 16 == 0 && (a.form == GmmForm::kNT || (int64_t)a.N * e % 16 == 0);
}
// ... and start on 16 bytes.
bool tile_ok(const GmmArgs& a) {
  return tile_sizes(a) && (a.form == GmmForm::kNN || aligned16(a.x)) && (a.form == GmmForm::kNT || aligned16(a.dy)) &&
         (a.form == GmmForm::kTN || aligned16(a.w));
}

int64_t out_elems(const GmmArgs& a) {
  return a.form == GmmForm::kTN ? (int64_t)a.G * a.N * a.K : a.max_rows * (a.form == GmmForm::kNT ? a.N : a.K);
}

// Ranges of the contraction for `items` output tiles (an upper bound) of about `steps` steps each: as many as let
// `slots` work-groups run, while every range keeps min_steps steps.  Joining them costs another launch and the
// partial sums' traffic, so a few long sums are split and a chip that is half full is left alone.
int split_of(int64_t items, int64_t steps, int64_t slots, int64_t min_steps) {
  constexpr int64_t kMaxSplit = 16;
  if (items <= 0) return 1;
  return (int)std::max<int64_t>(1, std::min({slots / items, steps / min_steps, kMaxSplit}));
}

// Steps of a sum (TN: of the average group's).
int64_t steps_of(const GmmArgs& a) {
  const int64_t depth = a.form == GmmForm::kNT ? a.K : a.form == GmmForm::kNN ? a.N : a.max_rows / a.G;
  return (depth * elem_bytes(a) + 127) / 128;
}

// Small tiles where the large ones would leave slots (two on a CU) empty.
int any_tile(const GmmArgs& a) { return gmm_any_grid(a, 128) < 2 * kCus ? 64 : 128; }
// Three work-groups to a CU, ranges of 6 steps: fp32 sums are bound by the matrix cores of few CUs (9 groups, 777
// rows, 1001 x 515, 32 steps: 56 us in one range, 29 in four; 16 groups, 128 rows, 8 steps: 9 us in one, 13 in
// two).
int any_split(const GmmArgs& a) { return split_of(gmm_any_grid(a, any_tile(a)), steps_of(a), 3 * kCus, 6); }

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }

// Waves of the tile kernel's work-groups: 8 (256 x 256 tiles, one work-group to a CU) move half the bytes per
// product through LDS, 4 (128 x 128, two to a CU) waste less of a small matrix, fill the chip with fewer
// tiles and hide one another's starts and ends.  Measured over 90 drawn sizes: 8 waves win where there
// are 512 tiles or more, or 160 with sums of 12 steps or more (4 groups, 3045 rows, N = 2952, K = 4808: 116 us
// against 146), unless whole tiles pad the output more (two groups, 37557 rows, K = 104: 34 against 27) or
// groups have few rows (48 groups, 512 rows, int8: 150 against 140).
int tile_waves(const GmmArgs& a) {
  const int64_t q = a.form == GmmForm::kNT ? a.N : a.K, rows = a.max_rows / a.G;
  int64_t large = padded(q, 256), small = padded(q, 128);
  if (a.form == GmmForm::kTN) {
    large *= padded(a.N, 256);
    small *= padded(a.N, 128);
  }
  if (large * 100 > small * 115) return 4;
  if (a.form != GmmForm::kTN && rows < 32) return 4;
  const int64_t items = gmm_tile_items(a, 8);
  return items >= 512 || (items >= 160 && steps_of(a) >= 12) ? 8 : 4;
}
// One work-group to a CU, ranges of 8 steps (64 rows, 7168 x 7168: 39 us in one range, 25.5 in four, 30 in
// eight; int8, 64 rows, 18432 x 7168, 144 tiles: 24.6 us in one range, 35.5 in two).
int tile_split(const GmmArgs& a) { return split_of(gmm_tile_items(a, tile_waves(a)), steps_of(a), kCus, 8); }

}  // namespace

// Grids of at most 2^32 threads: the 64 x 64 tiles are the most work-groups (of 256 threads); the 256 x 256 ones
// (512 threads) are fewer even where their number is rounded up to twice.
bool gmm_grid_ok(const GmmArgs& a) { return 512 * gmm_any_grid(a, 64) < (int64_t(1) << 32); }

size_t gmm_workspace(const GmmArgs& a) {
  const int split = std::max(any_split(a), tile_sizes(a) ? tile_split(a) : 1);
  return split > 1 ? (size_t)split * out_elems(a) * sizeof(float) : 0;
}

hipError_t launch_gmm(const GmmArgs& args, void* workspace, hipStream_t s) {
  GmmArgs a = args;
  const bool tile = tile_ok(a);
  a.split = tile ? tile_split(a) : any_split(a);
  a.part = static_cast<float*>(workspace);
  const int waves = tile_waves(a);
  hipError_t e;
  if (!tile)
    e = launch_gmm_any(a, any_tile(a), s);
  else if (a.form == GmmForm::kNN)
    e = launch_gmm_tile_nn(a, waves, s);
  else if (a.form == GmmForm::kTN)
    e = launch_gmm_tile_tn(a, waves, s);
  else
    e = a.type == GmmType::kI8 ? launch_gmm_tile_i8(a, waves, s) : launch_gmm_tile_nt(a, waves, s);
  return e == hipSuccess && a.split > 1 ? launch_gmm_join(a, s) : e;
}

}  // namespace moe

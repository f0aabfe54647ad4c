// Which kernel a grouped product runs on, and into how many ranges its contraction is cut.
#include <algorithm>

#include "gmm.h"

namespace moe {
namespace {

constexpr int64_t kCus = 256;
constexpr int64_t kCacheBytes = 256 << 20;  // the last-level cache

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

// TN: rows of the ranges that a group's sum is cut into, 0: none cut.  One group's matrix is `tiles` output tiles;
// `slots` work-groups run.  Group sizes are known on the device alone, so the rule goes by their number and all rows, and
// a group that fits one range is written as if nothing was cut.  Ranges keep min_steps steps.
//   * Groups that leave slots idle: as many ranges as fill them, with 1/32 to spare, so that nearly equal groups have
//     equally many (without: 0.96 to 1.23 of the time, 1.01 over 24 sizes), and as many on every XCD where that leaves
//     out at most a quarter of them (rounded down always: up to 1.9, 3 groups, 48782 rows, 264 x 602 in bf16: 171 us
//     against 90; never: up to 1.17, 55 groups, 57305 rows, 108 x 28 in fp32: 50 against 42; 120 sizes).
//     10 groups, 12688 skewed rows, 1088 x 120 in bf16: 19 us, 29 with as many ranges to every group.
//   * Groups that fill the slots: ranges of twice the average group, for the one that holds more than others, where a
//     quarter of all rows in one sum would take half again as long as the rest and 8 steps more (an item's start
//     and end counted as 6 steps).  30 sizes, uncut -> cut: skewed by 1 / rank^1.1 all gain, 1.06 to 7.6 times (105
//     groups, 56522 rows, 118 x 134 in fp32: 935 -> 124 us); equal ones pay 2 to 5 us, the join's launch and its
//     search (285 groups, 17372 rows, 32 x 56 in bf16: 5.3 -> 8.4).  Without the condition: 130 groups, 8237 skewed
//     rows, 1280 x 576: 70 -> 80.
int64_t range_of(const GmmArgs& a, int64_t tiles, int64_t slots, int64_t min_steps) {
  const int64_t step = 128 / elem_bytes(a), steps = (a.max_rows + step - 1) / step, mean = (a.max_rows + a.G - 1) / a.G;
  int64_t each = std::min(slots / (tiles * a.G), mean / (min_steps * step));
  if (const int64_t e8 = each * a.G / 8 * 8 / a.G; e8 >= 2 && e8 * 4 >= each * 3) each = e8;  // the same on each XCD
  int64_t rows;
  if (each >= 2) {
    rows = (mean + each - 1) / each;
    if (a.G > 1) rows += rows / 32;
  } else {
    const int64_t others = tiles * a.G * (steps / a.G + 6) / slots;
    if (tiles * 2 > slots || steps / 4 <= others * 3 / 2 + 8) return 0;
    rows = std::max({2 * mean, a.max_rows * tiles / slots, min_steps * step});
  }
  rows = (rows + step - 1) / step * step;
  return rows < a.max_rows ? rows : 0;
}
int64_t matrix_tiles(const GmmArgs& a, int64_t tile) { return ((a.N + tile - 1) / tile) * ((a.K + tile - 1) / tile); }

// Steps of a sum (TN: of the average group's).
int64_t steps_of(const GmmArgs& a) {
  const int64_t depth = a.form == GmmForm::kNT ? a.K : a.form == GmmForm::kNN ? a.N : a.max_rows / a.G;
  return (depth * elem_bytes(a) + 127) / 128;
}

int64_t padded(int64_t n, int64_t tile) { return (n + tile - 1) / tile * tile; }

// Small tiles where the large ones would leave slots (two on a CU) empty, and where they pad the output by over 15%
// more, in fp32, which the matrix cores bound (72 groups, 50704 rows, 3608 -> 133: 735 us against 1009), and in the
// weight gradient, whose sums are short (358 groups, 4008 rows, 192 x 471 in bf16: 48 against 68).  Not for rows of
// bytes, which the loads bound (63951 rows, 6722 -> 320: 833 against 668).
int any_tile(const GmmArgs& a) {
  if (gmm_any_grid(a, 128) < 2 * kCus) return 64;
  if (a.type != GmmType::kF32 && a.form != GmmForm::kTN) return 128;
  const int64_t q = a.form == GmmForm::kNT ? a.N : a.K;
  int64_t large = padded(q, 128), small = padded(q, 64);
  if (a.form == GmmForm::kTN) {
    large *= padded(a.N, 128);
    small *= padded(a.N, 64);
  }
  return large * 100 > small * 115 ? 64 : 128;
}
// Three work-groups to a CU, ranges of 6 steps: fp32 sums are bound by the matrix cores of few CUs (9 groups, 777
// rows, 1001 x 515, 32 steps: 56 us in one range, 29 in four; 16 groups, 128 rows, 8 steps: 9 us in one, 13 in
// two).
int any_split(const GmmArgs& a) { return split_of(gmm_any_grid(a, any_tile(a)), steps_of(a), 3 * kCus, 6); }
int64_t any_range(const GmmArgs& a) { return range_of(a, matrix_tiles(a, any_tile(a)), 3 * kCus, 6); }


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
// One work-group to a CU, ranges of 8 steps (64 rows, 7168 x 7168: 37 us in one range, 24 in four, 27 in
// eight; int8, 64 rows, 18432 x 7168, 144 tiles: 24.6 us in one range, 35.5 in two).
int tile_split(const GmmArgs& a) { return split_of(gmm_tile_items(a, tile_waves(a)), steps_of(a), kCus, 8); }
int64_t tile_range(const GmmArgs& a) { return range_of(a, matrix_tiles(a, 32 * tile_waves(a)), kCus, 8); }

// Whether the kernel reads the weights of groups of one row tile, which nothing reads again, with the non-temporal
// policy: where tiles have room for the average group, where the weights exceed the 256 MB of last-level cache that
// a next call could find them in, and where their rows are whole 128-byte lines (a line that two steps or tiles share
// would be fetched twice).  Against the default policy, 18 to 20 sizes each, groups even, skewed by 1 / rank^1.1, and
// all rows in one:
//   as here: 0.88 to 0.97, 0.87 to 1.02, 1.00 to 1.01 (384 groups of 1.3 rows, 7168 x 2048: 1455 us -> 1306), but for
//     weights just past the cache (300 MB, 32 rows of 32 groups: 27.9 us -> 29.9)
//   rows of other lengths: 0.96 to 1.24 (61 groups, 3294 rows, 4560 x 2720 in int8: 200 us -> 248)
//   groups of several row tiles as well: skewed 0.91 to 1.12, all rows in one up to 1.49 (55 us -> 82)
//   132 MB of int8 weights, called again and again: 36 us -> 40
bool tile_once(const GmmArgs& a, int waves) {
  if ((int64_t)a.K * elem_bytes(a) % 128 || reinterpret_cast<uintptr_t>(a.w) % 128) return false;
  return a.form != GmmForm::kTN && a.max_rows <= (int64_t)a.G * 32 * waves &&
         (int64_t)a.G * a.N * a.K * elem_bytes(a) > kCacheBytes;
}

size_t range_bytes(const GmmArgs& a, int64_t range) {
  return range ? (size_t)(2 * ((a.max_rows + range - 1) / range)) * a.N * a.K * sizeof(float) : 0;
}

}  // namespace

// The 64 x 64 tiles are the most work-groups; the others are fewer even where their number is rounded up to twice.
bool gmm_grid_ok(const GmmArgs& a) { return gmm_any_grid(a, 64) <= (int64_t(1) << 31); }

size_t gmm_workspace(const GmmArgs& a) {
  if (a.form == GmmForm::kTN)
    return std::max(range_bytes(a, any_range(a)), tile_sizes(a) ? range_bytes(a, tile_range(a)) : 0);
  const int split = std::max(any_split(a), tile_sizes(a) ? tile_split(a) : 1);
  return split > 1 ? (size_t)split * out_elems(a) * sizeof(float) : 0;
}

GmmPlan gmm_plan(const GmmArgs& args, void* workspace) {
  static const char* const kNames[2][2] = {{"matmul_tile128", "matmul_tile128_nt"}, {"matmul_tile256", "matmul_tile256_nt"}};
  GmmPlan p{args, tile_ok(args), tile_waves(args), any_tile(args), false, false, nullptr};
  GmmArgs& a = p.args;
  a.part = static_cast<float*>(workspace);
  if (a.form == GmmForm::kTN)
    a.range_rows = p.tile ? tile_range(a) : any_range(a);
  else
    a.split = p.tile ? tile_split(a) : any_split(a);
  p.once = p.tile && tile_once(a, p.waves);
  p.join = a.split > 1 || a.range_rows;
  p.name = p.tile ? kNames[p.waves == 8][p.once] : p.edge == 64 ? "matmul_any64" : "matmul_any128";
  return p;
}

hipError_t launch_gmm(const GmmPlan& p, hipStream_t s) {
  const GmmArgs& a = p.args;
  if (!p.tile) return launch_gmm_any(a, p.edge, s);
  if (a.form == GmmForm::kNN) return launch_gmm_tile_nn(a, p.waves, p.once, s);
  if (a.form == GmmForm::kTN) return launch_gmm_tile_tn(a, p.waves, s);
  return a.type == GmmType::kI8 ? launch_gmm_tile_i8(a, p.waves, p.once, s) : launch_gmm_tile_nt(a, p.waves, p.once, s);
}

}  // namespace moe

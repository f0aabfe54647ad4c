// Launchers of the grouped matrix products and of the row quantizer.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// One product over groups of rows (forms and operands: gmm_core.h).  Sizes are W's: [G, N, K].
enum class GmmForm { kNT, kNN, kTN };  // y = x W^T, dx = dy W, dW = dy^T x
enum class GmmType { kF32, kBf16, kI8 };
struct GmmArgs {
  GmmForm form;
  GmmType type;
  int32_t G, N, K;
  const int32_t* group_offsets;  // [G+1] device, or null: one group of max_rows rows
  int64_t max_rows;
  const void* x;                 // NT, TN: rows of K
  int64_t x_rows;                // rows x has (gathers are kept inside them)
  const int32_t* row_index;      // NT, TN: x row of each row, or null
  const void* dy;                // NN, TN: rows of N
  const void* w;                 // NT, NN
  const float* x_scales;         // kI8: [x_rows]
  const float* w_scales;         // kI8: [G, N]
  void* out;
  int32_t out_bf16;
  // Set by gmm_plan.  NT, NN: the contraction cut into `split` ranges whose partial sums (fp32; int32 for kI8)
  // go to part, [split, output rows, output columns], for launch_gmm_join.
  int32_t split = 1;
  // TN: the rows of a group cut into ranges of range_rows (0: not cut); those of groups with more than one go to
  // part, [2 ceil(max_rows / range_rows), N, K] (gmm_core.h says where).
  int64_t range_rows = 0;
  float* part = nullptr;
};
// The sum over the ranges, in range order, scaled and rounded once into out.
hipError_t launch_gmm_join(const GmmArgs& a, hipStream_t s);
// The kernel that a product's sizes and alignment call for, and how its sums are split.
struct GmmPlan {
  GmmArgs args;      // with split, range_rows and part
  bool tile;         // the tile kernel, with work-groups of `waves`; or the plain one, with tiles of `edge`
  int waves, edge;
  bool once;         // tile: weights that are read once come with the non-temporal policy
  bool join;         // launch_gmm_join follows
  const char* name;  // of the kernel
};
GmmPlan gmm_plan(const GmmArgs& a, void* workspace);
hipError_t launch_gmm(const GmmPlan& p, hipStream_t s);
// The workspace bytes it needs (decided by type, form and sizes alone).
size_t gmm_workspace(const GmmArgs& a);
// A grid of n work-groups (n < 2^32) of up to 1024 threads: a launch takes fewer than 2^32 threads in each dimension, so
// those past kGmmGridX go to further rows of the grid.  A multiple of 8, so that work-group n still runs on XCD n % 8.
// The last row may have work-groups past n: kernels return for them.
constexpr unsigned kGmmGridX = 1u << 21;
inline dim3 gmm_grid(int64_t n) {
  return n <= kGmmGridX ? dim3((unsigned)n) : dim3(kGmmGridX, (unsigned)((n + kGmmGridX - 1) / kGmmGridX));
}
// Whether the work-groups of every kernel number fewer than 2^32.
bool gmm_grid_ok(const GmmArgs& a);
// Any sizes and any element alignment, in tiles of 64 x 64 or 128 x 128 (gmm_any_grid of them at most).
hipError_t launch_gmm_any(const GmmArgs& a, int tile, hipStream_t s);
int64_t gmm_any_grid(const GmmArgs& a, int tile);
// Tiles of 32 waves x 32 waves (waves 8 or 4 per work-group) on rows of whole 16-byte pieces (bf16; int8 for the
// forward); gmm_tile_items of them at most.
hipError_t launch_gmm_tile_nt(const GmmArgs& a, int waves, bool once, hipStream_t s);
hipError_t launch_gmm_tile_i8(const GmmArgs& a, int waves, bool once, hipStream_t s);
hipError_t launch_gmm_tile_nn(const GmmArgs& a, int waves, bool once, hipStream_t s);
hipError_t launch_gmm_tile_tn(const GmmArgs& a, int waves, hipStream_t s);
int64_t gmm_tile_items(const GmmArgs& a, int waves);

// codes[r] = rint(127 v / max|v|), scales[r] = max|v| / 127 of each row v (swiglu: v = SiLU(gate) * up of a
// row gate | up of 2 cols values).
hipError_t launch_quantize_rows(const void* x, bool x_bf16, int64_t rows, int64_t cols, bool swiglu, int8_t* codes,
                                float* scales, hipStream_t s);

}  // namespace moe

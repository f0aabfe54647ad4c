// Launchers of the microscaled 4-bit operators.
//
// A row of K values (K a multiple of 32) is K / 2 bytes of codes, two to a byte with the earlier value in the low
// half, and one scale byte s for every 32 of them: value = e2m1(code) 2^(s - 127), s = 255: NaN.  Rows of scales are
// padded to whole 16 bytes (512 values): what a work-group reads at a time.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

__host__ __device__ inline int mx4_scale_cols(int K) { return (K + 511) / 512 * 16; }

struct Mx4Args {
  int32_t G, N, K;
  const int32_t* group_offsets;  // [G + 1] device, or null: one group of max_rows rows
  int64_t max_rows;
  const uint8_t* x;              // codes [x_rows, K / 2]
  const uint8_t* xs;             // scales [x_rows, mx4_scale_cols(K)]
  int64_t x_rows;
  const int32_t* row_index;      // x row of each row, or null
  const uint8_t* w;              // [G, N, K / 2]
  const uint8_t* ws;             // [G, N, mx4_scale_cols(K)]
  void* out;
  int32_t out_bf16;
  uint8_t* packed = nullptr;     // tile kernel: the scales in the order of its reads (launch_mx4_pack), or null
};
// The stream kernel's items, 16 p_blocks (1 to 4) rows x 16 q_blocks (1 or 2) columns.
struct Mx4Stream {
  int p_blocks, q_blocks;
};
enum class Mx4Kernel { kStream, kRing, kTile };
// The kernel that a product's sizes call for.
struct Mx4Plan {
  Mx4Args args;
  Mx4Kernel kernel;
  Mx4Stream stream;
  int tile_waves;    // kTile: of a work-group
  const char* name;  // of the kernel
  bool pack = false;    // launch_mx4_pack comes first
  bool stream_w = false;  // kTile: the weights are read past the caches
};
Mx4Plan mx4_plan(const Mx4Args& a, void* workspace);
// The workspace bytes it needs (decided by sizes alone).
size_t mx4_workspace(const Mx4Args& a);
// Whether its work-groups number at most 2^31.
bool mx4_grid_ok(const Mx4Args& a);
hipError_t launch_mx4(const Mx4Plan& p, hipStream_t s);
hipError_t launch_mx4_stream(const Mx4Args& a, const Mx4Stream& c, hipStream_t s);
int64_t mx4_stream_grid(const Mx4Args& a, const Mx4Stream& c);
// Items of 16 rows x 128 columns; mx4_ring_items of them at most.
hipError_t launch_mx4_ring(const Mx4Args& a, hipStream_t s);
int64_t mx4_ring_items(const Mx4Args& a);
// stream: the weights are read past the caches (not with packed scales).
hipError_t launch_mx4_tile(const Mx4Args& a, int waves, bool stream, hipStream_t s);
int64_t mx4_tile_grid(const Mx4Args& a, int waves);
// Packs the scales of x and w for work-groups of 8 waves into a.packed, mx4_packed_bytes of it.
hipError_t launch_mx4_pack(const Mx4Args& a, hipStream_t s);
size_t mx4_packed_bytes(const Mx4Args& a);

hipError_t launch_quantize_mx4(const void* x, bool x_bf16, int64_t rows, int32_t cols, bool swiglu, uint8_t* codes,
                               uint8_t* scales, hipStream_t s);
hipError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* y,
                                 bool y_bf16, hipStream_t s);

}  // namespace moe

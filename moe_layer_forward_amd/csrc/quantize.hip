// Rows quantized to 8-bit integers with one scale per row: a = max |v|, scale = a / 127,
// code = rint(127 v / a) (ties to the even code), v the row itself or SiLU(gate) * up of a row that holds
// gate | up side by side.
//
// The quotient is the correctly rounded one of 127 v without a division per value (row_core.h).
// A row with an infinity or a NaN gets the scale NaN and codes 0, so that everything computed from it
// is NaN; a row of zeros gets the scale 0.
//
// Bound: HBM, each value read once: a row stays in registers between the maximum and the codes (16-byte loads
// of 8 values a lane, up to kHeld of them); only what is longer is read again.  Short rows are taken by
// one wave each (no barrier), long ones by four.  About 10 vector instructions a value (a division per value
// took 20 and bound the kernel: 8192 x 7168 bf16 rows in 50 us).
// Now 8192 x 7168: bf16 44 us (4.0 TB/s of reads and writes), fp32 54 us (5.5 TB/s); 65536 x 2048 bf16 79 us (5.1).
#include "row_core.h"

namespace moe {
namespace {

constexpr int kHeld = 8;  // chunks of 8 values a lane holds: 64 registers
constexpr int kQuantThreads = 256;

// kLanes lanes per row: 64 (a wave) or 256 (the work-group).
template <class In, bool kSwiglu, int kLanes>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(const In* x, int64_t rows, int64_t cols,
                                                                      int8_t* codes, float* scales) {
  const int lane = threadIdx.x % kLanes;
  const int64_t r = ((int64_t)blockIdx.y * kGmmGridX + blockIdx.x) * (kQuantThreads / kLanes) + threadIdx.x / kLanes;
  if (r >= rows) return;  // a whole wave or work-group
  const In* row = x + r * cols * (kSwiglu ? 2 : 1);
  float held[kHeld][8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int64_t c = 8 * ((int64_t)j * kLanes + lane);
    if (c < cols) {
      row_values<In, kSwiglu>(row, c, cols, held[j]);
      m = abs_bits_max(held[j], m);
    }
  }
  for (int64_t c = 8 * ((int64_t)kHeld * kLanes + lane); c < cols; c += 8 * kLanes) {
    float v[8];
    row_values<In, kSwiglu>(row, c, cols, v);
    m = abs_bits_max(v, m);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d, 64);
    m = o > m ? o : m;
  }
  if constexpr (kLanes > 64) {
    __shared__ uint32_t part[kLanes / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLanes / 64; ++i) m = part[i] > m ? part[i] : m;
  }
  const bool finite = m < 0x7f800000u;
  if (lane == 0) scales[r] = finite ? __fdiv_rn(__uint_as_float(m), 127.f) : __uint_as_float(0x7fc00000u);
  const RowScale rs = row_scale(finite ? m : 0u);
  int8_t* out = codes + r * cols;
  const auto put = [&](int64_t c, float(&v)[8]) {
    if (!finite) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    store_codes8(out + c, cols - c >= 8 ? 8 : (int)(cols - c), v, rs);
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int64_t c = 8 * ((int64_t)j * kLanes + lane);
    if (c < cols) put(c, held[j]);
  }
  for (int64_t c = 8 * ((int64_t)kHeld * kLanes + lane); c < cols; c += 8 * kLanes) {
    float v[8];
    row_values<In, kSwiglu>(row, c, cols, v);
    put(c, v);
  }
}

template <class In, bool kSwiglu>
hipError_t launch_q(const void* x, int64_t rows, int64_t cols, int8_t* codes, float* scales, hipStream_t s) {
  const In* p = static_cast<const In*>(x);
  if (cols <= 64 * 8 * kHeld / 2) {  // half the held chunks: a wave still has loads of several rows in flight
    const int64_t grid = (rows + kQuantThreads / 64 - 1) / (kQuantThreads / 64);
    quantize_rows_kernel<In, kSwiglu, 64><<<gmm_grid(grid), dim3(kQuantThreads), 0, s>>>(p, rows, cols, codes, scales);
  } else {
    quantize_rows_kernel<In, kSwiglu, kQuantThreads><<<gmm_grid(rows), dim3(kQuantThreads), 0, s>>>(p, rows, cols, codes,
                                                                                                   scales);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, bool x_bf16, int64_t rows, int64_t cols, bool swiglu, int8_t* codes,
                                float* scales, hipStream_t s) {
  if (x_bf16)
    return swiglu ? launch_q<uint16_t, true>(x, rows, cols, codes, scales, s)
                  : launch_q<uint16_t, false>(x, rows, cols, codes, scales, s);
  return swiglu ? launch_q<float, true>(x, rows, cols, codes, scales, s)
                : launch_q<float, false>(x, rows, cols, codes, scales, s);
}

}  // namespace moe

// Rows to microscaled 4 bits and back (layout: mx4.h).  A block of 32 values with a = max |v| gets the scale
// 2^X, X = max(floor(log2 a) - 2, -127), which brings a into [4, 8); a value's code is the nearest of
// +-{0, 1/2, 1, 3/2, 2, 3, 4, 6} to v 2^-X, ties to the even code, beyond 6 to 6 (v_cvt_scalef32_pk_fp4_f32: exact,
// since the scale is a power of two).  A block with an infinity or a NaN gets the scale 255 (NaN) and codes 0.
//
// Bound: HBM.  A wave takes 512 values of a row at a time, 8 a lane: four lanes share a block, and its codes and scales
// leave as 256 and 16 consecutive bytes.
#include "mx4.h"
#include "row_core.h"

namespace moe {
namespace {

constexpr int kMx4Threads = 256, kMx4Window = 512;

// Windows of 512 values, numbered row by row; `turns` consecutive ones to a wave.
struct Windows {
  int64_t row;
  int win;
  __device__ __forceinline__ Windows(int64_t first, int per_row) {
    row = first / per_row;
    win = (int)(first - row * per_row);
  }
  __device__ __forceinline__ void next(int per_row) {
    if (++win == per_row) {
      win = 0;
      ++row;
    }
  }
};

// max over the four lanes of a block
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true);  // lane ^ 1
  m = o > m ? o : m;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, true);  // lane ^ 2
  return o > m ? o : m;
}

template <class In, bool kSwiglu>
__global__ __launch_bounds__(kMx4Threads) void quantize_mx4_kernel(const In* x, int64_t rows, int cols, int per_row,
                                                                   int turns, uint8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = ((int64_t)blockIdx.y * kGmmGridX + blockIdx.x) * (kMx4Threads / 64) + (threadIdx.x >> 6);
  Windows at(wave * turns, per_row);
  for (int t = 0; t < turns; ++t, at.next(per_row)) {
    if (at.row >= rows) return;
    const int c = at.win * kMx4Window + 8 * lane;
    float v[8] = {};
    if (c < cols) row_values<In, kSwiglu>(x + at.row * cols * (kSwiglu ? 2 : 1), c, cols, v);
    const uint32_t m = quad_max(abs_bits_max(v, 0));
    const bool finite = m < 0x7f800000u;
    const uint32_t e = m >> 23, s = e > 2 ? e - 2 : 0;
    const float unit = __uint_as_float(s ? s << 23 : 0x00400000u);
    uint32_t q = 0;
    if (finite) {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], unit, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], unit, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], unit, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], unit, 3);
    }
    if (c < cols) __builtin_memcpy(codes + at.row * (cols / 2) + c / 2, &q, 4);
    if ((lane & 3) == 0)
      scales[(at.row * per_row + at.win) * 16 + lane / 4] = (uint8_t)(c >= cols ? 0 : finite ? s : 255);
  }
}

template <class Out>
__global__ __launch_bounds__(kMx4Threads) void dequantize_mx4_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                     int64_t rows, int cols, int per_row, int turns,
                                                                     Out* y) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = ((int64_t)blockIdx.y * kGmmGridX + blockIdx.x) * (kMx4Threads / 64) + (threadIdx.x >> 6);
  Windows at(wave * turns, per_row);
  for (int t = 0; t < turns; ++t, at.next(per_row)) {
    if (at.row >= rows) return;
    const int c = at.win * kMx4Window + 8 * lane;
    if (c >= cols) continue;
    uint32_t q;
    __builtin_memcpy(&q, codes + at.row * (cols / 2) + c / 2, 4);
    const uint32_t s = scales[(at.row * per_row + at.win) * 16 + lane / 4];
    const float unit = __uint_as_float(s == 255 ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // e2m1 -> fp32: exponent field 0 is the value m / 2
      const uint32_t code = q >> (4 * i) & 15, e = code >> 1 & 3, f = code & 1;
      const float mag = e ? __uint_as_float((126 + e) << 23 | f << 22) : 0.5f * f;
      v[i] = (code & 8 ? -mag : mag) * unit;
    }
    Out* to = y + at.row * cols + c;
    if constexpr (sizeof(Out) == 2) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
      __builtin_memcpy(to, u, 16);
    } else {
      __builtin_memcpy(to, v, 32);
    }
  }
}

struct Mx4Grid {
  int per_row, turns;
  dim3 grid;
  Mx4Grid(int64_t rows, int32_t cols) {
    per_row = mx4_scale_cols(cols) / 16;
    const int64_t windows = rows * per_row;
    turns = windows >= (int64_t)1 << 17 ? 4 : 1;
    const int64_t per = (int64_t)turns * (kMx4Threads / 64);
    grid = gmm_grid((windows + per - 1) / per);
  }
};

template <class In>
void launch_q(const Mx4Grid& g, const void* x, int64_t rows, int32_t cols, bool swiglu, uint8_t* codes, uint8_t* scales,
              hipStream_t s) {
  const In* p = static_cast<const In*>(x);
  if (swiglu) quantize_mx4_kernel<In, true><<<g.grid, kMx4Threads, 0, s>>>(p, rows, cols, g.per_row, g.turns, codes, scales);
  else quantize_mx4_kernel<In, false><<<g.grid, kMx4Threads, 0, s>>>(p, rows, cols, g.per_row, g.turns, codes, scales);
}

}  // namespace

hipError_t launch_quantize_mx4(const void* x, bool x_bf16, int64_t rows, int32_t cols, bool swiglu, uint8_t* codes,
                               uint8_t* scales, hipStream_t s) {
  const Mx4Grid g(rows, cols);
  if (x_bf16) launch_q<uint16_t>(g, x, rows, cols, swiglu, codes, scales, s);
  else launch_q<float>(g, x, rows, cols, swiglu, codes, scales, s);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* y,
                                 bool y_bf16, hipStream_t s) {
  const Mx4Grid g(rows, cols);
  if (y_bf16)
    dequantize_mx4_kernel<<<g.grid, kMx4Threads, 0, s>>>(codes, scales, rows, cols, g.per_row, g.turns,
                                                         static_cast<uint16_t*>(y));
  else
    dequantize_mx4_kernel<<<g.grid, kMx4Threads, 0, s>>>(codes, scales, rows, cols, g.per_row, g.turns,
                                                         static_cast<float*>(y));
  return hipGetLastError();
}

}  // namespace moe

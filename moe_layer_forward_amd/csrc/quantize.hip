// Rows quantized to 8-bit integers with one scale per row: a = max |v|, scale = a / 127,
// code = rint(127 v / a) (ties to the even code), v the row itself or SiLU(gate) * up of a row that holds
// gate | up side by side.
//
// The quotient is the correctly rounded one of 127 v (exact for bf16 values, so that the codes are
// those of the formula) without a division per value: with y = 1 / a correctly rounded, q0 = t y,
// r = t - q0 a (exact in one fused multiply-add) and q0 + r y rounds to the correctly rounded t / a (P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34,
// 1990).  Both sides are first scaled by a power of two that brings a into [1, 2), where nothing overflows.
// A row with an infinity or a NaN gets the scale NaN and codes 0, so that everything computed from it
// is NaN; a row of zeros gets the scale 0.
//
// Bound: HBM, each value read once: a row stays in registers between the maximum and the codes (16-byte loads
// of 8 values a lane, up to kHeld of them); only what is longer is read again.  Short rows are taken by
// one wave each (no barrier), long ones by four.  About 10 vector instructions a value (a division per value
// took 20 and bound the kernel: 8192 x 7168 bf16 rows in 50 us).
// Now 8192 x 7168: bf16 44 us (4.0 TB/s of reads and writes), fp32 54 us (5.5 TB/s); 65536 x 2048 bf16 79 us (5.1).
#include "gmm.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kHeld = 8;  // chunks of 8 values a lane holds: 64 registers
constexpr int kQuantThreads = 256;

template <class In>
__device__ __forceinline__ void load8(const In* p, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (sizeof(In) == 2) {
      uint32_t u[4];
      __builtin_memcpy(u, p, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      __builtin_memcpy(v, p, 32);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.f;
    if (i < n) {
      if constexpr (sizeof(In) == 2)
        v[i] = bf16_to_f32(p[i]);
      else
        v[i] = p[i];
    }
  }
}

// 8 values of the row from column c on (n of them exist)
template <class In, bool kSwiglu>
__device__ __forceinline__ void row_values(const In* row, int64_t c, int64_t cols, float (&v)[8]) {
  const int n = cols - c >= 8 ? 8 : (int)(cols - c);
  load8(row + c, n, v);
  if constexpr (kSwiglu) {
    float u[8];
    load8(row + cols + c, n, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = swiglu_f32(v[i], u[i]);
  }
}

__device__ __forceinline__ uint32_t abs_bits_max(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // as integers, infinity and NaN compare above every finite value
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}

// How a row's values become codes: t = (v s1) s2, code = t / a rounded.
struct RowScale {
  float s1, s2, a, y;
};

// m: bits of max |v|, finite.  v s1 s2 = 127 v 2^-e and a = max |v| 2^-e in [1, 2).
__device__ __forceinline__ RowScale row_scale(uint32_t m) {
  RowScale r;
  // max |v| below 2^-63 (subnormal ones too) or from 2^65 on: into the range where 2^-e is a normal number
  r.s1 = m < 0x20000000u ? 0x1p80f : m >= 0x60000000u ? 0x1p-64f : 1.f;
  const uint32_t b = __float_as_uint(__uint_as_float(m) * r.s1);
  const float down = __uint_as_float((254u << 23) - (b & 0x7f800000u));  // 2^-e
  r.a = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
  r.s2 = 127.f * down;
  r.y = __fdiv_rn(1.f, r.a);
  if (m == 0) {  // a row of zeros: codes 0
    r.s2 = 0.f;
    r.a = r.y = 1.f;
  }
  return r;
}

__device__ __forceinline__ void store8(int8_t* p, int n, const float (&v)[8], const RowScale& s) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = v[i] * s.s1 * s.s2;
    const float q0 = t * s.y;
    const float q = fmaf(fmaf(-q0, s.a, t), s.y, q0);
    u[i] = __float_as_uint(q + 12582912.f);  // 1.5 * 2^23: rounds to an integer, its low byte the code
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // low bytes of four words
    const uint32_t lo = __builtin_amdgcn_perm(u[4 * h + 1], u[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(u[4 * h + 3], u[4 * h + 2], 0x0c0c0400u);
    w[h] = lo | (hi << 16);
  }
  if (n >= 8) {
    __builtin_memcpy(p, w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

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
    store8(out + c, cols - c >= 8 ? 8 : (int)(cols - c), v, rs);
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

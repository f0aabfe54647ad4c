// Rows in chunks of 8 values a lane, at any alignment, and their 8-bit codes (quantize.hip, norm.hip,
// mx4_quantize.hip).
//
// The codes' quotient is the correctly rounded one of 127 v (exact for bf16 values, so that the codes are
// those of the formula) without a division per value: with y = 1 / a correctly rounded, q0 = t y,
// r = t - q0 a (exact in one fused multiply-add) and q0 + r y rounds to the correctly rounded t / a (P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34,
// 1990).  Both sides are first scaled by a power of two that brings a into [1, 2), where nothing overflows.
#pragma once
#include "gmm.h"
#include "kernels.h"

namespace moe {

// bf16 matrices from this size on are read, and written where nothing reads them next, with the non-temporal policy:
// they leave the last-level cache (256 MB) to others, and the stores do not wait for lines.  Norm, gradients: 56 MB
// 43.8 -> 42.7 us, 48.7 -> 52.8; 82 MB 66.7 -> 59.7, 76.2 -> 70.1; 224 MB 167 -> 160, 185 -> 168; 8192 x 7168 to
// 4-bit codes 28 -> 26, back 31 -> 24.  Not fp32, where a lane's 32 bytes are two halves of other lanes' lines: 128
// MB 99 -> 108.
constexpr int64_t kStreamBytes = 72 << 20;
template <class T>
inline bool row_streams(int64_t values) {
  return sizeof(T) == 2 && values * (int64_t)sizeof(T) >= kStreamBytes;
}

// 8 values as loaded; they are widened where they are used, so that nothing waits between the loads of a row.
template <class T>
struct Raw8 {
  uint32_t u[2 * sizeof(T)];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
  }
  // kNt: with the non-temporal policy
  typedef uint32_t Piece __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any element
  static constexpr int kPieces = sizeof(T) / 2;
  template <bool kNt = false>
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const Piece* at = reinterpret_cast<const Piece*>(p) + i;
      Piece v;
      if constexpr (kNt) v = __builtin_nontemporal_load(at);
      else v = *at;
#pragma unroll
      for (int j = 0; j < 4; ++j) u[4 * i + j] = v[j];
    }
  }
  template <bool kNt = false>
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      Piece* at = reinterpret_cast<Piece*>(p) + i;
      const Piece v = {u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]};
      if constexpr (kNt) __builtin_nontemporal_store(v, at);
      else *at = v;
    }
  }
  // from fp32, rounded once
  __device__ __forceinline__ void round(const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[i]);
    } else {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * i], v[2 * i + 1]}, bf16x2));
    }
  }
};

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

__device__ __forceinline__ void store_codes8(int8_t* p, int n, const float (&v)[8], const RowScale& s) {
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

}  // namespace moe

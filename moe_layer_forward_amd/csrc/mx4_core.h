// Building blocks of the microscaled 4-bit products: loads, the scaled matrix instruction, stores.
#pragma once
#include "gmm_items.h"
#include "mx4.h"
#include "tile_core.h"

namespace moe {

typedef __amdgpu_buffer_rsrc_t Mx4Rsrc;
constexpr uint32_t kMx4Outside = 0xfffffff0u;  // an offset past every record count: reads zeros

__device__ __forceinline__ Mx4Rsrc mx4_rsrc(const uint8_t* base, uint32_t records) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(gmm_uniform(reinterpret_cast<const char*>(base))), (short)0,
                                           gmm_uniform((int)records), 0x00020000);
}
__device__ __forceinline__ gmm_u32x4 mx4_load128(Mx4Rsrc r, uint32_t off) {
  return __builtin_bit_cast(gmm_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ uint32_t mx4_load32(Mx4Rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}

// c += q p^T over 128 values: lane l holds 32 of row l % 16 of each and their scale, byte TQ (TP) of sq (sp); lane l,
// element e of c is row l % 16 of p, row 4 (l / 16) + e of q.
template <int TQ, int TP>
__device__ __forceinline__ f32x4 mx4_mfma(gmm_u32x4 q, uint32_t sq, gmm_u32x4 p, uint32_t sp, f32x4 c) {
  typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 qv{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0}, pv{(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
  constexpr int kE2M1 = 4;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(qv, pv, c, kE2M1, kE2M1, TQ, (int)sq, TP, (int)sp);
}

// The bytes of four scales that belong to the `left` blocks a row still has: padding is not multiplied (a NaN there
// would reach the sum).
__device__ __forceinline__ uint32_t mx4_scale_mask(int left) {
  return left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
}

// The row of x that row r gathers, kept inside x.
__device__ __forceinline__ int64_t mx4_gathered(const Mx4Args& a, int64_t r) {
  const int64_t i = a.row_index[r];
  return i < 0 ? 0 : i >= a.x_rows ? a.x_rows - 1 : i;
}

// Up to four consecutive outputs (n of them exist), at any alignment.
__device__ __forceinline__ void mx4_store4(void* out, bool bf16, int64_t at, int n, f32x4 v) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    const uint32_t u[2] = {gmm_bf16x2(v[0], v[1]), gmm_bf16x2(v[2], v[3])};
    if (n >= 4) {
      __builtin_memcpy(p, u, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) p[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* p = static_cast<float*>(out) + at;
    if (n >= 4) {
      __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) p[e] = v[e];
    }
  }
}

}  // namespace moe

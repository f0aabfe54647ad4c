// Building blocks of the microscaled 4-bit products: loads, the scaled matrix instruction, stores.
#pragma once
#include "gmm_items.h"
#include "mx4.h"
#include "tile_core.h"

namespace moe {

typedef __amdgpu_buffer_rsrc_t Mx4Rsrc;
constexpr uint32_t kMx4Outside = 0xfffffff0u;  // an offset past every record count: reads zeros

__device__ __forceinline__ Mx4Rsrc mx4_rsrc(const uint8_t* base, uint32_t records) {
  const char* const at = gmm_uniform(reinterpret_cast<const char*>(base));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), (short)0, gmm_uniform((int)records), 0x00020000);
}
__device__ __forceinline__ gmm_u32x4 mx4_load128(Mx4Rsrc r, uint32_t off) {
  return __builtin_bit_cast(gmm_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// The row tiles of the groups, `tile` rows each: the full ones first, in the order of their groups, then every
// group's last, partial one, by their blocks of 32 rows, the longest first, so that the chip's last round is a short
// one (48 groups of 21 to 2118 rows, 2048 x 7168: 137 -> 133 us).  GmmTiles walks a lane's groups one by one; here
// the lanes' loads go out together and a tile is found in the registers, since with few rows the search is a good
// part of an item.  More than 512 groups go through GmmTiles, in the order of the groups.
struct Mx4Tiles {
  static constexpr int kHeld = 8;  // groups of a lane whose rows stay in registers: 512 in all
  static constexpr int kClasses = 8;  // blocks of 32 rows of a tile
  GmmTiles t;
  int n_full;  // of this lane's groups
  // partial tiles of class c (8 - blocks), 10 bits each: this lane's, and up to its end
  uint32_t n_part[3], part_to[3];
  int off[kHeld + 1];

  __device__ __forceinline__ static int scan(int v) {  // inclusive sum over the lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1, 2, 4, 8: rows of 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 to rows 2 and 3
    return v;
  }
  __device__ __forceinline__ static int clamp(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }
  __device__ __forceinline__ static int per_lane(const Mx4Args& a) { return (a.G + 63) / 64; }
  // The class of a partial tile of `rows` rows; kClasses of none.
  __device__ __forceinline__ static int part_class(int rows, int tile) { return kClasses - (rows % tile + 31) / 32; }

  __device__ __forceinline__ void count(const Mx4Args& a, int tile) {
    const int lane = threadIdx.x & 63, per = per_lane(a), most = (int)a.max_rows;
    if (!a.group_offsets) {
      t.full = most / tile;
      t.partial = most % tile != 0;
      return;
    }
    if (per > kHeld) return t.count(a.group_offsets, a.G, a.max_rows, tile);
#pragma unroll
    for (int j = 0; j <= kHeld; ++j) {  // as gmm_group_rows: inside [0, most], not decreasing
      const int at = lane * per + j;
      off[j] = j <= per ? a.group_offsets[at < a.G ? at : a.G] : 0;
    }
    n_full = 0;
    uint64_t lo = 0;  // classes 0 to 5
    uint32_t hi = 0;  // 6 and 7
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int b = clamp(off[j], 0, most), rows = clamp(off[j + 1], b, most) - b, c = part_class(rows, tile);
      const bool mine = j < per && lane * per + j < a.G;
      n_full += mine ? rows / tile : 0;
      lo += mine && c < 6 ? (uint64_t)1 << (c * 10 + (c >= 3 ? 2 : 0)) : 0;
      hi += mine && c >= 6 && c < kClasses ? 1u << (c - 6) * 10 : 0;
    }
    n_part[0] = (uint32_t)lo;
    n_part[1] = (uint32_t)(lo >> 32);
    n_part[2] = hi;
    t.full_to = scan(n_full);
    t.full = __builtin_amdgcn_readlane(t.full_to, 63);
    t.partial = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      part_to[i] = (uint32_t)scan((int)n_part[i]);
      const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)part_to[i], 63);
      t.partial += (int)((all & 1023) + (all >> 10 & 1023) + (all >> 20));
    }
  }

  // Tile t0 (below full + partial): rows [beg, end) of group g.
  __device__ __forceinline__ void find(const Mx4Args& a, int tile, int t0, int& g, int64_t& beg, int64_t& end) const {
    const int lane = threadIdx.x & 63, per = per_lane(a), most = (int)a.max_rows;
    if (!a.group_offsets) {
      g = 0;
      beg = (int64_t)t0 * tile;
      end = beg + tile < most ? beg + tile : most;
      return;
    }
    if (per > kHeld) {
      t.find(a.group_offsets, a.G, a.max_rows, tile, t0, g, beg, end);
      return;
    }
    const bool is_full = t0 < t.full;
    int rel = t0, to = t.full_to, n = n_full, cls = -1;
    if (!is_full) {
      rel -= t.full;
#pragma unroll
      for (int c = 0; c < kClasses; ++c) {
        const int sh = c % 3 * 10;
        const int of = (int)(part_to[c / 3] >> sh & 1023), all = __builtin_amdgcn_readlane(of, 63);
        if (cls < 0) {
          if (rel < all) {
            cls = c;
            to = of;
            n = (int)(n_part[c / 3] >> sh & 1023);
          } else {
            rel -= all;
          }
        }
      }
    }
    const int owner = __ffsll((unsigned long long)__ballot(to > rel)) - 1;
    int left = rel - (to - n), gj = 0, b = 0, e = 0;  // each lane among its own groups; the owner's are read
    bool found = false;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int bj = clamp(off[j], 0, most), ej = clamp(off[j + 1], bj, most), rows = ej - bj;
      const int k = j < per ? is_full ? rows / tile : part_class(rows, tile) == cls : 0;
      if (!found && left < k) {
        found = true;
        gj = lane * per + j;
        b = is_full ? bj + left * tile : bj + rows / tile * tile;
        e = is_full ? b + tile : ej;
      }
      left -= k;
    }
    g = __builtin_amdgcn_readlane(gj, owner);
    beg = __builtin_amdgcn_readlane(b, owner);
    end = __builtin_amdgcn_readlane(e, owner);
  }
};

// c += q p^T over 128 values: lane l holds 32 of row l % 16 of each and their scale, byte TQ (TP) of sq (sp); lane l,
// element e of c is row l % 16 of p, row 4 (l / 16) + e of q.
template <int TQ, int TP>
__device__ __forceinline__ f32x4 mx4_mfma(gmm_u32x4 q, uint32_t sq, gmm_u32x4 p, uint32_t sp, f32x4 c) {
  typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 qv{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
  const i32x8 pv{(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
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

// Building blocks of the grouped matrix products (gmm_any.hip, gmm_tile.hip): element types, LDS
// stages and fragments, and the mapping of row tiles to groups.
//
// The products, over groups of rows [off[g], off[g+1]) and weights W [G, N, K]:
//   NT  y[r, n]     = sum_k x[idx(r), k] W[g(r), n, k]     contraction K: contiguous in x and in W
//   NN  dx[r, k]    = sum_n dy[r, n] W[g(r), n, k]         contraction N: contiguous in dy, a row index of W
//   TN  dW[g, n, k] = sum_{r in g} dy[r, n] x[idx(r), k]   contraction r: a row index of both
//
// In every form the output tile is P rows x Q columns: the P operand gives the output's rows (x or dy
// rows; for TN the columns of dy), the Q operand its columns, which are contiguous in memory (W rows;
// for NN and TN the columns of W and of x).  One step of the contraction is 128 bytes of each operand
// row whatever the type: 64 bf16, 128 int8 or 32 fp32 values, so that one LDS stage, one 16-byte
// fragment read and one swizzle serve the three types:
//   * bf16: v_mfma_f32_16x16x32_bf16, lane l holds k = 8 (l / 16) .. + 7 of row l % 16
//   * int8: v_mfma_i32_16x16x64_i8, lane l holds k = 16 (l / 16) .. + 15 of row l % 16, exact int32 sums
//   * fp32: four v_mfma_f32_16x16x4_f32 (full fp32 products), the t-th taking element t of each lane's
//     four: k = 4 (l / 16) + t.  Both operands use the same order, so the sum is over the same k.
// The Q fragment is the MFMA's first operand, so lane l, element e of a 16 x 16 accumulator block is
// output row l % 16, column 4 (l / 16) + e: four consecutive columns per lane.
#pragma once
#include <type_traits>

#include "gmm.h"
#include "kernels.h"

namespace moe {

typedef uint32_t gmm_u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t gmm_i32x4 __attribute__((ext_vector_type(4)));

struct GmmBf16 {
  typedef f32x4 Acc;
  static constexpr int kBytes = 2;
  __device__ static __forceinline__ Acc mfma(gmm_u32x4 q, gmm_u32x4 p, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, q), __builtin_bit_cast(bf16x8, p), c, 0,
                                                   0, 0);
  }
};

struct GmmI8 {
  typedef gmm_i32x4 Acc;
  static constexpr int kBytes = 1;
  __device__ static __forceinline__ Acc mfma(gmm_u32x4 q, gmm_u32x4 p, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(gmm_i32x4, q), __builtin_bit_cast(gmm_i32x4, p), c,
                                                 0, 0, 0);
  }
};

struct GmmF32 {
  typedef f32x4 Acc;
  static constexpr int kBytes = 4;
  __device__ static __forceinline__ Acc mfma(gmm_u32x4 q, gmm_u32x4 p, Acc c) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(q[t]), __uint_as_float(p[t]), c, 0, 0, 0);
    return c;
  }
};

constexpr int kGmmStepBytes = 128;  // bytes of an operand row per contraction step

// Two fp32 values rounded to bf16 (nearest even), the first in the low half: one v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t gmm_bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// LDS stage of an operand whose rows run along the contraction: OUTER rows of 128 bytes, 16-byte chunk c
// of row r at c ^ ((r >> 1) & 7), so that the 16 rows of one fragment read fall in 16 bank groups.
template <class T, int OUTER>
struct GmmAlong {
  static constexpr bool kAlong = true;
  static constexpr int kChunks = 8;  // 16-byte chunks per row
  static constexpr int kRows = OUTER;
  static constexpr int kStageBytes = OUTER * kGmmStepBytes;
  __device__ static __forceinline__ int swz(int r) { return (r >> 1) & 7; }
  __device__ static __forceinline__ int pos(int r, int c) { return r * kGmmStepBytes + ((c ^ swz(r)) << 4); }
  // Per-lane byte offsets of a fragment read inside a 16-row block (block b at b * 2048).
  struct Lane {
    int off[2];
  };
  __device__ static __forceinline__ Lane lane() {
    const int l = threadIdx.x & 63, x = l & 15, g = l >> 4;
    return Lane{{pos(x, g), pos(x, 4 + g)}};
  }
};

// LDS stage of an operand whose rows run across the contraction: one row per contraction index (64 bf16
// or 32 fp32 of them), OUTER columns wide.
//   bf16: a fragment is two ds_read_b64_tr_b16.  Each transposes a 4 x 16 block per 16 lanes: lane i
//     names 4 columns (i % 4) of row i / 4 and receives column i of the 4 rows.  The 16 columns of a
//     block are one 32-byte unit; unit u of row r sits at u ^ s(r), s = (r & 3) | (r >> 1 & 4) (rows
//     of 128 bytes, two to a turn of the banks: (r >> 1 & 1) | (r >> 2 & 2)), so that the 8 rows x 32
//     bytes that 32 lanes read, rows 8 g + 0..3 for two g, fall in all 64 banks.
//   fp32: a fragment is four 4-byte reads (element t from row 4 (l / 16) + t); the 16 columns are one
//     64-byte unit, at u ^ (r >> 2 & 3), so that the four rows of one read fall in all 64 banks.
template <class T, int OUTER>
struct GmmAcross {
  static constexpr bool kAlong = false;
  static constexpr int kRows = kGmmStepBytes / T::kBytes;
  static constexpr int kRowBytes = OUTER * T::kBytes;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kStageBytes = kRows * kRowBytes;
  static constexpr int kUnit = 16 * T::kBytes;  // bytes of 16 columns
  static_assert((T::kBytes == 2 || T::kBytes == 4) && OUTER % 64 == 0, "types");
  __device__ static __forceinline__ int swz(int r) {
    if constexpr (T::kBytes == 4) return (r >> 2) & 3;
    return kRowBytes >= 256 ? (r & 3) | ((r >> 1) & 4) : ((r >> 1) & 1) | ((r >> 2) & 2);
  }
  // chunk that belongs at chunk position p of row r, and (the same involution) the position of chunk c
  __device__ static __forceinline__ int chunk_at(int r, int p) {
    constexpr int kSub = kUnit / 16;
    return ((p / kSub) ^ swz(r)) * kSub + p % kSub;
  }
  __device__ static __forceinline__ int pos(int r, int c) { return r * kRowBytes + (chunk_at(r, c) << 4); }
  struct Lane {
    int row;  // byte offset of the lane's first row, plus its place inside a unit
    int s;    // its swizzle
  };
  __device__ static __forceinline__ Lane lane() {
    const int l = threadIdx.x & 63, i = l & 15, g = l >> 4;
    if constexpr (T::kBytes == 2) {
      const int r = 8 * g + (i >> 2);
      return Lane{r * kRowBytes + (i & 3) * 8, swz(r)};
    } else {
      return Lane{4 * g * kRowBytes + i * 4, swz(4 * g)};
    }
  }
  // the fragment whose first row (of this lane) is at p
  __device__ static __forceinline__ gmm_u32x4 read_at(const char* p) {
    if constexpr (T::kBytes == 2) {
#if defined(__HIP_DEVICE_COMPILE__)
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) s16x4* Ptr;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(p)));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(p + 4 * kRowBytes)));
      return gmm_u32x4{lo[0], lo[1], hi[0], hi[1]};
#else
      return gmm_u32x4{};
#endif
    } else {
      gmm_u32x4 v;
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = *reinterpret_cast<const uint32_t*>(p + t * kRowBytes);
      return v;
    }
  }
};

template <GmmForm F, class T, int OUTER>
using GmmP = std::conditional_t<F == GmmForm::kTN, GmmAcross<T, OUTER>, GmmAlong<T, OUTER>>;
template <GmmForm F, class T, int OUTER>
using GmmQ = std::conditional_t<F == GmmForm::kNT, GmmAlong<T, OUTER>, GmmAcross<T, OUTER>>;

// A wave's fragment reads: block i of its blocks is 16-row block b0 + kStride i of the stage.
template <class L, int kStride>
struct GmmFrags {
  uint32_t off[L::kAlong ? 2 : 4];
  __device__ __forceinline__ void init(int b0) {
    const auto ln = L::lane();
    if constexpr (L::kAlong) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) off[kk] = (uint32_t)(b0 * 16 * kGmmStepBytes + ln.off[kk]);
    } else {  // (b0 + kStride m) below 8 per group of 8 units, so the swizzle stays inside it
#pragma unroll
      for (int m = 0; m < 4; ++m) off[m] = (uint32_t)(ln.row + ((b0 + kStride * m) ^ ln.s) * L::kUnit);
    }
  }
  __device__ __forceinline__ gmm_u32x4 read(const char* st, int i, int kk) const {
    if constexpr (L::kAlong)
      return *reinterpret_cast<const gmm_u32x4*>(st + off[kk] + i * kStride * 16 * kGmmStepBytes);
    else
      return L::read_at(st + off[i & 3] + (i >> 2) * 4 * kStride * L::kUnit + kk * (L::kRows / 2) * L::kRowBytes);
  }
};

// A value that every lane has, in scalar registers (the compiler cannot tell behind the lanes' search for the
// tile; a descriptor in vector registers costs a loop over the lanes per load).
__device__ __forceinline__ int gmm_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* gmm_uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = (uint32_t)gmm_uniform((int)v), hi = (uint32_t)gmm_uniform((int)(v >> 32));
  return reinterpret_cast<const char*>(lo | hi << 32);
}

// Rows [beg, end) of group g, kept inside [0, max_rows] whatever the offsets hold (null: one group of
// all rows).
__device__ __forceinline__ void gmm_group_rows(const int32_t* off, int64_t max_rows, int g, int64_t& beg,
                                               int64_t& end) {
  beg = off ? off[g] : 0;
  end = off ? off[g + 1] : max_rows;
  beg = beg < 0 ? 0 : beg > max_rows ? max_rows : beg;
  end = end < beg ? beg : end > max_rows ? max_rows : end;
}

// The row tiles of the groups, bm rows each: the full ones first (in group order), then every group's last,
// partial one.  Every wave of a work-group counts and finds them by itself: lane l sums over ceil(G / 64)
// consecutive groups, a scan over the lanes finds the lane, and the wave walks that lane's groups.  No
// plan launch and no workspace; G = 384 costs six loads per lane.
struct GmmTiles {
  int full = 0, partial = 0;        // tiles of the call
  int full_to = 0, partial_to = 0;  // up to and including this lane's groups
  int full_n = 0, partial_n = 0;    // of this lane's groups

  __device__ __forceinline__ void count(const int32_t* off, int G, int64_t max_rows, int bm) {
    const int lane = threadIdx.x & 63;
    const int per = (G + 63) / 64;
    for (int j = 0; j < per; ++j) {
      const int gg = lane * per + j;
      if (gg < G) {
        int64_t b, e;
        gmm_group_rows(off, max_rows, gg, b, e);
        const int rows = (int)(e - b);
        full_n += rows / bm;
        partial_n += rows % bm != 0;
      }
    }
    full_to = full_n;
    partial_to = partial_n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int f = __shfl_up(full_to, d, 64), p = __shfl_up(partial_to, d, 64);
      if (lane >= d) {
        full_to += f;
        partial_to += p;
      }
    }
    full = __builtin_amdgcn_readlane(full_to, 63);
    partial = __builtin_amdgcn_readlane(partial_to, 63);
  }

  // Tile t (below full + partial): its group and rows.  Returns the rows of the group.
  __device__ __forceinline__ int find(const int32_t* off, int G, int64_t max_rows, int bm, int t, int& g,
                                       int64_t& beg, int64_t& end) const {
    const bool is_full = t < full;
    int rel = is_full ? t : t - full;
    const int to = is_full ? full_to : partial_to, n = is_full ? full_n : partial_n;
    const int owner = __ffsll((unsigned long long)__ballot(to > rel)) - 1;
    rel -= __builtin_amdgcn_readlane(to - n, owner);
    const int per = (G + 63) / 64;
    g = owner * per;
    int64_t b, e;
    for (;; ++g) {  // ends inside this lane's groups, whose tiles number more than rel
      gmm_group_rows(off, max_rows, g, b, e);
      const int rows = (int)(e - b), k = is_full ? rows / bm : rows % bm != 0;
      if (rel < k || g + 1 >= G) break;
      rel -= k;
    }
    const int64_t rows = e - b;
    g = __builtin_amdgcn_readfirstlane(g);
    beg = is_full ? b + (int64_t)rel * bm : b + rows / bm * bm;
    end = is_full ? beg + bm : e;
    beg = __builtin_amdgcn_readfirstlane((int)beg);  // rows fit 31 bits
    end = __builtin_amdgcn_readfirstlane((int)end);
    return __builtin_amdgcn_readfirstlane((int)rows);
  }
};

// Work-group number of a grid of gmm_grid.
__device__ __forceinline__ unsigned gmm_block() { return blockIdx.y * kGmmGridX + blockIdx.x; }

// Share sp of nk contraction steps cut into `split` nearly equal ranges.
__device__ __forceinline__ void gmm_range(int nk, int split, int sp, int& first, int& n) {
  first = (int)((int64_t)nk * sp / split);
  n = (int)((int64_t)nk * (sp + 1) / split) - first;
}

// What a work-group of the TN form sums: rows [beg, end) of group g, all of them (whole) or one range of
// range_rows.  Sum t < G is group t's, or its first range; the further ranges of all groups follow in order, found as
// GmmTiles finds tiles.  The partial sums of full ranges go to the even places of part, those of a group's
// last, shorter one to the odd ones, numbered by where the range starts: two full ranges, and two last ones of
// groups that have a full one, start range_rows or more apart.
struct GmmSum {
  int g;
  int64_t beg, end;
  bool whole;

  // false past the last sum
  __device__ __forceinline__ bool find(const GmmArgs& a, int64_t t) {
    const int64_t range = a.range_rows;
    whole = true;
    if (t < a.G) {
      g = (int)t;
      gmm_group_rows(a.group_offsets, a.max_rows, g, beg, end);
      if (range && end - beg > range) {
        whole = false;
        end = beg + range;
      }
      return true;
    }
    if (!range) return false;
    const int lane = threadIdx.x & 63, per = (a.G + 63) / 64;
    const auto further = [&](int gg) {
      gmm_group_rows(a.group_offsets, a.max_rows, gg, beg, end);
      return end > beg ? (int)(end - beg - 1) / (int)range : 0;
    };
    int n = 0;
    for (int j = 0; j < per; ++j)
      if (lane * per + j < a.G) n += further(lane * per + j);
    int to = n, rel = (int)(t - a.G);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(to, d, 64);
      if (lane >= d) to += v;
    }
    if (rel >= __builtin_amdgcn_readlane(to, 63)) return false;
    const int owner = __ffsll((unsigned long long)__ballot(to > rel)) - 1;
    rel -= __builtin_amdgcn_readlane(to - n, owner);
    for (g = owner * per;; ++g) {  // ends inside this lane's groups, which have more than rel
      const int k = further(g);
      if (rel < k || g + 1 >= a.G) break;
      rel -= k;
    }
    whole = false;
    g = __builtin_amdgcn_readfirstlane(g);
    beg = __builtin_amdgcn_readfirstlane((int)(beg + (rel + 1) * range));
    end = __builtin_amdgcn_readfirstlane((int)end);
    end = end - beg > range ? beg + range : end;
    return true;
  }
  // its place in part
  __device__ __forceinline__ static int64_t place(int64_t beg, int64_t rows, int64_t range_rows) {
    return 2 * (beg / range_rows) + (rows < range_rows);
  }
  // first element of its matrix
  __device__ __forceinline__ char* matrix(const GmmArgs& a) const {
    const int64_t n = (int64_t)a.N * a.K;
    return whole ? static_cast<char*>(a.out) + g * n * (a.out_bf16 ? 2 : 4)
                 : reinterpret_cast<char*>(a.part + place(beg, end - beg, a.range_rows) * n);
  }
};

// Most sums that the groups have.
__host__ __device__ inline int64_t gmm_max_sums(const GmmArgs& a) { return a.G + (a.range_rows ? a.max_rows / a.range_rows : 0); }

// Most row tiles of bm rows that G groups over max_rows rows can have.
inline int64_t gmm_max_tiles(int64_t max_rows, int G, int bm) {
  const int64_t full = max_rows / bm + G;
  return full < max_rows ? full : max_rows;
}

}  // namespace moe

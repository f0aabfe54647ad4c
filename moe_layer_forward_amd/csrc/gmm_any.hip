// Grouped matrix products for any sizes, alignment and type: the kernel of the fp32 products and of rows
// that are not whole 16-byte pieces.
//
// Tile kTile x kTile (128 or 64), 4 waves in 2 x 2; a wave owns every other 16-row block of the P rows and half
// the Q columns (4 x 4 or 2 x 2 accumulator blocks), and skips the blocks that its group has no rows for.
// Both operands are read into registers two steps ahead, 16 bytes a lane at whatever alignment the rows
// have, with the ends of rows filled with zeros element by element, and stored into one of two LDS
// stages while the other is multiplied.  Contraction indices past the end are zero in both operands, so
// no neighbouring row's values, finite or not, enter a sum.  Outputs leave through LDS as 16-byte
// pieces of rows.  Two (128) or three (64) work-groups share a CU and hide one another's waits.
//
// Bound: fp32 by v_mfma_f32_16x16x4_f32 (256 FLOP a clock and CU): 53928 rows in 3 groups, 256 -> 3904, 1046 us, 103
// TFLOP/s; 65068 rows in 4 groups, dW 2560 x 1472, 106 (a library product of fp32 reaches 152).  Odd bf16 rows
// by the loads and their trip through registers; small calls by the latency of a step's loads.
// The branches around the ends of rows make the compiler wait for each load before the next branch, so a
// wave alone keeps few in flight.  Loads without branches (addresses kept inside the matrix, what does not
// belong masked on the way to LDS, two or four steps in flight) were measured over 32 drawn sizes: 7 to 23% faster
// on a few long sums, 5 to 15% slower on short ones, 1 to 3% slower over all; not kept.
#include <algorithm>

#include "gmm_core.h"

namespace moe {
namespace {

constexpr int kAnyThreads = 256;

// nv of the n elements at p (n = 16 bytes of them), zeros after them.  before: elements of the row in front of p; the
// last elements of a row of 16 bytes or more come from the 16 bytes that end with it, shifted down.
template <class T>
__device__ __forceinline__ gmm_u32x4 load_chunk(const char* p, int nv, int64_t before) {
  constexpr int kN = 16 / T::kBytes;
  gmm_u32x4 v = {0, 0, 0, 0};
  if (nv >= kN) {
    __builtin_memcpy(&v, p, 16);
  } else if (nv > 0) {
    const int drop = kN - nv;
    if (before >= drop) {
      unsigned __int128 u;
      __builtin_memcpy(&u, p - drop * T::kBytes, 16);
      v = __builtin_bit_cast(gmm_u32x4, u >> (8 * T::kBytes * drop));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (i < nv) {
          uint32_t u;
          if constexpr (T::kBytes == 1) u = *reinterpret_cast<const uint8_t*>(p + i);
          if constexpr (T::kBytes == 2) u = *reinterpret_cast<const uint16_t*>(p + 2 * i);
          if constexpr (T::kBytes == 4) u = *reinterpret_cast<const uint32_t*>(p + 4 * i);
          v[i * T::kBytes / 4] |= u << (8 * T::kBytes * (i % (4 / T::kBytes)));
        }
      }
    }
  }
  return v;
}

// One operand's share of a thread: kC chunks of a stage (kTile rows of 8 chunks over 256 threads).
// L = GmmAlong: chunk q is chunk q % 8 of tile row q / 8, whose elements run along the contraction.
// L = GmmAcross: chunk q is columns of contraction row q / kChunks.
template <class T, class L>
struct AnyOperand {
  static constexpr int kN = 16 / T::kBytes;
  static constexpr int kC = L::kStageBytes / 16 / kAnyThreads;
  const char* ptr[kC];      // Along: the chunk's row, at its chunk of step 0.  Across (not gathered): likewise
  int n;                    // Along: elements of the row from the chunk of step 0 on.  Across: of the columns
  int64_t before;           // elements of the row in front of the chunk (Along: of step 0)
  int have;                 // Along: bit j: the row of chunk j exists
  int64_t ld;               // Across: bytes between contraction rows
  int depth;                // Across: contraction rows
  const char* base;         // gathered Across: the matrix at the chunk's column
  const int32_t* index;
  int32_t index_last;

  // Along: rows [0, rows) of the tile, row r at base + row_of(r) * ld
  template <class RowOf>
  __device__ __forceinline__ void init_along(const char* b, int64_t ld_, int depth_, int rows, RowOf row_of) {
    const int c = (threadIdx.x % L::kChunks) * kN;  // 256 threads: the same chunk of each of the four rows
    n = depth_ - c;
    before = c;
    have = 0;
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int r = (threadIdx.x + kAnyThreads * j) / L::kChunks;
      ptr[j] = b + (r < rows ? row_of(r) : 0) * ld_ + c * T::kBytes;
      have |= (r < rows) << j;
    }
  }
  // Across: columns [col0, cols) of contraction rows [0, depth)
  __device__ __forceinline__ void init_across(const char* b, int64_t ld_, int depth_, int64_t col0, int64_t cols,
                                              const int32_t* index_, int64_t index_rows) {
    const int c = (threadIdx.x % L::kChunks) * kN;
    const int64_t left = cols - col0 - c;
    n = left > kN ? kN : (int)left;
    before = col0 + c;
    ld = ld_;
    depth = depth_;
    index = index_;
    index_last = (int32_t)index_rows - 1;
    base = b + (col0 + c) * T::kBytes;
#pragma unroll
    for (int j = 0; j < kC; ++j) ptr[j] = base + (int64_t)((threadIdx.x + kAnyThreads * j) / L::kChunks) * ld;
  }

  __device__ __forceinline__ void load(int kt, gmm_u32x4 (&v)[kC]) const {
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      v[j] = gmm_u32x4{0, 0, 0, 0};
      if constexpr (L::kAlong) {
        const int nv = (have >> j) & 1 ? n - kt * (kGmmStepBytes / T::kBytes) : 0;
        if (nv > 0) v[j] = load_chunk<T>(ptr[j] + (int64_t)kt * kGmmStepBytes, nv, before + kt * (kGmmStepBytes / T::kBytes));
      } else {
        const int r = kt * L::kRows + (threadIdx.x + kAnyThreads * j) / L::kChunks;
        if (r < depth && n > 0) {
          const char* p = ptr[j] + (int64_t)kt * L::kRows * ld;
          if (index) {
            int32_t i = index[r];
            i = i < 0 ? 0 : i > index_last ? index_last : i;
            p = base + (int64_t)i * ld;
          }
          v[j] = load_chunk<T>(p, n, before);
        }
      }
    }
  }
  __device__ static __forceinline__ void store(char* stage, const gmm_u32x4 (&v)[kC]) {
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int q = threadIdx.x + kAnyThreads * j;
      *reinterpret_cast<gmm_u32x4*>(stage + L::pos(q / L::kChunks, q % L::kChunks)) = v[j];
    }
  }
};

// TN: whether the ranges are shorter than the average group; the sums of the grid, then a multiple of 8 where they
// are many.
__host__ __device__ inline bool any_sums_first(const GmmArgs& a) {
  return a.range_rows && a.range_rows * a.G < a.max_rows;
}
__host__ __device__ inline int64_t any_sums(const GmmArgs& a) {
  const int64_t n = gmm_max_sums(a);
  return any_sums_first(a) && n >= 2 * kXcds ? (n + kXcds - 1) / kXcds * kXcds : n;
}

template <GmmForm F, class T, int kTile>
__global__ __launch_bounds__(kAnyThreads, kTile == 128 ? 2 : 4) void gmm_any_kernel(GmmArgs a) {
  using LP = GmmP<F, T, kTile>;
  using LQ = GmmQ<F, T, kTile>;
  constexpr int kAnyStage = kTile * kGmmStepBytes, kB = kTile / 32;  // 16-blocks of a wave's rows and columns
  constexpr int kOutRow = kTile * 4;                                 // bytes of a staged output row
  static_assert(LP::kStageBytes == kAnyStage && LQ::kStageBytes == kAnyStage, "stages");
  __shared__ __align__(16) char lds[4 * kAnyStage];  // P stages 0, 1, Q stages 0, 1; then the output tile

  // which tile: NT / NN a row tile of a group x a column slab, TN a (group, n tile, k tile); which range
  const int64_t q_len = F == GmmForm::kNT ? a.N : a.K;
  const int q_tiles = (int)((q_len + kTile - 1) / kTile);
  const int sp = (int)(gmm_block() % (unsigned)a.split);
  int64_t item = gmm_block() / (unsigned)a.split;
  if constexpr (F == GmmForm::kTN) {
    // Where every group is cut, consecutive work-groups take different sums: the tiles of one read the same rows,
    // and so fall on few XCDs (work-group b runs on XCD b % 8), whose L2 hold them.
    if (any_sums_first(a)) {
      const int64_t tiles = ((int64_t)a.N + kTile - 1) / kTile * q_tiles, sums = any_sums(a);
      item = item % sums * tiles + item / sums;
    }
  }
  const int64_t t = item / q_tiles;
  const int64_t q0 = (item % q_tiles) * kTile;
  int g;
  int64_t beg, end, p0 = 0;
  [[maybe_unused]] GmmSum sum;
  if constexpr (F == GmmForm::kTN) {
    const int64_t p_tiles = ((int64_t)a.N + kTile - 1) / kTile;
    if (!sum.find(a, t / p_tiles)) return;
    p0 = (t % p_tiles) * kTile;
    g = sum.g;
    beg = sum.beg;
    end = sum.end;
  } else {
    GmmTiles tiles;
    tiles.count(a.group_offsets, a.G, a.max_rows, kTile);
    if (t >= tiles.full + tiles.partial) return;
    tiles.find(a.group_offsets, a.G, a.max_rows, kTile, (int)t, g, beg, end);
  }
  // output rows of this tile (TN: columns of dy, rows of dW[g])
  const int rows = (int)(F == GmmForm::kTN ? (a.N - p0 < kTile ? a.N - p0 : kTile) : end - beg);
  const int cols = (int)(q_len - q0 < kTile ? q_len - q0 : kTile);
  const int64_t ldn = (int64_t)a.N * T::kBytes, ldk = (int64_t)a.K * T::kBytes;
  const char* w = static_cast<const char*>(a.w);
  if (F != GmmForm::kTN) w += (int64_t)g * a.N * ldk;
  const auto x_row = [&](int r) -> int64_t {
    if (!a.row_index) return beg + r;
    const int64_t i = a.row_index[beg + r];
    return i < 0 ? 0 : i >= a.x_rows ? a.x_rows - 1 : i;
  };

  AnyOperand<T, LP> p;
  AnyOperand<T, LQ> q;
  int depth;
  if constexpr (F == GmmForm::kNT) {
    depth = a.K;
    p.init_along(static_cast<const char*>(a.x), ldk, depth, rows, x_row);
    q.init_along(w + q0 * ldk, ldk, depth, cols, [](int r) -> int64_t { return r; });
  } else if constexpr (F == GmmForm::kNN) {
    depth = a.N;
    p.init_along(static_cast<const char*>(a.dy) + beg * ldn, ldn, depth, rows, [](int r) -> int64_t { return r; });
    q.init_across(w, ldk, depth, q0, a.K, nullptr, 0);
  } else {
    depth = (int)(end - beg);
    p.init_across(static_cast<const char*>(a.dy) + beg * ldn, ldn, depth, p0, a.N, nullptr, 0);
    q.init_across(static_cast<const char*>(a.x) + (a.row_index ? 0 : beg * ldk), ldk, depth, q0, a.K,
                  a.row_index ? a.row_index + beg : nullptr, a.x_rows);
  }

  const int lane = threadIdx.x & 63, wave = gmm_uniform(threadIdx.x >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  const int blocks = gmm_uniform((rows + 15) / 16);
  GmmFrags<LP, 2> fp;
  fp.init(wr);
  GmmFrags<LQ, 1> fq;
  fq.init(kB * wc);
  typename T::Acc acc[kB][kB];
#pragma unroll
  for (int i = 0; i < kB; ++i)
#pragma unroll
    for (int s = 0; s < kB; ++s) acc[i][s] = typename T::Acc{0, 0, 0, 0};

  constexpr int kStep = kGmmStepBytes / T::kBytes;
  int first, nk;
  gmm_range(gmm_uniform((depth + kStep - 1) / kStep), a.split, sp, first, nk);
  using OP = AnyOperand<T, LP>;
  using OQ = AnyOperand<T, LQ>;
  gmm_u32x4 pv[2][OP::kC], qv[2][OQ::kC];  // steps kt + 1 and kt + 2, by parity of the step
  if (nk > 0) {
    p.load(first, pv[0]);
    q.load(first, qv[0]);
  }
  if (nk > 1) {
    p.load(first + 1, pv[1]);
    q.load(first + 1, qv[1]);
  }
  if (nk > 0) {
    OP::store(lds, pv[0]);
    OQ::store(lds + 2 * kAnyStage, qv[0]);
  }
  __syncthreads();
  const auto step = [&](int kt, auto parity) {
    constexpr int cur = decltype(parity)::value;
    const char *ps = lds + cur * kAnyStage, *qs = lds + (2 + cur) * kAnyStage;
    if (kt + 2 < nk) {
      p.load(first + kt + 2, pv[cur]);
      q.load(first + kt + 2, qv[cur]);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      gmm_u32x4 qf[kB];
#pragma unroll
      for (int s = 0; s < kB; ++s) qf[s] = fq.read(qs, s, kk);
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        if (wr + 2 * i < blocks) {
          const gmm_u32x4 pf = fp.read(ps, i, kk);
#pragma unroll
          for (int s = 0; s < kB; ++s) acc[i][s] = T::mfma(qf[s], pf, acc[i][s]);
        }
      }
    }
    if (kt + 1 < nk) {
      OP::store(lds + (cur ^ 1) * kAnyStage, pv[cur ^ 1]);
      OQ::store(lds + (2 + (cur ^ 1)) * kAnyStage, qv[cur ^ 1]);
    }
    __syncthreads();
  };
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, std::integral_constant<int, 0>{});
    if (kt + 1 < nk) step(kt + 1, std::integral_constant<int, 1>{});
  }

  // The output tile through LDS, as fp32 (int32 partial sums as they are): row r of kOutRow bytes, its
  // 16-byte piece c at c ^ (r & 15); the last barrier above freed the stages.
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const int r = 16 * (wr + 2 * i) + (lane & 15);
    if (wr + 2 * i < blocks) {
      float sx = 1.f;
      if constexpr (std::is_same_v<T, GmmI8>)
        if (a.split == 1) sx = a.x_scales[x_row(r < rows ? r : rows - 1)];
#pragma unroll
      for (int s = 0; s < kB; ++s) {
        const int col = 16 * (kB * wc + s) + 4 * (lane >> 4);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (std::is_same_v<T, GmmI8>) {
            const int c = col + e < cols ? col + e : cols - 1;
            v[e] = a.split == 1 ? (float)acc[i][s][e] * sx * a.w_scales[(int64_t)g * a.N + q0 + c]
                                : __int_as_float(acc[i][s][e]);
          } else {
            v[e] = acc[i][s][e];
          }
        }
        *reinterpret_cast<f32x4*>(lds + r * kOutRow + (((col >> 2) ^ (r & 15)) << 4)) = v;
      }
    }
  }
  __syncthreads();
  const bool whole = F == GmmForm::kTN ? sum.whole : a.split == 1, bf16 = whole && a.out_bf16;
  char* out = F == GmmForm::kTN ? sum.matrix(a)
              : whole           ? static_cast<char*>(a.out)
                                : reinterpret_cast<char*>(a.part + sp * a.max_rows * q_len);
  out += ((F == GmmForm::kTN ? p0 : beg) * q_len + q0) * (bf16 ? 2 : 4);
  // 8 columns a thread, at the alignment that the row has
  for (int ch = threadIdx.x; ch < rows * (kTile / 8); ch += kAnyThreads) {
    const int r = ch / (kTile / 8), c = (ch % (kTile / 8)) * 8;
    if (c >= cols) continue;
    f32x4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = *reinterpret_cast<const f32x4*>(lds + r * kOutRow + (((c / 4 + h) ^ (r & 15)) << 4));
    const int n = cols - c;
    if (bf16) {
      const uint32_t h[4] = {gmm_bf16x2(v[0][0], v[0][1]), gmm_bf16x2(v[0][2], v[0][3]), gmm_bf16x2(v[1][0], v[1][1]),
                             gmm_bf16x2(v[1][2], v[1][3])};
      char* o = out + ((int64_t)r * q_len + c) * 2;
      if (n >= 8) {
        __builtin_memcpy(o, h, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
      }
    } else {
      char* o = out + ((int64_t)r * q_len + c) * 4;
      if (n >= 8) {
        __builtin_memcpy(o, v, 32);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) reinterpret_cast<float*>(o)[e] = v[e >> 2][e & 3];
      }
    }
  }
}

// 4 (or n) values of out from element i on, rounded once
__device__ __forceinline__ void store_sums(const GmmArgs& a, int64_t i, int n, const float (&sum)[4]) {
  if (a.out_bf16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + i;
    const uint32_t h[2] = {gmm_bf16x2(sum[0], sum[1]), gmm_bf16x2(sum[2], sum[3])};
    if (n == 4) {
      __builtin_memcpy(o, h, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) o[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* o = static_cast<float*>(a.out) + i;
    if (n == 4) {
      __builtin_memcpy(o, sum, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) o[e] = sum[e];
    }
  }
}

// NT, NN: out = the sum over the ranges of part, in range order; one work-group per 1024 columns of a row.
template <GmmForm F, bool kI8>
__global__ __launch_bounds__(256) void gmm_join_kernel(GmmArgs a) {
  const int64_t q_len = F == GmmForm::kNT ? a.N : a.K;
  const int per_row = (int)((q_len + 1023) / 1024);
  const int64_t row = blockIdx.x / per_row;
  const int64_t col = (int64_t)(blockIdx.x % per_row) * 1024 + threadIdx.x * 4;
  if (a.group_offsets) {  // rows past the last group have no sums
    int64_t beg, end;
    gmm_group_rows(a.group_offsets, a.max_rows, a.G - 1, beg, end);
    if (row >= end) return;
  }
  const int n = q_len - col < 4 ? (int)(q_len - col) : 4;
  if (n <= 0) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int isum[4] = {0, 0, 0, 0};
  const float* p = a.part + row * q_len + col;
  for (int s = 0; s < a.split; ++s, p += a.max_rows * q_len) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (n == 4) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) v[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kI8)
        isum[e] += __float_as_int(v[e]);
      else
        sum[e] += v[e];
    }
  }
  if constexpr (kI8) {
    int64_t i = row;
    if (a.row_index) {
      i = a.row_index[row];
      i = i < 0 ? 0 : i >= a.x_rows ? a.x_rows - 1 : i;
    }
    int g = 0;  // the row's group: the first whose end is past it
    if (a.group_offsets) {
      int hi = a.G - 1;
      while (g < hi) {
        const int mid = (g + hi) / 2;
        if (a.group_offsets[mid + 1] > row)
          hi = mid;
        else
          g = mid + 1;
      }
    }
    const float sx = a.x_scales[i];
    const float* sw = a.w_scales + (int64_t)g * a.N + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = (float)isum[e] * sx * (e < n ? sw[e] : 0.f);
  }
  store_sums(a, row * q_len + col, n, sum);
}

// TN: the same for the groups of more than one range; one work-group per `share` elements of a group's matrix.
// Where groups are more than further ranges can be, a group is found by its second range, and work-groups of
// other ranges do nothing.  Very many of those cost equal groups more than longer joins cost skewed ones.  Shares of
// 4096 elements against 1024, 60 sizes, groups equal and skewed by 1 / rank^1.1 (time of the whole call):
//   8192 work-groups of 1024 elements or more: equal 0.89 to 1.00, skewed 0.98 to 1.04 (152 groups, 94200 rows,
//     1152 x 184 in bf16: equal 93.5 us -> 83.9, skewed 134 -> 139)
//   fewer: equal 0.90 to 1.01, skewed 1.00 to 2.0 (394 groups, 41681 rows, 40 x 96 in fp32: equal 18.4 us, skewed 42.0 ->
//     85.4; 159 groups, 13065 rows, 408 x 240: equal 74.6 -> 68.5, skewed 83.9 -> 100.3)
//   groups not searched for (no work-group idles): 1.04 to 2.8
__global__ __launch_bounds__(256) void gmm_join_sums_kernel(GmmArgs a, int per_matrix, int share) {
  const int64_t range = a.range_rows;
  int g = (int)(blockIdx.x / (unsigned)per_matrix);
  int64_t b, e, second = -1;
  if (a.G > a.max_rows / range) {
    GmmSum sum;
    if (!sum.find(a, (int64_t)a.G + g)) return;
    g = sum.g;
    second = sum.beg;
  }
  gmm_group_rows(a.group_offsets, a.max_rows, g, b, e);
  if (second >= 0 ? second != b + range : e - b <= range) return;
  const int64_t all = (int64_t)a.N * a.K;
  const int64_t first = (int64_t)(blockIdx.x % (unsigned)per_matrix) * share;
  for (int64_t i = first + threadIdx.x * 4; i < first + share && i < all; i += 1024) {
    const int n = all - i < 4 ? (int)(all - i) : 4;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int64_t r = b; r < e; r += range) {
      const float* p = a.part + GmmSum::place(r, e - r, range) * all + i;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (n == 4) {
        __builtin_memcpy(v, p, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) v[j] = p[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += v[j];
    }
    store_sums(a, g * all + i, n, sum);
  }
}

template <GmmForm F, class T>
hipError_t launch_any(const GmmArgs& a, int tile, hipStream_t s) {
  const dim3 grid = gmm_grid(gmm_any_grid(a, tile) * a.split), block(kAnyThreads);
  if (tile == 64)
    gmm_any_kernel<F, T, 64><<<grid, block, 0, s>>>(a);
  else
    gmm_any_kernel<F, T, 128><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t gmm_any_grid(const GmmArgs& a, int tile) {
  const int64_t q_tiles = ((a.form == GmmForm::kNT ? a.N : a.K) + tile - 1) / tile;
  const int64_t p_tiles = a.form == GmmForm::kTN ? any_sums(a) * ((a.N + tile - 1) / tile)
                                                 : gmm_max_tiles(a.max_rows, a.G, tile);
  return p_tiles * q_tiles;
}

hipError_t launch_gmm_any(const GmmArgs& a, int tile, hipStream_t s) {
  switch (a.form) {
    case GmmForm::kNT:
      if (a.type == GmmType::kI8) return launch_any<GmmForm::kNT, GmmI8>(a, tile, s);
      return a.type == GmmType::kBf16 ? launch_any<GmmForm::kNT, GmmBf16>(a, tile, s)
                                      : launch_any<GmmForm::kNT, GmmF32>(a, tile, s);
    case GmmForm::kNN:
      return a.type == GmmType::kBf16 ? launch_any<GmmForm::kNN, GmmBf16>(a, tile, s)
                                      : launch_any<GmmForm::kNN, GmmF32>(a, tile, s);
    default:
      return a.type == GmmType::kBf16 ? launch_any<GmmForm::kTN, GmmBf16>(a, tile, s)
                                      : launch_any<GmmForm::kTN, GmmF32>(a, tile, s);
  }
}

hipError_t launch_gmm_join(const GmmArgs& a, hipStream_t s) {
  const dim3 block(256);
  if (a.form == GmmForm::kTN) {
    const int64_t further = a.max_rows / a.range_rows;
    const int64_t all = (int64_t)a.N * a.K, turns = std::min<int64_t>(a.G, further);
    const int share = a.G > further && turns * all >= 8192 * 1024 ? 4096 : 1024;
    const int per_matrix = (int)((all + share - 1) / share);
    gmm_join_sums_kernel<<<dim3((unsigned)(turns * per_matrix)), block, 0, s>>>(a, per_matrix, share);
    return hipGetLastError();
  }
  const int64_t q_len = a.form == GmmForm::kNT ? a.N : a.K;
  const dim3 grid((unsigned)(a.max_rows * ((q_len + 1023) / 1024)));
  if (a.type == GmmType::kI8)
    gmm_join_kernel<GmmForm::kNT, true><<<grid, block, 0, s>>>(a);
  else if (a.form == GmmForm::kNT)
    gmm_join_kernel<GmmForm::kNT, false><<<grid, block, 0, s>>>(a);
  else
    gmm_join_kernel<GmmForm::kNN, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe

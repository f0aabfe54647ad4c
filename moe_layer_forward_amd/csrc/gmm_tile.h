// Tile kernel of the grouped matrix products (bf16 and int8): rows that are multiples of 16 bytes from
// 16-byte boundaries.  Forms, types and LDS stages: gmm_core.h.
//
// Work item = 256 (P) x 256 (Q) outputs of one group, 8 waves in 2 x 4; a wave owns every other 16-row
// block of the P rows and 64 Q columns (at most 8 x 4 accumulator blocks, 128 registers).
//   * Both operands go straight from memory to LDS (buffer_load_dwordx4 ... lds), one instruction 1 KiB:
//     8 rows of 128 bytes (rows along the contraction) or 2 rows of 512 bytes (across it).  Two stages of
//     P and three of Q, 5 x 32 KiB, each its own __shared__ array and the loop unrolled by six, so that
//     every access names its stage and the compiler's own waits stay exact.  P is loaded one step
//     ahead, Q two.
//   * Ends: a chunk past the end of a row gets an offset past the descriptor's record count, a
//     contraction row past the end lies past the count itself; both put zeros into LDS and read nothing.
//     So the sums see zeros past the end on both sides, never a neighbour's values.  P rows and Q columns
//     past the tile's end hold whatever is there and are not stored.
//   * The loop is instantiated per number of P blocks a wave multiplies, so that rows a group does not
//     have cost no products and no loads.
//   * Outputs are staged in LDS and leave as 16-byte pieces of whole rows.
#pragma once
#include "gmm_core.h"
#include "tile_core.h"

namespace moe {
namespace {

constexpr int kGmmTile = 256;
constexpr int kGmmThreads = 512, kGmmWaves = 8;
constexpr int kGmmStage = 32 * 1024;
constexpr int kGmmLoads = 4;        // 1 KiB loads per wave, operand and step
constexpr uint32_t kGmmOutside = 0xfffffff0u;  // an offset past every record count
constexpr int kGmmSuper = 4;        // row tiles that run side by side on one XCD

typedef __amdgpu_buffer_rsrc_t GmmRsrc;
typedef __attribute__((address_space(3))) void* GmmLds;

__device__ __forceinline__ GmmRsrc gmm_rsrc(const char* base, uint32_t records) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, (int)records, 0x00020000);
}

// Loads of an operand whose rows run along the contraction.
template <class T>
struct GmmLoadAlong {
  static constexpr bool kAllPieces = false;
  const char* base;    // uniform
  uint32_t records;
  uint32_t off[kGmmLoads];  // lane's row and chunk of pieces w, w + 8, ...
  uint32_t chunk;      // the lane's chunk, in bytes (the same in each of the wave's pieces)
  uint32_t row_bytes;
  int step0 = 0;       // first step of this item's range

  // rows: tile row rl is matrix row row_of(rl), relative to base
  template <class RowOf>
  __device__ __forceinline__ void init(const char* b, uint32_t rec, int64_t ld, int wave, RowOf row_of) {
    using L = GmmAlong<T, kGmmTile>;
    const int lane = threadIdx.x & 63;
    base = gmm_uniform(b);
    records = (uint32_t)gmm_uniform((int)rec);
    row_bytes = (uint32_t)ld;
    chunk = (uint32_t)(((lane & 7) ^ L::swz(wave * 8 + (lane >> 3))) << 4);
#pragma unroll
    for (int j = 0; j < kGmmLoads; ++j) {
      const int rl = (wave + kGmmWaves * j) * 8 + (lane >> 3);
      off[j] = (uint32_t)(row_of(rl) * ld) + chunk;
    }
  }
  __device__ __forceinline__ void prefetch(int) {}
  template <int NL>
  __device__ __forceinline__ void issue(int step, char* stage, int wave) const {
    const uint32_t kb = (uint32_t)(step0 + step) * kGmmStepBytes;
    const bool in = kb + chunk < row_bytes;
    const GmmRsrc rs = gmm_rsrc(base, records);
#pragma unroll
    for (int j = 0; j < NL; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + kGmmWaves * j) * 1024), 16,
                                               in ? off[j] + kb : kGmmOutside, 0, 0, 0);
  }
};

// Loads of an operand whose rows run across the contraction, optionally gathered.
template <class T, bool kGather>
struct GmmLoadAcross {
  static constexpr bool kAllPieces = true;  // every piece holds columns of all blocks
  static constexpr int kRows = GmmAcross<T, kGmmTile>::kRows;
  const char* base;    // first contraction row (gathered: the matrix), uniform
  int64_t ld;          // bytes between rows
  int depth;           // contraction rows
  int step0 = 0;       // first step of this item's range
  uint32_t off[kGmmLoads];  // lane's row of the stage and column (gathered: column only)
  const int32_t* index;
  int32_t index_last;
  int32_t rows, next;  // gathered: lane l's row number of the step issued next, and of the one after

  __device__ static __forceinline__ int stage_row(int wave, int j) {
    constexpr int kRowsPer = 1024 / (kGmmTile * T::kBytes);
    return (wave + kGmmWaves * j) * kRowsPer + (threadIdx.x & 63) / (64 / kRowsPer);
  }
  __device__ __forceinline__ void init(const char* b, int64_t ld_, int depth_, int64_t col0, int wave,
                                       const int32_t* index_, int64_t index_rows) {
    using L = GmmAcross<T, kGmmTile>;
    base = gmm_uniform(b);
    ld = ld_;
    depth = gmm_uniform(depth_);
    index = index_;
    index_last = (int32_t)index_rows - 1;
#pragma unroll
    for (int j = 0; j < kGmmLoads; ++j) {
      const int r = stage_row(wave, j);
      const int c = L::chunk_at(r, (threadIdx.x & 63) % L::kChunks);
      off[j] = (uint32_t)(col0 * T::kBytes + c * 16) + (kGather ? 0u : (uint32_t)(r * ld));
    }
    rows = next = 0;
  }
  // gathered: the 64 row numbers of a step, a lane each, read one step before its loads (issue(step - 1)
  // follows)
  __device__ __forceinline__ void prefetch(int step) {
    if constexpr (kGather) {
      static_assert(kRows == 64, "a lane per row");
      rows = next < 0 ? 0 : next > index_last ? index_last : next;
      const uint32_t r = (uint32_t)((step0 + step) * kRows) + (threadIdx.x & 63);
      next = (int)r < depth ? index[r] : 0;
    }
  }
  template <int NL>
  __device__ __forceinline__ void issue(int step, char* stage, int wave) const {
    step += step0;
    int left = depth - step * kRows;
    left = left < 0 ? 0 : left > kRows ? kRows : left;
    if constexpr (kGather) {
      const GmmRsrc rs = gmm_rsrc(base, (uint32_t)gmm_uniform((int)((index_last + 1) * ld)));
#pragma unroll
      for (int j = 0; j < NL; ++j) {  // two rows a piece, one for each half of the wave
        const int r = (wave + kGmmWaves * j) * 2;
        const uint32_t r0 = r < left ? (uint32_t)__builtin_amdgcn_readlane(rows, r) * (uint32_t)ld : kGmmOutside;
        const uint32_t r1 = r + 1 < left ? (uint32_t)__builtin_amdgcn_readlane(rows, r + 1) * (uint32_t)ld : kGmmOutside;
        const uint32_t o = threadIdx.x & 32 ? r1 : r0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + kGmmWaves * j) * 1024), 16,
                                                 o == kGmmOutside ? kGmmOutside : o + off[j], 0, 0, 0);
      }
    } else {
      const GmmRsrc rs = gmm_rsrc(gmm_uniform(base + (int64_t)step * kRows * ld),
                                  (uint32_t)gmm_uniform((int)(left * ld)));
#pragma unroll
      for (int j = 0; j < NL; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + kGmmWaves * j) * 1024), 16, off[j], 0, 0,
                                                 0);
    }
  }
};

struct GmmRings {
  char* p[2];
  char* q[3];
};

// What a step hands to the next: the fragments it has already read from the next step's stages.
struct GmmCarry {
  gmm_u32x4 q[4], p[2];
};

template <int NB, class FP, class FQ>
__device__ __forceinline__ void gmm_read_first(const char* ps, const char* qs, const FP& fp, const FQ& fq, GmmCarry& c) {
#pragma unroll
  for (int s = 0; s < 4; ++s) c.q[s] = fq.read(qs, s, 0);
  c.p[0] = fp.read(ps, 0, 0);
  c.p[1] = fp.read(ps, 1 % NB, 1 / NB);
}

// One step kt (kt % 6 == D): NB P blocks x 4 Q blocks x 2 contraction halves of MFMAs, as 2 NB P fragments of 4
// products, each P fragment read two fragments ahead, the second half's Q fragments two before that half
// (a scheduling barrier after each fragment's products fixes the order).  Before the last two
// fragments every read of the step's stages has been issued; there the work-group meets (its reads
// done, the loads of step kt + 1 landed), P(kt + 2) and Q(kt + 3) are loaded into the stages that step kt
// leaves, and the first fragments of step kt + 1 are read, behind the products that remain.
// Per wave the vector-memory operations run Q0 P0 Q1 P1 Q2 | P2 Q3 | P3 Q4 | ... (a gathered Q reads its next
// row numbers before the P loads): when the work-group meets in step kt, only Q(kt + 2) may be in
// flight, kGmmLoads operations.  An operation more in between makes the wait stricter, never laxer.
// Steps past the last are loaded too: they lie past the ends, read nothing and put zeros into stages that
// nobody multiplies, so that every step is the same code with the same wait.
template <class T, int NB, int D, class LoadP, class LoadQ, class FP, class FQ>
__device__ __forceinline__ void gmm_step(LoadP& lp, LoadQ& lq, int kt, const GmmRings& r, const FP& fp, const FQ& fq,
                                         int wave, GmmCarry& c, typename T::Acc (&acc)[NB][4]) {
  constexpr int NF = 2 * NB;
  constexpr int kSecond = NB >= 2 ? NB - 2 : 0;
  constexpr int kPLoads = LoadP::kAllPieces ? kGmmLoads : (NB + 1) / 2;  // 4 NB pieces over 8 waves
  const char *ps = r.p[D % 2], *qs = r.q[D % 3];
  gmm_u32x4 q[2][4], p[NF];
#pragma unroll
  for (int s = 0; s < 4; ++s) q[0][s] = c.q[s];
  p[0] = c.p[0];
  p[1] = c.p[1];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    if (f + 2 < NF) p[f + 2] = fp.read(ps, (f + 2) % NB, (f + 2) / NB);
    if (f == kSecond) {
#pragma unroll
      for (int s = 0; s < 4; ++s) q[1][s] = fq.read(qs, s, 1);
    }
    if (f == NF - 2) {
      wait_vmcnt<kGmmLoads>();
      block_sync_lds();
      lq.prefetch(kt + 4);
      lp.template issue<kPLoads>(kt + 2, r.p[D % 2], wave);
      lq.template issue<kGmmLoads>(kt + 3, r.q[D % 3], wave);
      __builtin_amdgcn_sched_barrier(0);
      gmm_read_first<NB>(r.p[(D + 1) % 2], r.q[(D + 1) % 3], fp, fq, c);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[f % NB][s] = T::mfma(q[f / NB][s], p[f], acc[f % NB][s]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The nk steps of the contraction.  Every load has landed when it returns.
template <class T, int NB, class LoadP, class LoadQ, class FP, class FQ>
__device__ __forceinline__ void gmm_loop(LoadP& lp, LoadQ& lq, int nk, const GmmRings& r, const FP& fp, const FQ& fq,
                                         int wave, typename T::Acc (&acc)[NB][4]) {
  constexpr int kPLoads = LoadP::kAllPieces ? kGmmLoads : (NB + 1) / 2;
  if (nk <= 0) return;
  lq.prefetch(0);
  static_for<3>([&](auto ic) {  // Q0 P0 Q1 P1 Q2
    constexpr int j = decltype(ic)::value;
    lq.prefetch(j + 1);
    lq.template issue<kGmmLoads>(j, r.q[j], wave);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (j < 2) lp.template issue<kPLoads>(j, r.p[j], wave);
    __builtin_amdgcn_sched_barrier(0);
  });
  wait_vmcnt<2 * kGmmLoads + kPLoads>();
  block_sync_lds();
  GmmCarry c;
  gmm_read_first<NB>(r.p[0], r.q[0], fp, fq, c);
  // step 0 by itself: with the loop's head at a step that the prologue does not lead into, the compiler's
  // own wait before the head's first read does not drain every load in flight
  gmm_step<T, NB, 0>(lp, lq, 0, r, fp, fq, wave, c, acc);
  int kt = 1;
  for (; kt + 6 <= nk; kt += 6) {
    static_for<6>([&](auto ic) {
      constexpr int j = decltype(ic)::value;
      gmm_step<T, NB, (j + 1) % 6>(lp, lq, kt + j, r, fp, fq, wave, c, acc);
    });
  }
  static_for<5>([&](auto ic) {  // the last 0 .. 5 steps
    constexpr int j = decltype(ic)::value;
    if (kt + j < nk) gmm_step<T, NB, (j + 1) % 6>(lp, lq, kt + j, r, fp, fq, wave, c, acc);
  });
  wait_vmcnt<0>();
}

// Where an output tile goes: rows [0, rows) x columns [0, cols) of out (leading dimension ld, in
// elements); pieces: whole 16-byte pieces of rows may be stored (ld and the start are multiples of 16
// bytes).
struct GmmOut {
  char* out;
  int64_t ld;
  int rows, cols;
  bool bf16, pieces;
};

// value(row block i, Q block s, element e, row, col) -> fp32
template <int NB, class Value>
__device__ __forceinline__ void gmm_store(const GmmOut& o, const GmmRings& r, int wr, int wc, const Value& value) {
  const int lane = threadIdx.x & 63;
  if (o.bf16 && o.pieces) {
    // staged as rows of 512 bytes, 64 rows to a stage; 16-byte piece c of row x at c ^ (x & 15)
    const auto stage = [&](int b) { return b == 0 ? r.p[0] : b == 1 ? r.p[1] : b == 2 ? r.q[0] : r.q[1]; };
    block_sync_lds();  // every wave is done reading the stages
    static_for<NB>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const int row = 16 * (wr + 2 * i) + (lane & 15);
      char* st = stage(i / 2) + (row & 63) * 512;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const int col = 64 * wc + 16 * s + 4 * (lane >> 4);
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = f32_to_bf16(value(i, s, e, row, col + e));
        *reinterpret_cast<u32x2*>(st + (((col >> 3) ^ (row & 15)) << 4) + (col & 7) * 2) =
            u32x2{(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
      }
    });
    block_sync_lds();
    const int n = o.rows * 32;
    for (int ch = threadIdx.x; ch < n; ch += kGmmThreads) {
      const int row = ch >> 5, c = ch & 31;
      if (8 * c >= o.cols) continue;
      const gmm_u32x4 v = *reinterpret_cast<const gmm_u32x4*>(stage(row >> 6) + (row & 63) * 512 + ((c ^ (row & 15)) << 4));
      *reinterpret_cast<gmm_u32x4*>(o.out + (row * o.ld + 8 * c) * 2) = v;
    }
    return;
  }
  static_for<NB>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    const int row = 16 * (wr + 2 * i) + (lane & 15);
    if (row < o.rows) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int col = 64 * wc + 16 * s + 4 * (lane >> 4);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = value(i, s, e, row, col + e);
        if (!o.bf16 && o.pieces) {  // rows of whole 16-byte pieces: four columns exist or none
          if (col < o.cols)
            *reinterpret_cast<f32x4*>(o.out + (row * o.ld + col) * 4) = f32x4{v[0], v[1], v[2], v[3]};
          continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (col + e >= o.cols) continue;
          if (o.bf16)
            *reinterpret_cast<uint16_t*>(o.out + (row * o.ld + col + e) * 2) = f32_to_bf16(v[e]);
          else
            *reinterpret_cast<float*>(o.out + (row * o.ld + col + e) * 4) = v[e];
        }
      }
    }
  });
}

// Work items are tiles x slabs, numbered so that kGmmSuper tiles run slab by slab, side by side: 32
// work-groups of an XCD then share kGmmSuper tiles' rows and 8 slabs in its L2.
__device__ __forceinline__ void gmm_unnumber(int64_t item, int64_t tiles, int slabs, int64_t& tile, int& slab) {
  const int64_t sup = item / ((int64_t)kGmmSuper * slabs), first = sup * kGmmSuper;
  const int rem = (int)(item - first * slabs);
  const int n = tiles - first < kGmmSuper ? (int)(tiles - first) : kGmmSuper;
  tile = first + rem % n;
  slab = rem / n;
}

// The hardware deals work-group b to XCD b % 8.  The items of the full tiles are cut into one contiguous range per
// XCD, and after them those of the partial tiles: every XCD gets the same share of both (to within one
// item), and the short items come last, where they fill the chip's last round.  False for padding.
__device__ __forceinline__ bool gmm_row_item(int64_t b, const GmmTiles& t, int slabs, int& tile, int& slab) {
  const int64_t xcd = b % kXcds;
  int64_t local = b / kXcds, nf = (int64_t)t.full * slabs, np = (int64_t)t.partial * slabs, tt;
  const int64_t per_f = (nf + kXcds - 1) / kXcds, per_p = (np + kXcds - 1) / kXcds;
  if (local < per_f) {
    const int64_t item = xcd * per_f + local;
    if (item >= nf) return false;
    gmm_unnumber(item, t.full, slabs, tt, slab);
    tile = (int)tt;
    return true;
  }
  local -= per_f;
  const int64_t item = xcd * per_p + local;
  if (local >= per_p || item >= np) return false;
  gmm_unnumber(item, t.partial, slabs, tt, slab);
  tile = t.full + (int)tt;
  return true;
}

// Work-groups that cover the items of any grouping of max_rows rows.
inline int64_t gmm_row_grid(const GmmArgs& a, int slabs) {
  const int64_t full = a.max_rows / kGmmTile, partial = a.max_rows < a.G ? a.max_rows : a.G;
  const auto per = [&](int64_t tiles) { return (tiles * slabs + kXcds - 1) / kXcds; };
  return (per(full) + per(partial)) * kXcds;
}

// TN: groups x n tiles x slabs, dealt to the XCDs in chunks of consecutive items (groups differ in length, so
// that long contiguous ranges could leave XCDs idle): 32 of them, what an XCD runs at once, when every
// XCD gets 4 chunks or more, else 8.
__device__ __forceinline__ bool gmm_weight_item(int64_t b, int64_t tiles, int slabs, int chunk, int64_t& tile, int& slab) {
  const int64_t local = b / kXcds, item = (local / chunk * kXcds + b % kXcds) * chunk + local % chunk;
  if (item >= tiles * slabs) return false;
  gmm_unnumber(item, tiles, slabs, tile, slab);
  return true;
}
inline int gmm_weight_chunk(int64_t items) { return items >= 8 * 32 * 4 ? 32 : 8; }
inline int64_t gmm_weight_grid(int64_t items) {
  const int64_t turn = (int64_t)kXcds * gmm_weight_chunk(items);
  return (items + turn - 1) / turn * turn;
}

#define MOE_GMM_SMEM                                                                                       \
  __shared__ __align__(16) char p0_[kGmmStage], p1_[kGmmStage], q0_[kGmmStage], q1_[kGmmStage], q2_[kGmmStage]; \
  const GmmRings rings{{p0_, p1_}, {q0_, q1_, q2_}};

// NT and NN: output rows are rows of a group.
template <GmmForm F, class T, int NB>
__device__ __forceinline__ void gmm_rows_body(const GmmArgs& a, const GmmRings& rings, int g, int64_t beg, int64_t end,
                                              int64_t q0, int sp) {
  using LP = GmmAlong<T, kGmmTile>;
  using LQ = GmmQ<F, T, kGmmTile>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave >> 2, wc = wave & 3;
  const int64_t depth = F == GmmForm::kNT ? a.K : a.N, q_len = F == GmmForm::kNT ? a.N : a.K;
  const int64_t ldp = depth * T::kBytes;
  const int rows = (int)(end - beg);
  const int32_t* index = F == GmmForm::kNT ? a.row_index : nullptr;
  GmmLoadAlong<T> lp;
  {
    const char* p = static_cast<const char*>(F == GmmForm::kNT ? a.x : a.dy) + (index ? 0 : beg * ldp);
    // rows past the end re-read the last one
    const uint32_t records = (uint32_t)((index ? a.x_rows : (int64_t)rows) * ldp);
    lp.init(p, records, ldp, wave, [&](int rl) -> int64_t {
      const int64_t rr = rl < rows ? rl : rows - 1;
      if (!index) return rr;
      const int64_t i = index[beg + rr];
      return i < 0 ? 0 : i >= a.x_rows ? a.x_rows - 1 : i;
    });
  }
  const char* w = static_cast<const char*>(a.w) + (int64_t)g * a.N * a.K * T::kBytes;
  std::conditional_t<F == GmmForm::kNT, GmmLoadAlong<T>, GmmLoadAcross<T, false>> lq;
  if constexpr (F == GmmForm::kNT) {
    const int cols = (int)(q_len - q0 < kGmmTile ? q_len - q0 : kGmmTile);
    lq.init(w + q0 * ldp, (uint32_t)(cols * ldp), ldp, wave, [&](int rl) -> int64_t { return rl < cols ? rl : cols - 1; });
  } else {
    lq.init(w, (int64_t)a.K * T::kBytes, (int)depth, q0, wave, nullptr, 0);
  }
  GmmFrags<LP, 2> fp;
  fp.init(wr);
  GmmFrags<LQ, 1> fq;
  fq.init(4 * wc);
  typename T::Acc acc[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[i][s] = typename T::Acc{0, 0, 0, 0};
  constexpr int kStep = kGmmStepBytes / T::kBytes;
  int nk;
  gmm_range((int)((depth + kStep - 1) / kStep), a.split, sp, lp.step0, nk);
  lq.step0 = lp.step0;
  gmm_loop<T, NB>(lp, lq, nk, rings, fp, fq, wave, acc);

  GmmOut o;
  const int e = a.split == 1 && a.out_bf16 ? 2 : 4;
  char* const out = a.split == 1 ? static_cast<char*>(a.out)
                                 : reinterpret_cast<char*>(a.part + sp * a.max_rows * q_len);
  o.out = out + (beg * q_len + q0) * e;
  o.ld = q_len;
  o.rows = rows;
  o.cols = (int)(q_len - q0 < kGmmTile ? q_len - q0 : kGmmTile);
  o.bf16 = e == 2;
  o.pieces = (q_len * e) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  if constexpr (std::is_same_v<T, GmmI8>) {
    if (a.split > 1) {  // int32 partial sums, as they are
      gmm_store<NB>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return __int_as_float(acc[i][s][j]); });
      return;
    }
    float sx[NB], sw[4][4];
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int row = 16 * (wr + 2 * i) + (lane & 15);
      int64_t rr = beg + (row < rows ? row : rows - 1);
      if (index) {
        rr = index[rr];
        rr = rr < 0 ? 0 : rr >= a.x_rows ? a.x_rows - 1 : rr;
      }
      sx[i] = a.x_scales[rr];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 64 * wc + 16 * s + 4 * (lane >> 4) + j;
        sw[s][j] = a.w_scales[(int64_t)g * a.N + q0 + (col < o.cols ? col : 0)];
      }
    gmm_store<NB>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return (float)acc[i][s][j] * sx[i] * sw[s][j]; });
  } else {
    gmm_store<NB>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return acc[i][s][j]; });
  }
}

template <GmmForm F, class T>
__global__ __launch_bounds__(kGmmThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void gmm_rows_kernel(GmmArgs a,
                                                                                                     int slabs) {
  MOE_GMM_SMEM
  int64_t beg, end;
  int t, slab, g;
  [[maybe_unused]] const int sp = (int)(blockIdx.x % (unsigned)a.split);
  GmmTiles tiles;
  tiles.count(a.group_offsets, a.G, a.max_rows, kGmmTile);
  if (!gmm_row_item(blockIdx.x / (unsigned)a.split, tiles, slabs, t, slab)) return;
  tiles.find(a.group_offsets, a.G, a.max_rows, kGmmTile, t, g, beg, end);
#if defined(__HIP_DEVICE_COMPILE__)
  const int64_t q0 = (int64_t)slab * kGmmTile;
  switch ((int)(end - beg + 31) / 32) {  // P blocks per wave
    case 8: gmm_rows_body<F, T, 8>(a, rings, g, beg, end, q0, sp); break;
    case 7: gmm_rows_body<F, T, 7>(a, rings, g, beg, end, q0, sp); break;
    case 6: gmm_rows_body<F, T, 6>(a, rings, g, beg, end, q0, sp); break;
    case 5: gmm_rows_body<F, T, 5>(a, rings, g, beg, end, q0, sp); break;
    case 4: gmm_rows_body<F, T, 4>(a, rings, g, beg, end, q0, sp); break;
    case 3: gmm_rows_body<F, T, 3>(a, rings, g, beg, end, q0, sp); break;
    case 2: gmm_rows_body<F, T, 2>(a, rings, g, beg, end, q0, sp); break;
    default: gmm_rows_body<F, T, 1>(a, rings, g, beg, end, q0, sp); break;
  }
#else
  (void)rings;
#endif
}

// TN: output rows are columns of dy.
template <class T, bool kGather>
__global__ __launch_bounds__(kGmmThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void gmm_weights_kernel(
    GmmArgs a, int64_t tiles, int slabs, int p_tiles, int chunk) {
  MOE_GMM_SMEM
  int64_t t;
  int slab;
  [[maybe_unused]] const int sp = (int)(blockIdx.x % (unsigned)a.split);
  if (!gmm_weight_item(blockIdx.x / (unsigned)a.split, tiles, slabs, chunk, t, slab)) return;
#if defined(__HIP_DEVICE_COMPILE__)
  using L = GmmAcross<T, kGmmTile>;
  const int g = (int)(t / p_tiles);
  const int64_t p0 = (t % p_tiles) * kGmmTile, q0 = (int64_t)slab * kGmmTile;
  int64_t beg, end;
  gmm_group_rows(a.group_offsets, a.max_rows, g, beg, end);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave >> 2, wc = wave & 3;
  const int64_t ldn = (int64_t)a.N * T::kBytes, ldk = (int64_t)a.K * T::kBytes;
  const int depth = (int)(end - beg);
  GmmLoadAcross<T, false> lp;
  lp.init(static_cast<const char*>(a.dy) + beg * ldn, ldn, depth, p0, wave, nullptr, 0);
  GmmLoadAcross<T, kGather> lq;
  lq.init(static_cast<const char*>(a.x) + (kGather ? 0 : beg * ldk), ldk, depth, q0, wave,
          kGather ? a.row_index + beg : nullptr, a.x_rows);
  GmmFrags<L, 2> fp;
  fp.init(wr);
  GmmFrags<L, 1> fq;
  fq.init(4 * wc);
  f32x4 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[i][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  int nk;
  gmm_range(gmm_uniform((depth + L::kRows - 1) / L::kRows), a.split, sp, lp.step0, nk);
  lq.step0 = lp.step0;
  gmm_loop<T, 8>(lp, lq, nk, rings, fp, fq, wave, acc);
  GmmOut o;
  const int e = a.split == 1 && a.out_bf16 ? 2 : 4;
  char* const out = a.split == 1 ? static_cast<char*>(a.out)
                                 : reinterpret_cast<char*>(a.part + (int64_t)sp * a.G * a.N * a.K);
  o.out = out + (((int64_t)g * a.N + p0) * a.K + q0) * e;
  o.ld = a.K;
  o.rows = (int)(a.N - p0 < kGmmTile ? a.N - p0 : kGmmTile);
  o.cols = (int)(a.K - q0 < kGmmTile ? a.K - q0 : kGmmTile);
  o.bf16 = e == 2;
  o.pieces = ((int64_t)a.K * e) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  gmm_store<8>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return acc[i][s][j]; });
#else
  (void)rings;
#endif
}

template <GmmForm F, class T>
hipError_t gmm_launch_rows(const GmmArgs& a, hipStream_t s) {
  const int slabs = ((F == GmmForm::kNT ? a.N : a.K) + kGmmTile - 1) / kGmmTile;
  gmm_rows_kernel<F, T><<<dim3((unsigned)(gmm_row_grid(a, slabs) * a.split)), dim3(kGmmThreads), 0, s>>>(a, slabs);
  return hipGetLastError();
}

}  // namespace
}  // namespace moe

// Tile kernel of the grouped matrix products (bf16 and int8): rows that are multiples of 16 bytes from
// 16-byte boundaries.  Forms, types and LDS stages: gmm_core.h.
//
// Work item = 256 (P) x 256 (Q) outputs of one group, 8 waves in 2 x 4; a wave owns every other 16-row
// block of the P rows and 64 Q columns (at most 8 x 4 accumulator blocks, 128 registers).
//   * Both operands go straight from memory to LDS (buffer_load_dwordx4 ... lds), one instruction 1 KiB:
//     8 rows of 128 bytes (rows along the contraction), 2 rows of 512 bytes (Q across it) or 4 of 256 (P
//     across it).  LDS holds two steps of P, each as two halves of 128 rows, and three of Q: 160 KiB, every
//     piece its own __shared__ array and the loop unrolled by six, so that every access names its array
//     and the compiler's own waits stay exact.
//   * A step multiplies its first half of P, then its second; by then all its Q fragments are in registers.
//     So the first half and Q are reloaded in the middle of the step and the second half at its end: a P
//     load leads its use by 1.5 steps, a Q load by 2.5.
//   * Ends: a chunk past the end of a row gets an offset past the descriptor's record count, a
//     contraction row past the end lies past the count itself; both put zeros into LDS and read nothing.
//     So the sums see zeros past the end on both sides, never a neighbour's values.  P rows and Q columns
//     past the tile's end hold whatever is there and are not stored.
//   * The loop is instantiated per number of P blocks a wave multiplies, so that rows a group does not
//     have cost no products and no loads.
//   * Outputs are staged in LDS and leave as 16-byte pieces of whole rows.
// W = 4 is the same with 128 x 128 outputs and 80 KiB of LDS, two work-groups to a CU; tile_waves says when.
//
// What bounds it, measured on 16384 x 4096 x 7168 bf16 in one group (four full tiles per CU, 727 us,
// 1.32 PFLOP/s; a library product of the same sizes takes 644 us): a step of 64 KiB takes 1.62 us.  Loads
// alone (products and LDS reads taken out) take 1.33 us a step, 23 bytes a clock and CU, whatever the order,
// the row length or the lead of the loads; products alone take 1.2 us, the matrix cores then busy at the 1.7 GHz
// that the chip holds under them (zeros as inputs run 16% faster).  Reloading all of P at the end of a step, wave
// priorities around products or loads, and 2, 6 or 8 tiles side by side on an XCD all measured within 2%.
// With about 170 rows a group (384 groups, K = 7168) the weights' stream bounds it: 5.1 TB/s, the same with the
// products taken out.  A short item pays its ends: about 5 us from launch to the first product and 4 us to
// store 128 KiB (a sum of 3 steps takes 4 us in between).
// Tried and not kept for short sums: work-groups that stay and issue an item's first loads before storing the
// last one's outputs (48 groups of 170 rows, 7168 x 2048: 530 us against 543, but 4 to 16% slower at 8 and
// more steps, where it needs registers the loop does not have); stores straight from the registers (690 us).
// Non-temporal stores of outputs of 256 MB and more: within 1% over 38 sizes; not kept.
#pragma once
#include "gmm_core.h"
#include "tile_core.h"

namespace moe {
namespace {

// A work-group of W waves, 2 x W / 2 of them (W = 8 or 4), and its tile of 32 W x 32 W outputs.
template <int W>
struct GmmShape {
  static constexpr int kThreads = 64 * W, kTile = 32 * W, kHalf = kTile / 2;  // kHalf: P rows per half
  static constexpr int kPStage = kHalf * kGmmStepBytes, kQStage = kTile * kGmmStepBytes;
};
constexpr int kGmmPLoads = 2;       // 1 KiB loads per wave of a half of P
constexpr int kGmmQLoads = 4;       // ... and of a step of Q
constexpr int kGmmNonTemporal = 2;  // the loads' cache policy operand: nt
constexpr uint32_t kGmmOutside = 0xfffffff0u;  // an offset past every record count
constexpr int kGmmSuper = 4;        // row tiles that run side by side on one XCD

typedef __amdgpu_buffer_rsrc_t GmmRsrc;
typedef __attribute__((address_space(3))) void* GmmLds;

__device__ __forceinline__ GmmRsrc gmm_rsrc(const char* base, uint32_t records) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, (int)records, 0x00020000);
}

// Loads of NL KiB per wave of an operand whose rows run along the contraction.  kOnce: nothing reads these bytes
// again soon (non-temporal policy).
template <class T, int W, int NL, bool kOnce>
struct GmmLoadAlong {
  const char* base;    // uniform
  uint32_t records;
  uint32_t off[NL];    // lane's row and chunk of pieces w, w + W, ...
  uint32_t chunk;      // the lane's chunk, in bytes (the same in each of the wave's pieces)
  uint32_t end;        // bytes of a row up to the end of this item's range
  int step0 = 0;       // first step of this item's range

  // stage row rl is matrix row row_of(rl), relative to base
  template <class RowOf>
  __device__ __forceinline__ void init(const char* b, uint32_t rec, int64_t ld, int wave, RowOf row_of) {
    using L = GmmAlong<T, NL * W * 8>;
    const int lane = threadIdx.x & 63;
    base = gmm_uniform(b);
    records = (uint32_t)gmm_uniform((int)rec);
    end = (uint32_t)ld;
    chunk = (uint32_t)(((lane & 7) ^ L::swz(wave * 8 + (lane >> 3))) << 4);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int rl = (wave + W * j) * 8 + (lane >> 3);
      off[j] = (uint32_t)(row_of(rl) * ld) + chunk;
    }
  }
  // only the n steps from `first` on
  __device__ __forceinline__ void range(int first, int n) {
    step0 = first;
    const uint32_t to = (uint32_t)(first + n) * kGmmStepBytes;
    end = to < end ? to : end;
  }
  __device__ __forceinline__ void prefetch(int) {}
  // the first n of them
  template <int n>
  __device__ __forceinline__ void issue(int step, char* stage, int wave) const {
    const uint32_t kb = (uint32_t)(step0 + step) * kGmmStepBytes;
    const bool in = kb + chunk < end;
    const GmmRsrc rs = gmm_rsrc(base, records);
#pragma unroll
    for (int j = 0; j < n; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + W * j) * 1024), 16,
                                               in ? off[j] + kb : kGmmOutside, 0, 0, kOnce ? kGmmNonTemporal : 0);
  }
};

// Loads of NL KiB per wave of an operand whose rows run across the contraction (NL * 8 W columns), optionally
// gathered.
template <class T, int W, int NL, bool kGather, bool kOnce>
struct GmmLoadAcross {
  using L = GmmAcross<T, NL * W * 8>;
  static constexpr int kRows = L::kRows, kRowsPer = 1024 / L::kRowBytes;  // rows of a step, of a piece
  const char* base;    // first contraction row (gathered: the matrix), uniform
  int64_t ld;          // bytes between rows
  int depth;           // contraction rows up to the end of this item's range
  int step0 = 0;       // first step of this item's range
  uint32_t off[NL];    // lane's row of the stage and column (gathered: column only)
  const int32_t* index;
  int32_t index_last;
  int32_t rows, next;  // gathered: lane l's row number of the step issued next, and of the one after

  __device__ __forceinline__ void init(const char* b, int64_t ld_, int depth_, int64_t col0, int wave,
                                       const int32_t* index_, int64_t index_rows) {
    base = gmm_uniform(b);
    ld = ld_;
    depth = gmm_uniform(depth_);
    index = index_;
    index_last = (int32_t)index_rows - 1;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int r = (wave + W * j) * kRowsPer + (threadIdx.x & 63) / L::kChunks;
      const int c = L::chunk_at(r, (threadIdx.x & 63) % L::kChunks);
      off[j] = (uint32_t)(col0 * T::kBytes + c * 16) + (kGather ? 0u : (uint32_t)(r * ld));
    }
    rows = next = 0;
  }
  // only the n steps from `first` on
  __device__ __forceinline__ void range(int first, int n) {
    step0 = first;
    const int to = gmm_uniform((first + n) * kRows);
    depth = to < depth ? to : depth;
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
  template <int n>
  __device__ __forceinline__ void issue(int step, char* stage, int wave) const {
    step += step0;
    int left = depth - step * kRows;
    left = left < 0 ? 0 : left > kRows ? kRows : left;
    if constexpr (kGather) {
      const GmmRsrc rs = gmm_rsrc(base, (uint32_t)gmm_uniform((int)((index_last + 1) * ld)));
#pragma unroll
      for (int j = 0; j < n; ++j) {  // kRowsPer rows, one for each part of the wave
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int r = (wave + W * j) * kRowsPer + i;
          const uint32_t at = r < left ? (uint32_t)__builtin_amdgcn_readlane(rows, r) * (uint32_t)ld : kGmmOutside;
          if ((int)(threadIdx.x & 63) / L::kChunks == i) o = at;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + W * j) * 1024), 16,
                                                 o == kGmmOutside ? kGmmOutside : o + off[j], 0, 0, 0);
      }
    } else {
      const GmmRsrc rs = gmm_rsrc(gmm_uniform(base + (int64_t)step * kRows * ld),
                                  (uint32_t)gmm_uniform((int)(left * ld)));
#pragma unroll
      for (int j = 0; j < n; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + W * j) * 1024), 16, off[j], 0, 0,
                                                 kOnce ? kGmmNonTemporal : 0);
    }
  }
};

struct GmmRings {
  char* p[2][2];  // step parity, half
  char* q[3];
};

// What a step hands to the next: the fragments it has already read from the next step's arrays.
struct GmmCarry {
  gmm_u32x4 q[4], p[2];
};

// The 2 NB fragments of a step: the first half's kH0 blocks for the step's two contraction halves, then the
// second half's kH1.
template <int W, int NB>
struct GmmOrder {
  static constexpr int kH0 = (NB + 1) / 2, kH1 = NB / 2;
  static constexpr int kLoads0 = (4 * kH0 + W - 1) / W, kLoads1 = (4 * kH1 + W - 1) / W;  // 4 kH pieces of 8 rows
  static constexpr int half(int f) { return f >= 2 * kH0; }
  static constexpr int kk(int f) { return half(f) ? (f - 2 * kH0) / (kH1 > 0 ? kH1 : 1) : f / kH0; }
  static constexpr int block(int f) { return half(f) ? (f - 2 * kH0) % (kH1 > 0 ? kH1 : 1) : f % kH0; }  // of the half
  static constexpr int acc(int f) { return half(f) ? kH0 + block(f) : block(f); }
};

template <int W, int NB, class FP>
__device__ __forceinline__ gmm_u32x4 gmm_read_p(char* const (&p)[2], const FP& fp, int f) {
  using O = GmmOrder<W, NB>;
  return fp.read(p[O::half(f)], O::block(f), O::kk(f));
}

template <int W, int NB, class FP, class FQ>
__device__ __forceinline__ void gmm_read_first(char* const (&p)[2], const char* q, const FP& fp, const FQ& fq,
                                               GmmCarry& c) {
#pragma unroll
  for (int s = 0; s < 4; ++s) c.q[s] = fq.read(q, s, 0);
  c.p[0] = gmm_read_p<W, NB>(p, fp, 0);
  if (NB > 1) c.p[1] = gmm_read_p<W, NB>(p, fp, 1);
}

// One step kt (kt % 6 == D): 2 NB P fragments of 4 products (Q blocks), each P fragment read two fragments ahead,
// the second contraction half's Q fragments two before their first use (a scheduling barrier after each
// fragment's products fixes the order).  The work-group meets twice, each time two fragments before the
// end of a half, when every read of that half has been issued:
//   in the middle: the reads of P's first half and of Q are done, so P0(kt + 2) and Q(kt + 3) are loaded into
//     their arrays; the loads of P1(kt), issued two steps before, have landed and its reads begin
//   at the end: P1(kt + 2) is loaded; P0(kt + 1) and Q(kt + 1) have landed and the next step's first fragments
//     are read behind the products that remain.
// Per wave the vector-memory operations run ... P0(kt+1) Q(kt+2) | P1(kt+1) | P0(kt+2) Q(kt+3) | P1(kt+2) ... (|: a
// meeting; a gathered Q reads its next row numbers before P0).  Counting what may still be in flight: in
// the middle of step kt what follows P1(kt), at its end what follows P0(kt + 1).  Operations more in between
// make a wait stricter, never laxer.  With one block (NB = 1) there is one half and one meeting.
// Steps past an item's last are loaded too: they lie past the end of its range (range() of the loads), read nothing
// and put zeros into arrays that nobody multiplies, so that every step is the same code with the same waits.
// kMidWait, kEndWait: operations that may be in flight at the two meetings; mid(), end(): what is loaded there.
template <class T, int W, int NB, int kMidWait, int kEndWait, class FP, class FQ, class Mid, class End>
__device__ __forceinline__ void gmm_step(char* const (&ps)[2], const char* qs, char* const (&ps_next)[2],
                                         const char* qs_next, const FP& fp, const FQ& fq, GmmCarry& c,
                                         typename T::Acc (&acc)[NB][4], const Mid& mid, const End& end) {
  using O = GmmOrder<W, NB>;
  constexpr int NF = 2 * NB, kMid = 2 * O::kH0 - 2;
  constexpr int kSecond = O::kH0 >= 2 ? O::kH0 - 2 : 0;
  gmm_u32x4 q[2][4], p[NF];
#pragma unroll
  for (int s = 0; s < 4; ++s) q[0][s] = c.q[s];
  p[0] = c.p[0];
  if (NB > 1) p[1] = c.p[1];
  else p[1] = gmm_read_p<W, NB>(ps, fp, 1);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    if (f == kSecond) {
#pragma unroll
      for (int s = 0; s < 4; ++s) q[1][s] = fq.read(qs, s, 1);
    }
    if (f == kMid) {
      wait_vmcnt<kMidWait>();
      block_sync_lds();
      mid();
      __builtin_amdgcn_sched_barrier(0);
    }
    if (f == NF - 2) {
      if (NB > 1) {
        wait_vmcnt<kEndWait>();
        block_sync_lds();
        end();
        __builtin_amdgcn_sched_barrier(0);
      }
      gmm_read_first<W, NB>(ps_next, qs_next, fp, fq, c);
    }
    if (f + 2 < NF) p[f + 2] = gmm_read_p<W, NB>(ps, fp, f + 2);
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[O::acc(f)][s] = T::mfma(q[O::kk(f)][s], p[f], acc[O::acc(f)][s]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Step kt (kt % 6 == D) of an item's loop.
template <class T, int W, int NB, int D, class LoadP, class LoadQ, class FP, class FQ>
__device__ __forceinline__ void gmm_loop_step(LoadP (&lp)[2], LoadQ& lq, int kt, const GmmRings& r, const FP& fp,
                                              const FQ& fq, int wave, GmmCarry& c, typename T::Acc (&acc)[NB][4]) {
  using O = GmmOrder<W, NB>;
  constexpr int n0 = O::kLoads0, n1 = O::kLoads1;
  gmm_step<T, W, NB, NB == 1 ? kGmmQLoads : kGmmQLoads + n0 + n1, 2 * kGmmQLoads + n0 + n1>(
      r.p[D % 2], r.q[D % 3], r.p[(D + 1) % 2], r.q[(D + 1) % 3], fp, fq, c, acc,
      [&] {
        lq.prefetch(kt + 4);
        lp[0].template issue<n0>(kt + 2, r.p[D % 2][0], wave);
        lq.template issue<kGmmQLoads>(kt + 3, r.q[D % 3], wave);
      },
      [&] { lp[1].template issue<n1>(kt + 2, r.p[D % 2][1], wave); });
}

// The nk steps of the contraction.  Every load has landed when it returns.
template <class T, int W, int NB, class LoadP, class LoadQ, class FP, class FQ>
__device__ __forceinline__ void gmm_loop(LoadP (&lp)[2], LoadQ& lq, int nk, const GmmRings& r, const FP& fp,
                                         const FQ& fq, int wave, typename T::Acc (&acc)[NB][4]) {
  using O = GmmOrder<W, NB>;
  constexpr int n0 = O::kLoads0, n1 = O::kLoads1;
  if (nk <= 0) return;
  // the steady state's order: Q0 P0(0) Q1 P1(0) P0(1) Q2 | P1(1)
  lq.prefetch(0);
  lq.prefetch(1);
  lq.template issue<kGmmQLoads>(0, r.q[0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[0].template issue<n0>(0, r.p[0][0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.prefetch(2);
  lq.template issue<kGmmQLoads>(1, r.q[1], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[1].template issue<n1>(0, r.p[0][1], wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.prefetch(3);
  lp[0].template issue<n0>(1, r.p[1][0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.template issue<kGmmQLoads>(2, r.q[2], wave);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<2 * kGmmQLoads + n0 + n1>();
  block_sync_lds();
  lp[1].template issue<n1>(1, r.p[1][1], wave);
  __builtin_amdgcn_sched_barrier(0);
  GmmCarry c;
  gmm_read_first<W, NB>(r.p[0], r.q[0], fp, fq, c);
  // step 0 by itself, and no exits inside the unrolled loop: with either the compiler's own wait before the
  // loop head's first read drains every load in flight
  gmm_loop_step<T, W, NB, 0>(lp, lq, 0, r, fp, fq, wave, c, acc);
  int kt = 1;
  for (; kt + 6 <= nk; kt += 6) {
    static_for<6>([&](auto ic) {
      constexpr int j = decltype(ic)::value;
      gmm_loop_step<T, W, NB, (j + 1) % 6>(lp, lq, kt + j, r, fp, fq, wave, c, acc);
    });
  }
  static_for<5>([&](auto ic) {  // the last 0 .. 5 steps
    constexpr int j = decltype(ic)::value;
    if (kt + j < nk) gmm_loop_step<T, W, NB, (j + 1) % 6>(lp, lq, kt + j, r, fp, fq, wave, c, acc);
  });
  wait_vmcnt<0>();
}

// Where an output tile goes: rows [0, rows) x columns [0, cols) of out (leading dimension ld, in elements).  Rows
// leave as 16-byte pieces at whatever alignment they have, the last one of a row element by element.
struct GmmOut {
  char* out;
  int64_t ld;
  int rows, cols;
  bool bf16;
};

// value(row block i, Q block s, element e, row, col) -> fp32
template <int W, int NB, class Value>
__device__ __forceinline__ void gmm_store(const GmmOut& o, const GmmRings& r, int wr, int wc, const Value& value) {
  const int lane = threadIdx.x & 63;
  if (o.bf16) {
    // staged as rows of 64 W bytes, 32 rows to each array or half of one; 16-byte piece c of row x at c ^ (x & 15)
    using S = GmmShape<W>;
    constexpr int kRowB = S::kTile * 2, kPieces = kRowB / 16;
    static_assert(32 * kRowB <= S::kPStage && 2 * S::kPStage <= S::kQStage, "staging");
    char* const stage[8] = {r.p[0][0], r.p[0][1], r.p[1][0], r.p[1][1],
                            r.q[0], r.q[0] + S::kPStage, r.q[1], r.q[1] + S::kPStage};
    block_sync_lds();  // every wave is done reading the arrays
    static_for<NB>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const int row = 16 * (wr + 2 * i) + (lane & 15);
      char* st = stage[i] + (row & 31) * kRowB;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const int col = 64 * wc + 16 * s + 4 * (lane >> 4);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = value(i, s, e, row, col + e);
        *reinterpret_cast<u32x2*>(st + (((col >> 3) ^ (row & 15)) << 4) + (col & 7) * 2) =
            u32x2{gmm_bf16x2(v[0], v[1]), gmm_bf16x2(v[2], v[3])};
      }
    });
    block_sync_lds();
    static_for<NB>([&](auto ic) {
      constexpr int b = decltype(ic)::value;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 32 rows over the work-group, two pieces a thread
        const int x = threadIdx.x / kPieces + 16 * h, c = threadIdx.x % kPieces, row = 32 * b + x;
        if (row >= o.rows || 8 * c >= o.cols) continue;
        const gmm_u32x4 v = *reinterpret_cast<const gmm_u32x4*>(stage[b] + x * kRowB + ((c ^ (row & 15)) << 4));
        typedef gmm_u32x4 Unaligned __attribute__((aligned(2)));
        char* const to = o.out + (row * o.ld + 8 * c) * 2;
        if (8 * c + 8 <= o.cols) {
          *reinterpret_cast<Unaligned*>(to) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * c + e < o.cols) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    });
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
        char* const to = o.out + (row * o.ld + col) * 4;
        if (col + 4 <= o.cols) {
          __builtin_memcpy(to, v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < o.cols) reinterpret_cast<float*>(to)[e] = v[e];
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
inline int64_t gmm_row_grid(const GmmArgs& a, int slabs, int tile) {
  const int64_t full = a.max_rows / tile, partial = a.max_rows < a.G ? a.max_rows : a.G;
  const auto per = [&](int64_t tiles) { return (tiles * slabs + kXcds - 1) / kXcds; };
  return (per(full) + per(partial)) * kXcds;
}

// TN: sums x n tiles x slabs, dealt to the XCDs in chunks of consecutive items (groups differ in length, so
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

#define MOE_GMM_SMEM(W)                                                                                              \
  __shared__ __align__(16) char p00_[GmmShape<W>::kPStage], p01_[GmmShape<W>::kPStage], p10_[GmmShape<W>::kPStage], \
      p11_[GmmShape<W>::kPStage], q0_[GmmShape<W>::kQStage], q1_[GmmShape<W>::kQStage], q2_[GmmShape<W>::kQStage];  \
  const GmmRings rings{{{p00_, p01_}, {p10_, p11_}}, {q0_, q1_, q2_}};

// NT and NN: output rows are rows of a group.  kOnce: weights that one row tile reads come with the non-temporal
// policy.
template <GmmForm F, class T, int W, bool kOnce, int NB>
__device__ __forceinline__ void gmm_rows_body(const GmmArgs& a, const GmmRings& rings, int g, int64_t beg, int64_t end,
                                              int64_t q0, int sp) {
  using S = GmmShape<W>;
  using LP = GmmAlong<T, S::kHalf>;
  using LQ = GmmQ<F, T, S::kTile>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave / (W / 2), wc = wave % (W / 2);
  const int64_t depth = F == GmmForm::kNT ? a.K : a.N, q_len = F == GmmForm::kNT ? a.N : a.K;
  const int64_t ldp = depth * T::kBytes;
  const int rows = (int)(end - beg);
  const int32_t* index = F == GmmForm::kNT ? a.row_index : nullptr;
  GmmLoadAlong<T, W, kGmmPLoads, false> lp[2];
  {
    const char* p = static_cast<const char*>(F == GmmForm::kNT ? a.x : a.dy) + (index ? 0 : beg * ldp);
    // rows past the end re-read the last one
    const uint32_t records = (uint32_t)((index ? a.x_rows : (int64_t)rows) * ldp);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      lp[h].init(p, records, ldp, wave, [&](int rl) -> int64_t {
        rl += h * 32 * GmmOrder<W, NB>::kH0;
        const int64_t rr = rl < rows ? rl : rows - 1;
        if (!index) return rr;
        const int64_t i = index[beg + rr];
        return i < 0 ? 0 : i >= a.x_rows ? a.x_rows - 1 : i;
      });
  }
  const char* w = static_cast<const char*>(a.w) + (int64_t)g * a.N * a.K * T::kBytes;
  std::conditional_t<F == GmmForm::kNT, GmmLoadAlong<T, W, kGmmQLoads, kOnce>,
                     GmmLoadAcross<T, W, kGmmQLoads, false, kOnce>>
      lq;
  if constexpr (F == GmmForm::kNT) {
    const int cols = (int)(q_len - q0 < S::kTile ? q_len - q0 : S::kTile);
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
  int first, nk;
  gmm_range((int)((depth + kStep - 1) / kStep), a.split, sp, first, nk);
  lp[0].range(first, nk);
  lp[1].range(first, nk);
  lq.range(first, nk);
  gmm_loop<T, W, NB>(lp, lq, nk, rings, fp, fq, wave, acc);

  GmmOut o;
  const int e = a.split == 1 && a.out_bf16 ? 2 : 4;
  char* const out = a.split == 1 ? static_cast<char*>(a.out)
                                 : reinterpret_cast<char*>(a.part + sp * a.max_rows * q_len);
  o.out = out + (beg * q_len + q0) * e;
  o.ld = q_len;
  o.rows = rows;
  o.cols = (int)(q_len - q0 < S::kTile ? q_len - q0 : S::kTile);
  o.bf16 = e == 2;
  if constexpr (std::is_same_v<T, GmmI8>) {
    if (a.split > 1) {  // int32 partial sums, as they are
      gmm_store<W, NB>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return __int_as_float(acc[i][s][j]); });
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
    gmm_store<W, NB>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return (float)acc[i][s][j] * sx[i] * sw[s][j]; });
  } else {
    gmm_store<W, NB>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return acc[i][s][j]; });
  }
}

template <GmmForm F, class T, int W, bool kOnce>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2))) void gmm_rows_kernel(GmmArgs a,
                                                                                                    int slabs) {
  MOE_GMM_SMEM(W)
  using S = GmmShape<W>;
  int64_t beg, end;
  int t, slab, g;
  [[maybe_unused]] const int sp = (int)(gmm_block() % (unsigned)a.split);
  GmmTiles tiles;
  tiles.count(a.group_offsets, a.G, a.max_rows, S::kTile);
  if (!gmm_row_item(gmm_block() / (unsigned)a.split, tiles, slabs, t, slab)) return;
  // the only row tile of its group: nothing else reads the group's weights
  [[maybe_unused]] const bool alone = tiles.find(a.group_offsets, a.G, a.max_rows, S::kTile, t, g, beg, end) <= S::kTile;
#if defined(__HIP_DEVICE_COMPILE__)
  const int64_t q0 = (int64_t)slab * S::kTile;
  const int nb = (int)(end - beg + 31) / 32;  // P blocks per wave
#define MOE_GMM_CASE(N)                                                                                      \
  if constexpr (N <= W)                                                                                      \
    if (nb == N) {                                                                                           \
      if constexpr (kOnce)                                                                                   \
        if (alone) return gmm_rows_body<F, T, W, true, N>(a, rings, g, beg, end, q0, sp);                    \
      return gmm_rows_body<F, T, W, false, N>(a, rings, g, beg, end, q0, sp);                                \
    }
  MOE_GMM_CASE(8)
  MOE_GMM_CASE(7)
  MOE_GMM_CASE(6)
  MOE_GMM_CASE(5)
  MOE_GMM_CASE(4)
  MOE_GMM_CASE(3)
  MOE_GMM_CASE(2)
  MOE_GMM_CASE(1)
#undef MOE_GMM_CASE
#else
  (void)rings;
#endif
}

// TN: output rows are columns of dy.
template <class T, int W, bool kGather>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2))) void gmm_weights_kernel(
    GmmArgs a, int64_t tiles, int slabs, int p_tiles, int chunk) {
  MOE_GMM_SMEM(W)
  int64_t t;
  int slab;
  if (!gmm_weight_item(gmm_block(), tiles, slabs, chunk, t, slab)) return;
#if defined(__HIP_DEVICE_COMPILE__)
  using S = GmmShape<W>;
  using LP = GmmAcross<T, S::kHalf>;
  using LQ = GmmAcross<T, S::kTile>;
  GmmSum sum;
  if (!sum.find(a, t / p_tiles)) return;
  const int64_t p0 = (t % p_tiles) * S::kTile, q0 = (int64_t)slab * S::kTile, beg = sum.beg, end = sum.end;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave / (W / 2), wc = wave % (W / 2);
  const int64_t ldn = (int64_t)a.N * T::kBytes, ldk = (int64_t)a.K * T::kBytes;
  const int depth = gmm_uniform((int)(end - beg));
  GmmLoadAcross<T, W, kGmmPLoads, false, false> lp[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    lp[h].init(static_cast<const char*>(a.dy) + beg * ldn, ldn, depth, p0 + h * S::kHalf, wave, nullptr, 0);
  GmmLoadAcross<T, W, kGmmQLoads, kGather, false> lq;
  lq.init(static_cast<const char*>(a.x) + (kGather ? 0 : beg * ldk), ldk, depth, q0, wave,
          kGather ? a.row_index + beg : nullptr, a.x_rows);
  GmmFrags<LP, 2> fp;
  fp.init(wr);
  GmmFrags<LQ, 1> fq;
  fq.init(4 * wc);
  f32x4 acc[W][4];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[i][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  gmm_loop<T, W, W>(lp, lq, (depth + LQ::kRows - 1) / LQ::kRows, rings, fp, fq, wave, acc);
  GmmOut o;
  const int e = sum.whole && a.out_bf16 ? 2 : 4;
  o.out = sum.matrix(a) + (p0 * a.K + q0) * e;
  o.ld = a.K;
  o.rows = (int)(a.N - p0 < S::kTile ? a.N - p0 : S::kTile);
  o.cols = (int)(a.K - q0 < S::kTile ? a.K - q0 : S::kTile);
  o.bf16 = e == 2;
  gmm_store<W, W>(o, rings, wr, wc, [&](int i, int s, int j, int, int) { return acc[i][s][j]; });
#else
  (void)rings;
#endif
}

template <GmmForm F, class T, int W, bool kOnce>
hipError_t gmm_launch_rows(const GmmArgs& a, hipStream_t s) {
  using S = GmmShape<W>;
  const int slabs = ((F == GmmForm::kNT ? a.N : a.K) + S::kTile - 1) / S::kTile;
  gmm_rows_kernel<F, T, W, kOnce>
      <<<gmm_grid(gmm_row_grid(a, slabs, S::kTile) * a.split), dim3(S::kThreads), 0, s>>>(a, slabs);
  return hipGetLastError();
}

template <GmmForm F, class T>
hipError_t gmm_launch_rows(const GmmArgs& a, int waves, bool once, hipStream_t s) {
  if (waves == 8) return once ? gmm_launch_rows<F, T, 8, true>(a, s) : gmm_launch_rows<F, T, 8, false>(a, s);
  return once ? gmm_launch_rows<F, T, 4, true>(a, s) : gmm_launch_rows<F, T, 4, false>(a, s);
}

}  // namespace
}  // namespace moe

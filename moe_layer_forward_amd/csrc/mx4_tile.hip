// Tile kernel of the microscaled 4-bit products, for groups of many rows: 256 x 256 outputs of one group and 8 waves,
// or 128 x 128 and 4.  Operands, stages and stores as in gmm_tile.h; what differs:
//   * A step is 128 bytes of a row, 256 values, 8 blocks; one 16-byte fragment of a lane is one block, and its scale
//     goes to the matrix instruction (v_mfma_scale_f32_16x16x128) as a byte of a register.  Lane l multiplies blocks
//     2 (l / 16) and 2 (l / 16) + 1 of a step, so that one 2-byte read brings both scales; in LDS they sit where the
//     fragment reads of gmm_core.h expect the step's chunks l / 16 and 4 + l / 16.
//   * Scales go to LDS too, a window of four steps (32 bytes of every row) at a time, two load instructions per wave,
//     and every lane's 2-byte reads pick its blocks.  Those bytes cost the memory path whole lines, a quarter of what
//     the codes cost (a half with windows of two steps: 64 groups of 256 rows, 2048 x 7168: 161 -> 157 us; 48 of 21
//     to 2118: 133 -> 128).  Large products therefore have their scales packed first (mx4_pack_kernel): for every
//     tile and pair of steps in the order of the reads, so that a load is 1 KiB of consecutive bytes and one 16-byte
//     and one 8-byte read bring a lane all scales of a step.
//   * LDS holds two steps of both operands and two windows of scales: 160 KiB (80 KiB, two work-groups to a CU).
// What bounds it: 8192 x 18432 x 7168 takes 470 to 490 us, 1.6 a step of a work-group: the matrix instructions 1.3
// (6.4 POP/s, what they reach from registers on random data, by power; 0.85 by their clocks), LDS about 1.4 (64 KiB
// written at 64 bytes a clock, 192 read at 128), the loads alone 0.7.  The same step with weights of its own for
// every work-group, 64 groups of 256 rows: 2.6.
#include "gmm_tile.h"
#include "mx4_core.h"

namespace moe {
namespace {

struct Mx4Type {};  // for the stages of gmm_core.h, whose rows are bytes

// Loads of NL KiB per wave of an operand: 8 rows of 128 bytes an instruction.  kNt: bytes that no cache is to keep.
template <int W, int NL, bool kNt = false>
struct Mx4Load {
  const char* base;  // uniform
  uint32_t records;
  uint32_t off[NL];  // lane's row and chunk of pieces w, w + W, ...
  uint32_t chunk;    // the lane's chunk of a step, in bytes
  uint32_t end;      // bytes of a row

  template <class RowOf>
  __device__ __forceinline__ void init(const uint8_t* b, uint32_t rec, uint32_t ld, int wave, RowOf row_of) {
    using L = GmmAlong<Mx4Type, NL * W * 8>;
    const int lane = threadIdx.x & 63;
    base = gmm_uniform(reinterpret_cast<const char*>(b));
    records = (uint32_t)gmm_uniform((int)rec);
    const int at = (lane & 7) ^ L::swz(wave * 8 + (lane >> 3));  // the fragment read's chunk: block 2 (at % 4) + at / 4
    chunk = (uint32_t)(2 * (at & 3) + (at >> 2)) << 4;
    end = ld;
#pragma unroll
    for (int j = 0; j < NL; ++j) off[j] = (uint32_t)row_of((wave + W * j) * 8 + (lane >> 3)) * ld + chunk;
  }
  // the first n of them
  template <int n>
  __device__ __forceinline__ void issue(int step, char* stage, int wave) const {
    const uint32_t kb = (uint32_t)step * kGmmStepBytes;
    const bool in = kb + chunk < end;
    const GmmRsrc rs = gmm_rsrc(base, records);
#pragma unroll
    for (int j = 0; j < n; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GmmLds)(stage + (wave + W * j) * 1024), 16,
                                               in ? off[j] + kb : kGmmOutside, 0, 0, kNt ? 2 : 0);
  }
};

// Bytes of two steps' scales, packed or not, for the 32 W rows of one operand of a tile.
template <int W>
constexpr int kMx4PairScales = 32 * W * 16;
// Of a window's, four steps of both operands.
template <int W>
constexpr int kMx4WindowScales = 4 * kMx4PairScales<W>;
constexpr int kMx4ScaleLoads = 2;  // instructions of a window

// The scales of a window, P's rows and then Q's, 64 rows a wave.  Not packed: 32 rows an instruction, the two chunks
// of a row in lanes side by side (in the other order in every second 8 rows, for the banks of the reads).  Packed:
// one pair of steps an instruction.
template <int W, bool kPacked>
struct Mx4LoadScales {
  const char* base;  // of the wave's operand, uniform
  uint32_t records, end;         // bytes of a row, or of the operand's packed scales
  uint32_t off[kMx4ScaleLoads];  // of window 0
  uint32_t chunk;                // the lane's 16 bytes of a window's 32 of a row, in bytes

  // row_of: the row that holds row rl of the operand's
  template <class RowOf>
  __device__ __forceinline__ void init(const uint8_t* b, uint32_t rec, uint32_t end_, int part, RowOf row_of) {
    base = gmm_uniform(reinterpret_cast<const char*>(b));
    records = (uint32_t)gmm_uniform((int)rec);
    end = end_;
    const int lane = threadIdx.x & 63;
    chunk = kPacked ? 0 : (uint32_t)((lane ^ lane >> 4) & 1) << 4;
#pragma unroll
    for (int j = 0; j < kMx4ScaleLoads; ++j)
      off[j] = kPacked ? (uint32_t)(j * kMx4PairScales<W> + part * 1024 + lane * 16)
                       : (uint32_t)row_of(64 * part + 32 * j + (lane >> 1)) * end + chunk;
  }
  __device__ __forceinline__ void issue(int win, char* stage, int wave) const {
    constexpr int kTo = kPacked ? 2 * kMx4PairScales<W> : 1024, kWave = kPacked ? 1024 : kMx4ScaleLoads * 1024;
    const uint32_t at = (uint32_t)win * (kPacked ? 2 * kMx4PairScales<W> : 32);
#pragma unroll
    for (int j = 0; j < kMx4ScaleLoads; ++j) {
      const bool in = at + (kPacked ? (uint32_t)(j * kMx4PairScales<W>) : chunk) < end;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(gmm_rsrc(base, records), (GmmLds)(stage + wave * kWave + j * kTo), 16,
                                               in ? off[j] + at : kGmmOutside, 0, 0, 0);
    }
  }
};

struct Mx4Rings {
  char* p[2][2];  // step parity, half
  char* q[2];
  char* s;        // two windows
};

typedef uint16_t mx4_u16x2 __attribute__((ext_vector_type(2)));

// What a step hands to the next: the fragments it has already read from the next step's arrays, and that step's scales:
// the 2 bytes of row blocks 2 i and 2 i + 1 in the halves of one register.
template <int NB>
struct Mx4Carry {
  gmm_u32x4 q[4], p[2];
  uint32_t sq[2], sp[(NB + 1) / 2];
};

// Where a lane's scales lie in a window's stage, and which of a step's two blocks the row has.
template <int W, bool kPacked>
struct Mx4Scales {
  uint32_t p, q;  // byte offsets of the lane's scales of a window's first step
  int left;       // not packed: blocks from this lane's first one of step 0 to the end of the row

  __device__ __forceinline__ void init(int wr, int wc, int blocks) {
    const int lane = threadIdx.x & 63, r = lane & 15, part = lane >> 4;
    if constexpr (kPacked) {  // [pair][operand][step][wave row][lane][block][2]
      p = (uint32_t)((wr * 64 + lane) * W * 2);
      q = (uint32_t)(kMx4PairScales<W> + (wc * 64 + lane) * 8);
    } else {  // [operand][row][pair, in the loads' order][step][block]
      p = (uint32_t)((16 * wr + r) * 32 + 2 * part + (r >> 3) * 16);
      q = p + (uint32_t)(2 * kMx4PairScales<W> + (64 * wc - 16 * wr) * 32);
    }
    left = blocks - 2 * part;
  }
  template <int kRows>  // rows between the two
  __device__ __forceinline__ static uint32_t pair(const char* at, bool both) {
    mx4_u16x2 v = {*reinterpret_cast<const uint16_t*>(at), 0};
    if (both) v[1] = *reinterpret_cast<const uint16_t*>(at + kRows * 32);
    return __builtin_bit_cast(uint32_t, v);
  }
  // Step kt, kt % 4 == D, of the window at st.
  template <int D, int NB>
  __device__ __forceinline__ void read(const char* st, int kt, Mx4Carry<NB>& c) const {
    if constexpr (kPacked) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const char* at = st + D / 2 * 2 * kMx4PairScales<W> + D % 2 * (kMx4PairScales<W> / 2);
      const u32x2 qs = *reinterpret_cast<const u32x2*>(at + q);
      c.sq[0] = qs[0];
      c.sq[1] = qs[1];
      static_assert(W == 8, "a lane's 16 bytes");
      const gmm_u32x4 ps = *reinterpret_cast<const gmm_u32x4*>(at + p);
#pragma unroll
      for (int i = 0; i < (NB + 1) / 2; ++i) c.sp[i] = ps[i];
    } else {
      const uint32_t pp = p ^ (D / 2 * 16), qq = q ^ (D / 2 * 16);
      const char* at = st + 8 * (D % 2);
      uint32_t mask = mx4_scale_mask(left - 8 * kt) & 0xffffu;  // no scales from the padding
      mask |= mask << 16;
#pragma unroll
      for (int s = 0; s < 2; ++s) c.sq[s] = pair<16>(at + qq + s * 2 * 16 * 32, true) & mask;
#pragma unroll
      for (int i = 0; i < (NB + 1) / 2; ++i) c.sp[i] = pair<32>(at + pp + i * 2 * 32 * 32, 2 * i + 1 < NB) & mask;
    }
  }
};

template <int W, int NB, int D, class FP, class FQ, class Scales>
__device__ __forceinline__ void mx4_read_first(char* const (&p)[2], const char* q, const char* s, int kt, const FP& fp,
                                               const FQ& fq, const Scales& sc, Mx4Carry<NB>& c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c.q[j] = fq.read(q, j, 0);
  c.p[0] = gmm_read_p<W, NB>(p, fp, 0);
  c.p[1] = gmm_read_p<W, NB>(p, fp, 1);
  sc.template read<D>(s, kt, c);
}

// Step kt (kt % 4 == D), as gmm_step with these loads:
//   in the middle: P0(kt + 2) and Q(kt + 2)
//   at its end: P1(kt + 2), and in a window's last step, when the next one's first scales have been read (the compiler
//     lets no read of the scales' array pass while a load into it is in flight), the scales of window (kt + 5) / 4,
//     whose slot the step's own scales have left
// The middle waits for P1(kt), behind which P0(kt + 1), Q(kt + 1) and P1(kt + 1) may be in flight; the end for P0(kt
// + 1) and Q(kt + 1), behind which P1(kt + 1), P0(kt + 2) and Q(kt + 2) may be; in a window's first step the scales,
// too. `next`: the window of step kt + 1.
template <int W, int NB, int D, class LoadP, class LoadQ, class LoadS, class FP, class FQ, class Scales>
__device__ __forceinline__ void mx4_step(const LoadP (&lp)[2], const LoadQ& lq, const LoadS& ls, int kt,
                                         const Mx4Rings& r, char* next, const FP& fp, const FQ& fq, const Scales& sc,
                                         int wave, Mx4Carry<NB>& c, f32x4 (&acc)[NB][4]) {
  using O = GmmOrder<W, NB>;
  constexpr int n0 = O::kLoads0, n1 = O::kLoads1;
  constexpr int NF = 2 * NB, kMid = 2 * O::kH0 - 2;
  constexpr int kSecond = O::kH0 >= 2 ? O::kH0 - 2 : 0;
  char* const(&ps)[2] = r.p[D % 2];
  gmm_u32x4 q[2][4], p[NF];
  const Mx4Carry<NB> now = c;
#pragma unroll
  for (int s = 0; s < 4; ++s) q[0][s] = c.q[s];
  p[0] = c.p[0];
  p[1] = c.p[1];
  static_for<NF>([&](auto fc) {
    constexpr int f = decltype(fc)::value;
    if (f == kSecond) {
#pragma unroll
      for (int s = 0; s < 4; ++s) q[1][s] = fq.read(r.q[D % 2], s, 1);
    }
    if (f == kMid) {
      wait_vmcnt<kGmmQLoads + n0 + n1 + (D == 0 ? kMx4ScaleLoads : 0)>();
      block_sync_lds();
      lp[0].template issue<n0>(kt + 2, r.p[D % 2][0], wave);
      lq.template issue<kGmmQLoads>(kt + 2, r.q[D % 2], wave);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (f == NF - 2) {
      wait_vmcnt<kGmmQLoads + n0 + n1 + (D == 0 ? kMx4ScaleLoads : 0)>();
      block_sync_lds();
      lp[1].template issue<n1>(kt + 2, r.p[D % 2][1], wave);
      __builtin_amdgcn_sched_barrier(0);
      mx4_read_first<W, NB, (D + 1) % 4>(r.p[(D + 1) % 2], r.q[(D + 1) % 2], next, kt + 1, fp, fq, sc, c);
      if (D == 3) ls.issue((kt + 5) / 4, r.s + (kt / 4 & 1) * kMx4WindowScales<W>, wave);
    }
    if constexpr (f + 2 < NF) p[f + 2] = gmm_read_p<W, NB>(ps, fp, f + 2);
    constexpr int kk = O::kk(f), i = O::acc(f);
    static_for<4>([&](auto scol) {
      constexpr int s = decltype(scol)::value;
      acc[i][s] = mx4_mfma<2 * (s % 2) + kk, 2 * (i % 2) + kk>(q[kk][s], now.sq[s / 2], p[f], now.sp[i / 2], acc[i][s]);
    });
    __builtin_amdgcn_sched_barrier(0);
  });
}

// The nk steps of the contraction.  Every load has landed when it returns.
template <int W, int NB, class LoadP, class LoadQ, class LoadS, class FP, class FQ, class Scales>
__device__ __forceinline__ void mx4_loop(const LoadP (&lp)[2], const LoadQ& lq, const LoadS& ls, int nk,
                                         const Mx4Rings& r, const FP& fp, const FQ& fq, const Scales& sc, int wave,
                                         f32x4 (&acc)[NB][4]) {
  using O = GmmOrder<W, NB>;
  constexpr int n0 = O::kLoads0, n1 = O::kLoads1;
  ls.issue(0, r.s, wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.template issue<kGmmQLoads>(0, r.q[0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[0].template issue<n0>(0, r.p[0][0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[1].template issue<n1>(0, r.p[0][1], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[0].template issue<n0>(1, r.p[1][0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.template issue<kGmmQLoads>(1, r.q[1], wave);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<kGmmQLoads + n0 + n1>();
  block_sync_lds();
  lp[1].template issue<n1>(1, r.p[1][1], wave);
  __builtin_amdgcn_sched_barrier(0);
  Mx4Carry<NB> c;
  mx4_read_first<W, NB, 0>(r.p[0], r.q[0], r.s, 0, fp, fq, sc, c);
  ls.issue(1, r.s + kMx4WindowScales<W>, wave);
  __builtin_amdgcn_sched_barrier(0);
  mx4_step<W, NB, 0>(lp, lq, ls, 0, r, r.s, fp, fq, sc, wave, c, acc);
  const auto window = [&](int step) { return r.s + (step / 4 & 1) * kMx4WindowScales<W>; };
  int kt = 1;
  for (; kt + 4 <= nk; kt += 4) {
    static_for<4>([&](auto ic) {
      constexpr int j = decltype(ic)::value;
      mx4_step<W, NB, (j + 1) % 4>(lp, lq, ls, kt + j, r, window(kt + j + 1), fp, fq, sc, wave, c, acc);
    });
  }
  static_for<3>([&](auto ic) {  // the last 0 .. 3 steps
    constexpr int j = decltype(ic)::value;
    if (kt + j < nk) mx4_step<W, NB, (j + 1) % 4>(lp, lq, ls, kt + j, r, window(kt + j + 1), fp, fq, sc, wave, c, acc);
  });
  wait_vmcnt<0>();
}

// Where the packed scales of the row tiles lie, and those of the slabs after them: `pairs` of steps to each.
template <int W>
struct Mx4Packed {
  const uint8_t *p, *q;
  __device__ __forceinline__ Mx4Packed(const Mx4Args& a, int tile, int g, int slabs, int slab, int pairs) {
    const int64_t each = (int64_t)pairs * kMx4PairScales<W>;
    p = a.packed + tile * each;
    q = a.packed + (gmm_max_tiles(a.max_rows, a.G, 32 * W) + (int64_t)g * slabs + slab) * each;
  }
};

template <int W, bool kPacked, bool kNt, int NB>
__device__ __forceinline__ void mx4_tile_body(const Mx4Args& a, const Mx4Rings& rings, int tile, int g, int64_t beg,
                                              int64_t end, int slabs, int slab) {
  using S = GmmShape<W>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave / (W / 2), wc = wave % (W / 2);
  const int q0 = slab * S::kTile;
  const int rows = (int)(end - beg), cols = a.N - q0 < S::kTile ? a.N - q0 : S::kTile;
  const uint32_t ld = (uint32_t)(a.K / 2), lds = (uint32_t)mx4_scale_cols(a.K);
  const int steps = (int)((ld + kGmmStepBytes - 1) / kGmmStepBytes);
  const int64_t w0 = (int64_t)g * a.N + q0, x0 = a.row_index ? 0 : beg, xn = a.row_index ? a.x_rows : rows;
  // rows past the end re-read the last one
  const auto x_row = [&](int rl) -> int64_t {
    rl = rl < rows ? rl : rows - 1;
    return a.row_index ? mx4_gathered(a, beg + rl) : rl;
  };
  const auto w_row = [&](int rl) -> int64_t { return rl < cols ? rl : cols - 1; };
  Mx4Load<W, kGmmPLoads> lp[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    lp[h].init(a.x + x0 * ld, (uint32_t)(xn * ld), ld, wave,
               [&](int rl) { return x_row(rl + h * 32 * GmmOrder<W, NB>::kH0); });
  Mx4Load<W, kGmmQLoads, kNt> lq;
  lq.init(a.w + w0 * ld, (uint32_t)cols * ld, ld, wave, w_row);
  Mx4LoadScales<W, kPacked> ls;
  const bool of_x = wave < W / 2;
  const int part = of_x ? wave : wave - W / 2;
  const auto scale_row = [&](int rl) -> int64_t { return of_x ? x_row(rl) : w_row(rl); };
  if constexpr (kPacked) {
    const Mx4Packed<W> packed(a, tile, g, slabs, slab, (int)lds / 16);
    const uint32_t bytes = lds / 16 * kMx4PairScales<W>;
    ls.init(of_x ? packed.p : packed.q, bytes, bytes, part, scale_row);
  } else {
    ls.init(of_x ? a.xs + x0 * lds : a.ws + w0 * lds, of_x ? (uint32_t)(xn * lds) : (uint32_t)cols * lds, lds, part,
            scale_row);
  }
  GmmFrags<GmmAlong<Mx4Type, S::kHalf>, 2> fp;
  fp.init(wr);
  GmmFrags<GmmAlong<Mx4Type, S::kTile>, 1> fq;
  fq.init(4 * wc);
  Mx4Scales<W, kPacked> sc;
  sc.init(wr, wc, a.K / 32);
  f32x4 acc[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[i][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  mx4_loop<W, NB>(lp, lq, ls, steps, rings, fp, fq, sc, wave, acc);

  GmmOut o;
  o.bf16 = a.out_bf16;
  o.out = static_cast<char*>(a.out) + (beg * a.N + q0) * (o.bf16 ? 2 : 4);
  o.ld = a.N;
  o.rows = rows;
  o.cols = cols;
  const GmmRings stage{{{rings.p[0][0], rings.p[0][1]}, {rings.p[1][0], rings.p[1][1]}},
                       {rings.q[0], rings.q[1], nullptr}};
  gmm_store<W, NB>(o, stage, wr, wc, [&](int i, int s, int j, int, int) { return acc[i][s][j]; });
}

// gmm_row_item for tiles whose partial ones are sorted: eight of those at a time, a tile to an XCD, so that its slabs
// share the rows of x, in turns of changing direction; the slabs of the last ones, fewer than eight, are dealt out.
__device__ __forceinline__ bool mx4_row_item(int64_t b, const GmmTiles& t, int slabs, int& tile, int& slab) {
  const int64_t nf = (int64_t)t.full * slabs, per_f = (nf + kXcds - 1) / kXcds, local = b / kXcds - per_f;
  if (local < 0) return gmm_row_item(b, t, slabs, tile, slab);
  const int xcd = (int)(b % kXcds), whole = t.partial / kXcds;
  if (local < (int64_t)whole * slabs) {
    const int turn = (int)(local / slabs);
    slab = (int)(local - (int64_t)turn * slabs);
    tile = t.full + turn * kXcds + (turn & 1 ? kXcds - 1 - xcd : xcd);
    return true;
  }
  const int64_t item = (local - (int64_t)whole * slabs) * kXcds + xcd;
  const int rest = (int)(item / slabs);
  slab = (int)(item - (int64_t)rest * slabs);
  tile = t.full + whole * kXcds + rest;
  return rest < t.partial - whole * kXcds;
}

template <int W, bool kPacked, bool kNt>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx4_tile_kernel(Mx4Args a, int slabs) {
  using S = GmmShape<W>;
  __shared__ __align__(16) char p00_[S::kPStage], p01_[S::kPStage], p10_[S::kPStage], p11_[S::kPStage], q0_[S::kQStage],
      q1_[S::kQStage], s_[2 * kMx4WindowScales<W>];
  const Mx4Rings rings{{{p00_, p01_}, {p10_, p11_}}, {q0_, q1_}, s_};
#if defined(__HIP_DEVICE_COMPILE__)
  int64_t beg, end;
  int t, slab, g;
  Mx4Tiles tiles;
  tiles.count(a, S::kTile);
  if (!mx4_row_item(gmm_block(), tiles.t, slabs, t, slab)) return;
  // offsets that overlap: no place among the packed
  if (kPacked && t >= gmm_max_tiles(a.max_rows, a.G, S::kTile)) return;
  tiles.find(a, S::kTile, t, g, beg, end);
  if (beg >= end) return;  // the same: more tiles than were counted
  // P blocks per wave.  Two at least: with one the loop has one meeting a step, which waits for all that is in flight
  // (32 rows, 18432 x 7168: 17.9 us, with two 15.3).
  const int nb = end - beg > 32 ? (int)(end - beg + 31) / 32 : 2;
#define MOE_MX4_CASE(N) \
  if constexpr (N <= W) \
    if (nb == N) return mx4_tile_body<W, kPacked, kNt, N>(a, rings, t, g, beg, end, slabs, slab);
  MOE_MX4_CASE(8)
  MOE_MX4_CASE(7)
  MOE_MX4_CASE(6)
  MOE_MX4_CASE(5)
  MOE_MX4_CASE(4)
  MOE_MX4_CASE(3)
  MOE_MX4_CASE(2)
#undef MOE_MX4_CASE
#else
  (void)rings;
#endif
}

// The scales of tile or slab gmm_block() (the row tiles' places first, then the slabs of every group), pairs
// blockIdx.z * kPackPairs on, into the order of the tile kernel's reads.  A work-group of 32 W threads, a row each.
constexpr int kPackPairs = 4;
template <int W>
__global__ __launch_bounds__(32 * W) void mx4_pack_kernel(Mx4Args a, int slabs, uint8_t* packed) {
  constexpr int kTile = 32 * W, kBytes = kMx4PairScales<W>;
  __shared__ __align__(16) uint16_t order[kPackPairs][kBytes / 2];
  const int64_t places = gmm_max_tiles(a.max_rows, a.G, kTile), at = gmm_block();
  const int lds = mx4_scale_cols(a.K), pairs = lds / 16, rl = threadIdx.x, r = rl & 15;
  const uint8_t* row;
  int place;                 // of the lane that reads this row's first block (l / 16 = 0), in units of 2 bytes,
  constexpr int kPart = 16;  // and from block to block
  int per;    // 2-byte scales of a lane
  if (at < places) {
    Mx4Tiles tiles;
    tiles.count(a, kTile);
    if (at >= tiles.t.full + tiles.t.partial) return;  // the whole work-group
    int g;
    int64_t beg, end;
    tiles.find(a, kTile, (int)at, g, beg, end);
    if (beg >= end) return;
    const int64_t i = beg + (beg + rl < end ? rl : end - beg - 1);
    row = a.xs + (a.row_index ? mx4_gathered(a, i) : i) * lds;
    per = W;  // row 16 (wr + 2 i) + r: scale i of lane r of wave row wr
    place = ((rl >> 4 & 1) * 64 + r) * per + (rl >> 5);
  } else {
    const int64_t s = at - places, q0 = s % slabs * kTile;
    if (s >= (int64_t)a.G * slabs) return;  // past the grid's last place
    const int64_t n = s / slabs * a.N + (q0 + rl < a.N ? q0 + rl : a.N - 1);
    row = a.ws + n * lds;
    per = 4;  // row 64 wc + 16 s + r: scale s of lane r of wave column wc
    place = ((rl >> 6) * 64 + r) * per + (rl >> 4 & 3);
  }
  const int first = blockIdx.z * kPackPairs;
#pragma unroll
  for (int j = 0; j < kPackPairs; ++j)
    if (first + j < pairs) {
      const gmm_u32x4 v = *reinterpret_cast<const gmm_u32x4*>(row + (first + j) * 16);
#pragma unroll
      for (int d = 0; d < 4; ++d) {  // dword d: step d / 2, lanes part 2 (d % 2) and the next
        const uint32_t m = v[d] & mx4_scale_mask(a.K / 32 - 16 * (first + j) - 4 * d);  // nothing from the padding
        uint16_t* to = order[j] + d / 2 * (kBytes / 4) + place + 2 * (d % 2) * kPart * per;
        to[0] = (uint16_t)m;
        to[kPart * per] = (uint16_t)(m >> 16);
      }
    }
  __syncthreads();
  uint8_t* out = packed + (at * pairs + first) * kBytes + threadIdx.x * 16;
#pragma unroll
  for (int j = 0; j < kPackPairs; ++j)
    if (first + j < pairs)
      *reinterpret_cast<gmm_u32x4*>(out + j * kBytes) = *reinterpret_cast<const gmm_u32x4*>(order[j] + threadIdx.x * 8);
}

int tile_slabs(const Mx4Args& a, int waves) { return (a.N + 32 * waves - 1) / (32 * waves); }

int64_t pack_places(const Mx4Args& a) { return gmm_max_tiles(a.max_rows, a.G, 256) + (int64_t)a.G * tile_slabs(a, 8); }

}  // namespace

int64_t mx4_tile_grid(const Mx4Args& a, int waves) {
  return gmm_row_grid(a.max_rows, a.G, tile_slabs(a, waves), 32 * waves);
}

size_t mx4_packed_bytes(const Mx4Args& a) {
  return (size_t)pack_places(a) * (mx4_scale_cols(a.K) / 16) * kMx4PairScales<8>;
}

hipError_t launch_mx4_pack(const Mx4Args& a, hipStream_t s) {
  const int pairs = mx4_scale_cols(a.K) / 16;
  dim3 grid = gmm_grid(pack_places(a));
  grid.z = (unsigned)((pairs + kPackPairs - 1) / kPackPairs);
  mx4_pack_kernel<8><<<grid, 256, 0, s>>>(a, tile_slabs(a, 8), a.packed);
  return hipGetLastError();
}

hipError_t launch_mx4_tile(const Mx4Args& a, int waves, bool stream, hipStream_t s) {
  const dim3 grid = gmm_grid(mx4_tile_grid(a, waves)), block(64 * waves);
  const int slabs = tile_slabs(a, waves);
  if (a.packed) mx4_tile_kernel<8, true, false><<<grid, block, 0, s>>>(a, slabs);
  else if (waves == 8 && stream) mx4_tile_kernel<8, false, true><<<grid, block, 0, s>>>(a, slabs);
  else if (waves == 8) mx4_tile_kernel<8, false, false><<<grid, block, 0, s>>>(a, slabs);
  else if (stream) mx4_tile_kernel<4, false, true><<<grid, block, 0, s>>>(a, slabs);
  else mx4_tile_kernel<4, false, false><<<grid, block, 0, s>>>(a, slabs);
  return hipGetLastError();
}

}  // namespace moe

// Tile kernel of the microscaled 4-bit products, for groups of many rows: 256 x 256 outputs of one group and 8 waves, or
// 128 x 128 and 4.  Operands, stages and stores as in gmm_tile.h; what differs:
//   * A step is 128 bytes of a row, 256 values, 8 blocks; one 16-byte fragment of a lane is one block, and its scale goes
//     to the matrix instruction (v_mfma_scale_f32_16x16x128) as a byte of a register.  Lane l multiplies blocks 2 (l / 16)
//     and 2 (l / 16) + 1 of a step, so that one 2-byte read brings both scales; in LDS they sit where the
//     fragment reads of gmm_core.h expect the step's chunks l / 16 and 4 + l / 16.
//   * Scales go to LDS too, a window of two steps (16 bytes of every row) at a time, one load instruction per wave, and
//     every lane's 2-byte reads pick its blocks. Those 16 bytes cost the memory path whole lines, a third of what a
//     step's codes cost, and the reads another twelfth of the time (8192 x 18432 x 7168: 546 us, 489 without these
//     loads, 385 without any).  Large products therefore have their scales packed first (mx4_pack_kernel): for every tile
//     and window in the order of the reads, so that a load is 1 KiB of consecutive bytes and one 16-byte and one 8-byte
//     read bring a lane all scales of a step.
//   * LDS holds two steps of both operands and two windows of scales: 144 KiB (72 KiB, two work-groups to a CU).
#include "gmm_tile.h"
#include "mx4_core.h"

namespace moe {
namespace {

struct Mx4Type {};  // for the stages of gmm_core.h, whose rows are bytes

// Loads of NL KiB per wave of an operand: 8 rows of 128 bytes an instruction.
template <int W, int NL>
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
                                               in ? off[j] + kb : kGmmOutside, 0, 0, 0);
  }
};

// Bytes of a window's scales, packed or not, for the 32 W rows of one operand of a tile.
template <int W>
constexpr int kMx4WindowScales = 32 * W * 16;

// The scales of a window, P's rows and then Q's, 64 rows a wave: one instruction.
struct Mx4LoadScales {
  const char* base;  // of the wave's operand, uniform
  uint32_t records, off, stride, end;  // bytes from a window to the next, and to the end of the last

  __device__ __forceinline__ void init(const uint8_t* b, uint32_t rec, uint32_t off_, uint32_t stride_, uint32_t end_) {
    base = gmm_uniform(reinterpret_cast<const char*>(b));
    records = (uint32_t)gmm_uniform((int)rec);
    off = off_;
    stride = stride_;
    end = end_;
  }
  __device__ __forceinline__ void issue(int win, char* stage, int wave) const {
    const uint32_t at = (uint32_t)win * stride;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(gmm_rsrc(base, records), (GmmLds)(stage + wave * 1024), 16,
                                             at < end ? off + at : kGmmOutside, 0, 0, 0);
  }
};

struct Mx4Rings {
  char* p[2][2];  // step parity, half
  char* q[2];
  char* s[2];     // window parity
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
  uint32_t p, q;  // byte offsets of the lane's first scales
  int left;       // not packed: blocks from this lane's first one of step 0 to the end of the row

  __device__ __forceinline__ void init(int wr, int wc, int blocks) {
    const int lane = threadIdx.x & 63, r = lane & 15, part = lane >> 4;
    if constexpr (kPacked) {  // [step][wave row][lane][block][2]
      p = (uint32_t)((wr * 64 + lane) * W * 2);
      q = (uint32_t)(kMx4WindowScales<W> + (wc * 64 + lane) * 8);
    } else {
      p = (uint32_t)((16 * wr + r) * 16 + 2 * part);
      q = (uint32_t)(kMx4WindowScales<W> + (64 * wc + r) * 16 + 2 * part);
    }
    left = blocks - 2 * part;
  }
  template <int kRows>  // rows between the two
  __device__ __forceinline__ static uint32_t pair(const char* at, bool both) {
    mx4_u16x2 v = {*reinterpret_cast<const uint16_t*>(at), 0};
    if (both) v[1] = *reinterpret_cast<const uint16_t*>(at + kRows * 16);
    return __builtin_bit_cast(uint32_t, v);
  }
  template <int NB>
  __device__ __forceinline__ void read(const char* st, int kt, Mx4Carry<NB>& c) const {
    if constexpr (kPacked) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const char* at = st + (kt & 1) * (kMx4WindowScales<W> / 2);
      const u32x2 qs = *reinterpret_cast<const u32x2*>(at + q);
      c.sq[0] = qs[0];
      c.sq[1] = qs[1];
      static_assert(W == 8, "a lane's 16 bytes");
      const gmm_u32x4 ps = *reinterpret_cast<const gmm_u32x4*>(at + p);
#pragma unroll
      for (int i = 0; i < (NB + 1) / 2; ++i) c.sp[i] = ps[i];
    } else {
      const char* at = st + 8 * (kt & 1);
      uint32_t mask = mx4_scale_mask(left - 8 * kt) & 0xffffu;  // no scales from the padding
      mask |= mask << 16;
#pragma unroll
      for (int s = 0; s < 2; ++s) c.sq[s] = pair<16>(at + q + s * 2 * 16 * 16, true) & mask;
#pragma unroll
      for (int i = 0; i < (NB + 1) / 2; ++i) c.sp[i] = pair<32>(at + p + i * 2 * 32 * 16, 2 * i + 1 < NB) & mask;
    }
  }
};

template <int W, int NB, class FP, class FQ, class Scales>
__device__ __forceinline__ void mx4_read_first(char* const (&p)[2], const char* q, const char* s, int kt, const FP& fp,
                                               const FQ& fq, const Scales& sc, Mx4Carry<NB>& c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c.q[j] = fq.read(q, j, 0);
  c.p[0] = gmm_read_p<W, NB>(p, fp, 0);
  if (NB > 1) c.p[1] = gmm_read_p<W, NB>(p, fp, 1);
  sc.read(s, kt, c);
}

// Step kt (kt % 4 == D), as gmm_step with these loads:
//   in the middle: P0(kt + 2) and Q(kt + 2), before them, in odd steps, the scales of window (kt + 3) / 2, whose slot
//     the step's own scales have left
//   at its end: P1(kt + 2)
// The middle waits for P1(kt), behind which P0(kt + 1), Q(kt + 1) and P1(kt + 1) may be in flight; the end for
// P0(kt + 1) and Q(kt + 1), behind which P1(kt + 1), P0(kt + 2) and Q(kt + 2) may be; scales in between make a wait
// stricter, and those of step kt + 1 came before what its end waits for.  With one block the only meeting waits for
// everything.
template <int W, int NB, int D, class LoadP, class LoadQ, class FP, class FQ, class Scales>
__device__ __forceinline__ void mx4_step(const LoadP (&lp)[2], const LoadQ& lq, const Mx4LoadScales& ls, int kt,
                                         const Mx4Rings& r, const FP& fp, const FQ& fq, const Scales& sc, int wave,
                                         Mx4Carry<NB>& c, f32x4 (&acc)[NB][4]) {
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
  if (NB > 1) p[1] = c.p[1];
  else p[1] = gmm_read_p<W, NB>(ps, fp, 1);
  static_for<NF>([&](auto fc) {
    constexpr int f = decltype(fc)::value;
    if (f == kSecond) {
#pragma unroll
      for (int s = 0; s < 4; ++s) q[1][s] = fq.read(r.q[D % 2], s, 1);
    }
    if (f == kMid) {
      wait_vmcnt<NB == 1 ? 0 : kGmmQLoads + n0 + n1>();
      block_sync_lds();
      if (D % 2) ls.issue((kt + 3) / 2, r.s[D / 2], wave);
      lp[0].template issue<n0>(kt + 2, r.p[D % 2][0], wave);
      lq.template issue<kGmmQLoads>(kt + 2, r.q[D % 2], wave);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (f == NF - 2) {
      if (NB > 1) {
        wait_vmcnt<kGmmQLoads + n0 + n1>();
        block_sync_lds();
        lp[1].template issue<n1>(kt + 2, r.p[D % 2][1], wave);
        __builtin_amdgcn_sched_barrier(0);
      }
      mx4_read_first<W, NB>(r.p[(D + 1) % 2], r.q[(D + 1) % 2], r.s[(D + 1) / 2 % 2], kt + 1, fp, fq, sc, c);
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
template <int W, int NB, class LoadP, class LoadQ, class FP, class FQ, class Scales>
__device__ __forceinline__ void mx4_loop(const LoadP (&lp)[2], const LoadQ& lq, const Mx4LoadScales& ls, int nk,
                                         const Mx4Rings& r, const FP& fp, const FQ& fq, const Scales& sc, int wave,
                                         f32x4 (&acc)[NB][4]) {
  using O = GmmOrder<W, NB>;
  constexpr int n0 = O::kLoads0, n1 = O::kLoads1;
  ls.issue(0, r.s[0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.template issue<kGmmQLoads>(0, r.q[0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[0].template issue<n0>(0, r.p[0][0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[1].template issue<n1>(0, r.p[0][1], wave);
  __builtin_amdgcn_sched_barrier(0);
  ls.issue(1, r.s[1], wave);
  __builtin_amdgcn_sched_barrier(0);
  lp[0].template issue<n0>(1, r.p[1][0], wave);
  __builtin_amdgcn_sched_barrier(0);
  lq.template issue<kGmmQLoads>(1, r.q[1], wave);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<kGmmQLoads + n0 + n1 + 1>();
  block_sync_lds();
  lp[1].template issue<n1>(1, r.p[1][1], wave);
  __builtin_amdgcn_sched_barrier(0);
  Mx4Carry<NB> c;
  mx4_read_first<W, NB>(r.p[0], r.q[0], r.s[0], 0, fp, fq, sc, c);
  mx4_step<W, NB, 0>(lp, lq, ls, 0, r, fp, fq, sc, wave, c, acc);
  int kt = 1;
  for (; kt + 4 <= nk; kt += 4) {
    static_for<4>([&](auto ic) {
      constexpr int j = decltype(ic)::value;
      mx4_step<W, NB, (j + 1) % 4>(lp, lq, ls, kt + j, r, fp, fq, sc, wave, c, acc);
    });
  }
  static_for<3>([&](auto ic) {  // the last 0 .. 3 steps
    constexpr int j = decltype(ic)::value;
    if (kt + j < nk) mx4_step<W, NB, (j + 1) % 4>(lp, lq, ls, kt + j, r, fp, fq, sc, wave, c, acc);
  });
  wait_vmcnt<0>();
}

// Where the packed scales of the row tiles lie, and those of the slabs after them: `windows` to each.
template <int W>
struct Mx4Packed {
  const uint8_t *p, *q;
  __device__ __forceinline__ Mx4Packed(const Mx4Args& a, int tile, int g, int slabs, int slab, int windows) {
    const int64_t each = (int64_t)windows * kMx4WindowScales<W>;
    p = a.packed + tile * each;
    q = a.packed + (gmm_max_tiles(a.max_rows, a.G, 32 * W) + (int64_t)g * slabs + slab) * each;
  }
};

template <int W, bool kPacked, int NB>
__device__ __forceinline__ void mx4_tile_body(const Mx4Args& a, const Mx4Rings& rings, int tile, int g, int64_t beg,
                                              int64_t end, int slabs, int slab) {
  using S = GmmShape<W>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave / (W / 2), wc = wave % (W / 2);
  const int lane = threadIdx.x & 63, q0 = slab * S::kTile;
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
    lp[h].init(a.x + x0 * ld, (uint32_t)(xn * ld), ld, wave, [&](int rl) { return x_row(rl + h * 32 * GmmOrder<W, NB>::kH0); });
  Mx4Load<W, kGmmQLoads> lq;
  lq.init(a.w + w0 * ld, (uint32_t)cols * ld, ld, wave, w_row);
  Mx4LoadScales ls;
  const bool of_x = wave < W / 2;
  if constexpr (kPacked) {
    const Mx4Packed<W> packed(a, tile, g, slabs, slab, (int)lds / 16);
    const uint32_t bytes = lds / 16 * kMx4WindowScales<W>;
    ls.init(of_x ? packed.p : packed.q, bytes, (uint32_t)(wave % (W / 2) * 1024 + lane * 16), kMx4WindowScales<W>, bytes);
  } else {
    ls.init(of_x ? a.xs + x0 * lds : a.ws + w0 * lds, of_x ? (uint32_t)(xn * lds) : (uint32_t)cols * lds,
            (uint32_t)(of_x ? x_row(64 * wave + lane) : w_row(64 * (wave - W / 2) + lane)) * lds, 16, lds);
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
  const GmmRings stage{{{rings.p[0][0], rings.p[0][1]}, {rings.p[1][0], rings.p[1][1]}}, {rings.q[0], rings.q[1], nullptr}};
  gmm_store<W, NB>(o, stage, wr, wc, [&](int i, int s, int j, int, int) { return acc[i][s][j]; });
}

template <int W, bool kPacked>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2))) void mx4_tile_kernel(Mx4Args a, int slabs) {
  using S = GmmShape<W>;
  constexpr int kSStage = 2 * kMx4WindowScales<W>;
  __shared__ __align__(16) char p00_[S::kPStage], p01_[S::kPStage], p10_[S::kPStage], p11_[S::kPStage], q0_[S::kQStage],
      q1_[S::kQStage], s0_[kSStage], s1_[kSStage];
  const Mx4Rings rings{{{p00_, p01_}, {p10_, p11_}}, {q0_, q1_}, {s0_, s1_}};
#if defined(__HIP_DEVICE_COMPILE__)
  int64_t beg, end;
  int t, slab, g;
  Mx4Tiles tiles;
  tiles.count(a, S::kTile);
  if (!gmm_row_item(gmm_block(), tiles.t, slabs, t, slab)) return;
  if (kPacked && t >= gmm_max_tiles(a.max_rows, a.G, S::kTile)) return;  // offsets that overlap: no place among the packed
  tiles.find(a, S::kTile, t, g, beg, end);
  const int nb = (int)(end - beg + 31) / 32;  // P blocks per wave
#define MOE_MX4_CASE(N) \
  if constexpr (N <= W) \
    if (nb == N) return mx4_tile_body<W, kPacked, N>(a, rings, t, g, beg, end, slabs, slab);
  MOE_MX4_CASE(8)
  MOE_MX4_CASE(7)
  MOE_MX4_CASE(6)
  MOE_MX4_CASE(5)
  MOE_MX4_CASE(4)
  MOE_MX4_CASE(3)
  MOE_MX4_CASE(2)
  MOE_MX4_CASE(1)
#undef MOE_MX4_CASE
#else
  (void)rings;
#endif
}

// The scales of tile or slab blockIdx.x (the row tiles' places first, then the slabs of every group), windows
// blockIdx.y * kPackWindows on, into the order of the tile kernel's reads.  A work-group of 32 W threads, a row each.
constexpr int kPackWindows = 4;
template <int W>
__global__ __launch_bounds__(32 * W) void mx4_pack_kernel(Mx4Args a, int slabs, uint8_t* packed) {
  constexpr int kTile = 32 * W, kBytes = kMx4WindowScales<W>;
  __shared__ __align__(16) uint16_t order[kPackWindows][kBytes / 2];
  const int64_t places = gmm_max_tiles(a.max_rows, a.G, kTile), at = blockIdx.x;
  const int lds = mx4_scale_cols(a.K), windows = lds / 16, rl = threadIdx.x, r = rl & 15;
  const uint8_t* row;
  int place;  // of the lane that reads this row's first block (l / 16 = 0), in units of 2 bytes, and from block to block
  constexpr int kPart = 16;
  int per;    // 2-byte scales of a lane
  if (at < places) {
    Mx4Tiles tiles;
    tiles.count(a, kTile);
    if (at >= tiles.t.full + tiles.t.partial) return;  // the whole work-group
    int g;
    int64_t beg, end;
    tiles.find(a, kTile, (int)at, g, beg, end);
    const int64_t i = beg + (beg + rl < end ? rl : end - beg - 1);
    row = a.xs + (a.row_index ? mx4_gathered(a, i) : i) * lds;
    per = W;  // row 16 (wr + 2 i) + r: scale i of lane r of wave row wr
    place = ((rl >> 4 & 1) * 64 + r) * per + (rl >> 5);
  } else {
    const int64_t s = at - places, q0 = s % slabs * kTile;
    const int64_t n = s / slabs * a.N + (q0 + rl < a.N ? q0 + rl : a.N - 1);
    row = a.ws + n * lds;
    per = 4;  // row 64 wc + 16 s + r: scale s of lane r of wave column wc
    place = ((rl >> 6) * 64 + r) * per + (rl >> 4 & 3);
  }
  const int first = blockIdx.y * kPackWindows;
#pragma unroll
  for (int j = 0; j < kPackWindows; ++j)
    if (first + j < windows) {
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
  uint8_t* out = packed + (at * windows + first) * kBytes + threadIdx.x * 16;
#pragma unroll
  for (int j = 0; j < kPackWindows; ++j)
    if (first + j < windows)
      *reinterpret_cast<gmm_u32x4*>(out + j * kBytes) = *reinterpret_cast<const gmm_u32x4*>(order[j] + threadIdx.x * 8);
}

int tile_slabs(const Mx4Args& a, int waves) { return (a.N + 32 * waves - 1) / (32 * waves); }

int64_t pack_places(const Mx4Args& a) { return gmm_max_tiles(a.max_rows, a.G, 256) + (int64_t)a.G * tile_slabs(a, 8); }

}  // namespace

int64_t mx4_tile_grid(const Mx4Args& a, int waves) {
  return gmm_row_grid(a.max_rows, a.G, tile_slabs(a, waves), 32 * waves);
}

size_t mx4_packed_bytes(const Mx4Args& a) {
  return (size_t)pack_places(a) * (mx4_scale_cols(a.K) / 16) * kMx4WindowScales<8>;
}

hipError_t launch_mx4_pack(const Mx4Args& a, hipStream_t s) {
  const int windows = mx4_scale_cols(a.K) / 16;
  const dim3 grid((unsigned)pack_places(a), (unsigned)((windows + kPackWindows - 1) / kPackWindows));
  mx4_pack_kernel<8><<<grid, 256, 0, s>>>(a, tile_slabs(a, 8), a.packed);
  return hipGetLastError();
}

hipError_t launch_mx4_tile(const Mx4Args& a, int waves, hipStream_t s) {
  const dim3 grid = gmm_grid(mx4_tile_grid(a, waves)), block(64 * waves);
  const int slabs = tile_slabs(a, waves);
  if (waves == 4) mx4_tile_kernel<4, false><<<grid, block, 0, s>>>(a, slabs);
  else if (a.packed) mx4_tile_kernel<8, true><<<grid, block, 0, s>>>(a, slabs);
  else mx4_tile_kernel<8, false><<<grid, block, 0, s>>>(a, slabs);
  return hipGetLastError();
}

}  // namespace moe

// Microscaled 4-bit products for groups of few rows: a stream of weights.
//
// Work item = up to 16 NB rows of one group x 64 QB columns, 16 QB to each of four waves.  A step is a window of 512
// values: 256 bytes of every row, whole lines, which go straight to LDS, four rows an instruction: the wave's own
// rows of weights, its quarter of the token rows, and in one more instruction the 16 bytes of scales of its weight
// rows and of one block of token rows.  In v_mfma_scale_f32_16x16x128 number t of a step lane l multiplies block 4 (l
// / 16) + t of row l % 16, so that one dword holds its scales, byte t for number t.  Row r keeps that block's 16
// bytes at position (4 t + l / 16) ^ r: the rows of one fragment read fall in different banks.
//
// Work-groups stay, two to a CU: each takes every 64th item of its XCD's share (neighbours read neighbouring
// weights), and the loads run ahead of the products, across the ends of items, so that the stream never stops.  One
// barrier a step: a stage is loaded again when every wave has passed the barrier of the step after it.
//
// Bound: HBM.  384 groups, 512 rows, 7168 x 2048: 328 us, 6.8 TB/s of weights (16-row x 64-byte loads into registers:
// 480, stopping at every item).  Two work-groups of 64 columns, three stages: 346; one of 128, four: 382; 32 or more
// rows to an item: slower than tiles wherever there are so many.
#include "mx4_core.h"

namespace moe {
namespace {

constexpr int kRingWaves = 4;
constexpr int kRingP = 1, kRingQ = 2, kRingPer = 2;  // NB, QB, work-groups to a CU
constexpr int kRingRow = 256;  // bytes of a row and step

// QB 16-column blocks to a wave; two stages, which let `per` work-groups run on a CU.
template <int NB, int QB, int per>
struct RingShape {
  static constexpr int kX = NB * 16 * kRingRow, kW = kRingWaves * QB * 16 * kRingRow, kS = kRingWaves * (QB + 1) * 256;
  static_assert(2 * per * (kX + kW + kS) <= 160 * 1024, "LDS");
};

struct RingStage {
  char *x, *w, *s;
};

// Row rl of the item's rows in x: uniform (scalar loads of the index: a vector load's wait would drain the stream).
__device__ __forceinline__ int ring_row(const Mx4Args& a, int64_t beg, int rows, int rl) {
  rl = rl < rows ? rl : rows - 1;  // rows past the end read the last one
  if (!a.row_index) return rl;
  typedef const __attribute__((address_space(4))) int32_t* Const;
  const int64_t i = ((Const)(uintptr_t)a.row_index)[beg + rl];
  return (int)(i < 0 ? 0 : i >= a.x_rows ? a.x_rows - 1 : i);
}

// What a lane loads of an item.
template <int NB, int QB>
struct RingLoads {
  const uint8_t *w, *x;  // uniform
  const uint8_t* s;      // the lane's row of scales
  uint32_t nw, nx;
  uint32_t wo[4 * QB], xo[NB];

  // which 16 bytes of a window of row r go where the lane's go
  __device__ __forceinline__ static uint32_t chunk(int r) {
    const int c = (threadIdx.x ^ r) & 15;
    return (uint32_t)(4 * (c & 3) + (c >> 2)) * 16;
  }
  __device__ __forceinline__ void init(const Mx4Args& a, int g, int64_t beg, int64_t end, int slab, int wave) {
    const int lane = threadIdx.x & 63, quarter = lane >> 4, q0 = (slab * kRingWaves + wave) * 16 * QB;
    const int rows = (int)(end - beg), cols = a.N - q0 < 1 ? 1 : a.N - q0 < 16 * QB ? a.N - q0 : 16 * QB;
    const uint32_t ld = (uint32_t)(a.K / 2), lds = (uint32_t)mx4_scale_cols(a.K);
    const int64_t w0 = (int64_t)g * a.N + (q0 < a.N ? q0 : a.N - 1), x0 = a.row_index ? 0 : beg;
    w = a.w + w0 * ld;
    x = a.x + x0 * ld;
    nw = (uint32_t)cols * ld;
    nx = (uint32_t)((a.row_index ? a.x_rows : rows) * ld);
#pragma unroll
    for (int i = 0; i < 4 * QB; ++i) {
      const int r = 4 * i + quarter;
      wo[i] = (uint32_t)(r < cols ? r : cols - 1) * ld + chunk(r);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      int row = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = ring_row(a, beg, rows, 16 * i + 4 * wave + k);
        row = quarter == k ? at : row;
      }
      xo[i] = (uint32_t)row * ld + chunk(4 * wave + quarter);
    }
    const int r = lane & 15;
    s = a.ws + (w0 + (lane < cols ? lane : cols - 1)) * lds;
    if (wave < NB) {
      int row = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int at = ring_row(a, beg, rows, 16 * wave + k);
        row = r == k ? at : row;
      }
      if (lane >= 16 * QB) s = a.xs + (x0 + row) * lds;
    }
  }
  // window `win` of the rows, which have ld bytes
  __device__ __forceinline__ void issue(const RingStage& st, int win, uint32_t ld, int wave) const {
    typedef __attribute__((address_space(3))) void* Lds;
    const int lane = threadIdx.x & 63, quarter = lane >> 4;
    const uint32_t kb = (uint32_t)win * kRingRow, left = ld - kb;
    const Mx4Rsrc rw = mx4_rsrc(w + kb, nw > kb ? nw - kb : 0), rx = mx4_rsrc(x + kb, nx > kb ? nx - kb : 0);
    // chunks past the end of a row put zeros into LDS and read nothing
#pragma unroll
    for (int i = 0; i < 4 * QB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (Lds)(st.w + (wave * 4 * QB + i) * 1024), 16,
                                               chunk(4 * i + quarter) < left ? wo[i] : kMx4Outside, 0, 0, 2);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (Lds)(st.x + (i * 4 + wave) * 1024), 16,
                                               chunk(4 * wave + quarter) < left ? xo[i] : kMx4Outside, 0, 0, 0);
    if (lane < 16 * QB + 16)
      __builtin_amdgcn_global_load_lds(s + kb / 16, (Lds)(st.s + wave * (QB + 1) * 256), 16, 0, 0);
  }
};

// The share of a work-group: items first, first + stride, ... below end.
struct RingShare {
  int first, end, stride;
  __device__ __forceinline__ RingShare(int items) {
    const int xcd = blockIdx.x % kXcds, share = (items + kXcds - 1) / kXcds;
    stride = gridDim.x / kXcds;
    first = xcd * share + blockIdx.x / kXcds;
    end = (xcd + 1) * share < items ? (xcd + 1) * share : items;
  }
  __device__ __forceinline__ int count() const { return first < end ? (end - first + stride - 1) / stride : 0; }
};

template <int NB, int QB, int per>
__global__ __launch_bounds__(64 * kRingWaves, per) void mx4_ring_kernel(Mx4Args a, int slabs) {
  using S = RingShape<NB, QB, per>;
  __shared__ __align__(16) char x0_[S::kX], w0_[S::kW], s0_[S::kS], x1_[S::kX], w1_[S::kW], s1_[S::kS];
  [[maybe_unused]] const auto stage = [&](auto odd) -> RingStage {
    if constexpr (decltype(odd)::value) return {x1_, w1_, s1_};
    else return {x0_, w0_, s0_};
  };
#if defined(__HIP_DEVICE_COMPILE__)
  Mx4Tiles tiles;
  tiles.count(a, 16 * NB);
  constexpr int64_t kMost = (int64_t)1 << 30;  // only offsets that overlap make more
  const int64_t items = (int64_t)(tiles.t.full + tiles.t.partial) * slabs;
  const RingShare share((int)(items < kMost ? items : kMost));
  const int mine = share.count();
  if (!mine) return;
  const int wave = gmm_uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, part = lane >> 4;
  const uint32_t ld = (uint32_t)(a.K / 2);
  const int windows = (int)((ld + kRingRow - 1) / kRingRow);
  RingLoads<NB, QB> loads;
  int g, load_item = share.first, load_win = 0, item = share.first, win = 0, done = 0;
  int64_t beg, end;
  const auto next_load = [&](const RingStage& st) {
    loads.issue(st, load_win, ld, wave);
    if (++load_win == windows) {
      load_win = 0;
      load_item += share.stride;
      if (load_item < share.end) {
        tiles.find(a, 16 * NB, load_item / slabs, g, beg, end);
        loads.init(a, g, beg, end, load_item % slabs, wave);
      } else {
        loads.nw = loads.nx = 0;  // past the last item no codes are read (its scales are); the waits stay the same
      }
    }
  };
  tiles.find(a, 16 * NB, load_item / slabs, g, beg, end);
  loads.init(a, g, beg, end, load_item % slabs, wave);
  next_load(stage(std::false_type{}));
  f32x4 acc[NB][QB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < QB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t turns = ((int64_t)mine * windows + 1) / 2;
  for (int64_t turn = 0; turn < turns; ++turn)
    static_for<2>([&](auto odd) {
      wait_vmcnt<0>();
      block_sync_lds();
      next_load(stage(std::bool_constant<!decltype(odd)::value>{}));
      __builtin_amdgcn_sched_barrier(0);
      const RingStage st = stage(odd);
      const uint32_t mask = mx4_scale_mask(a.K / 32 - 16 * win - 4 * part);  // no scales from the padding
      const char* const scales = st.s + r * 16 + part * 4;
      uint32_t sw[QB], sx[NB];
#pragma unroll
      for (int j = 0; j < QB; ++j)
        sw[j] = *reinterpret_cast<const uint32_t*>(scales + (wave * (QB + 1) + j) * 256) & mask;
#pragma unroll
      for (int i = 0; i < NB; ++i)
        sx[i] = *reinterpret_cast<const uint32_t*>(scales + (i * (QB + 1) + QB) * 256) & mask;
      static_for<4>([&](auto tc) {
        constexpr int t = decltype(tc)::value;
        const int at = r * kRingRow + (((4 * t + part) ^ r) << 4);
        gmm_u32x4 w[QB], x[NB];
#pragma unroll
        for (int j = 0; j < QB; ++j) w[j] = *reinterpret_cast<const gmm_u32x4*>(st.w + (wave * QB + j) * 4096 + at);
#pragma unroll
        for (int i = 0; i < NB; ++i) x[i] = *reinterpret_cast<const gmm_u32x4*>(st.x + i * 4096 + at);
#pragma unroll
        for (int j = 0; j < QB; ++j)
#pragma unroll
          for (int i = 0; i < NB; ++i) acc[i][j] = mx4_mfma<t, t>(w[j], sw[j], x[i], sx[i], acc[i][j]);
      });
      if (++win == windows) {
        if (done < mine) {
          int gg;
          int64_t b, e;
          tiles.find(a, 16 * NB, item / slabs, gg, b, e);
          const int q0 = (item % slabs * kRingWaves + wave) * 16 * QB;
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < QB; ++j) {
              const int col = q0 + 16 * j + 4 * part;
              if (b + 16 * i + r < e && col < a.N)
                mx4_store4(a.out, a.out_bf16, (b + 16 * i + r) * a.N + col, a.N - col, acc[i][j]);
              acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
        win = 0;
        item += share.stride;
        ++done;
      }
    });
  wait_vmcnt<0>();  // no load may land in LDS that belongs to someone else
#endif
}

int ring_slabs(const Mx4Args& a) { return (a.N + 64 * kRingQ - 1) / (64 * kRingQ); }

}  // namespace

int64_t mx4_ring_items(const Mx4Args& a) { return gmm_max_tiles(a.max_rows, a.G, 16 * kRingP) * ring_slabs(a); }

hipError_t launch_mx4_ring(const Mx4Args& a, hipStream_t s) {
  const int64_t items = (mx4_ring_items(a) + kXcds - 1) / kXcds * kXcds, most = 256 * kRingPer;
  const dim3 grid((unsigned)(items < most ? items : most));
  mx4_ring_kernel<kRingP, kRingQ, kRingPer><<<grid, 64 * kRingWaves, 0, s>>>(a, ring_slabs(a));
  return hipGetLastError();
}

}  // namespace moe

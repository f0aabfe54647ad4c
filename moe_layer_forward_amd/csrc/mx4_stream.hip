// Grouped product of microscaled 4-bit rows and weights, operands straight from memory to registers:
//   y[r, n] = sum over blocks b of 32: 2^(sx[i, b] + sw[g, n, b] - 254) sum_{k in b} qx[i, k] qw[g, n, k]
// with v_mfma_scale_f32_16x16x128: lane l holds 32 values of row l % 16 of each operand, 16 bytes, which is one block
// and its scale.  A window of 512 values is four products: lane l takes block 4 t + l / 16 in the t-th, so that every
// load instruction reads 64 consecutive bytes of each of 16 rows, and its scale is byte l / 16 of the t-th dword of
// the window's 16 bytes.
//
// Work item = up to 16 PB rows of one group x 16 QB columns; the W waves of a work-group take every W-th window each
// and join their sums in LDS, in a fixed order.  (4 or 16 waves: within 2%, and up to 30% slower.)
//
// Bound: the way of weights through registers: a wave holds one window of both operands and asks for the next when it
// has multiplied this one, and many waves on a CU cover that (asking earlier takes registers from other waves: 17.3
// us against 13.7 with one row).  18432 x 7168 (70 MB with scales), one row: 13.7 us where the weights come from the
// last-level cache, 16.3 from HBM; 32 rows, 7168 x 18432: 21.4 and 23.7.
#include "mx4_core.h"

namespace moe {
namespace {

constexpr int W = 8;  // waves of a work-group

template <int PB, int QB>
__global__ __launch_bounds__(64 * W, PB * QB >= 4 ? 2 : 4) void mx4_stream_kernel(Mx4Args a, int slabs) {
  __shared__ f32x4 sums[W * PB * QB * 64];
#if defined(__HIP_DEVICE_COMPILE__)
  Mx4Tiles tiles;
  tiles.count(a, 16 * PB);
  int t0, slab, g;
  if (!gmm_row_item(gmm_block(), tiles.t, slabs, t0, slab)) return;
  int64_t beg, end;
  tiles.find(a, 16 * PB, t0, g, beg, end);
  if (beg >= end) return;  // offsets that overlap: more tiles than were counted
  const int wave = gmm_uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, part = lane >> 4;
  const int q0 = slab * 16 * QB, rows = (int)(end - beg), cols = a.N - q0 < 16 * QB ? a.N - q0 : 16 * QB;
  const uint32_t ld = (uint32_t)(a.K / 2), lds = (uint32_t)mx4_scale_cols(a.K);
  const int windows = (int)(lds / 16);
  const int64_t w0 = (int64_t)g * a.N + q0, x0 = a.row_index ? 0 : beg, xn = a.row_index ? a.x_rows : rows;
  const Mx4Rsrc rw = mx4_rsrc(a.w + w0 * ld, (uint32_t)cols * ld);
  const Mx4Rsrc rws = mx4_rsrc(a.ws + w0 * lds, (uint32_t)cols * lds);
  const Mx4Rsrc rx = mx4_rsrc(a.x + x0 * ld, (uint32_t)(xn * ld));
  const Mx4Rsrc rxs = mx4_rsrc(a.xs + x0 * lds, (uint32_t)(xn * lds));
  uint32_t wrow[QB], xrow[PB];  // rows past the end read the last one
#pragma unroll
  for (int j = 0; j < QB; ++j) wrow[j] = (uint32_t)(16 * j + r < cols ? 16 * j + r : cols - 1);
#pragma unroll
  for (int i = 0; i < PB; ++i) {
    const int rl = 16 * i + r < rows ? 16 * i + r : rows - 1;
    xrow[i] = (uint32_t)(a.row_index ? mx4_gathered(a, beg + rl) : rl);
  }
  f32x4 acc[PB][QB];
#pragma unroll
  for (int i = 0; i < PB; ++i)
#pragma unroll
    for (int j = 0; j < QB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int win = wave; win < windows; win += W) {
    const uint32_t kb = (uint32_t)win * 256 + 16 * part, ks = (uint32_t)win * 16;
    gmm_u32x4 w[QB][4], x[PB][4], sw[QB], sx[PB];
#pragma unroll
    for (int j = 0; j < QB; ++j) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        w[j][t] = mx4_load128(rw, kb + 64 * t < ld ? wrow[j] * ld + kb + 64 * t : kMx4Outside);
      sw[j] = mx4_load128(rws, wrow[j] * lds + ks);
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        x[i][t] = mx4_load128(rx, kb + 64 * t < ld ? xrow[i] * ld + kb + 64 * t : kMx4Outside);
      sx[i] = mx4_load128(rxs, xrow[i] * lds + ks);
    }
    __builtin_amdgcn_sched_barrier(0);  // every load of a window is in flight before the first product waits
    const int left = a.K / 32 - 16 * win - part;  // no scales from the padding
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t qs[QB], ps[PB];
#pragma unroll
      for (int j = 0; j < QB; ++j) qs[j] = 4 * t < left ? sw[j][t] >> (8 * part) : 0;
#pragma unroll
      for (int i = 0; i < PB; ++i) ps[i] = 4 * t < left ? sx[i][t] >> (8 * part) : 0;
#pragma unroll
      for (int j = 0; j < QB; ++j)
#pragma unroll
        for (int i = 0; i < PB; ++i) acc[i][j] = mx4_mfma<0, 0>(w[j][t], qs[j], x[i][t], ps[i], acc[i][j]);
    }
  }
  // every block's sums joined by one of the waves, in their order
#pragma unroll
  for (int b = 0; b < PB * QB; ++b) sums[(wave * PB * QB + b) * 64 + lane] = acc[b / QB][b % QB];
  __syncthreads();
  static_assert(PB * QB <= W, "a block to a wave");
  if (wave >= PB * QB) return;
  f32x4 v = sums[wave * 64 + lane];
#pragma unroll
  for (int k = 1; k < W; ++k) v += sums[(k * PB * QB + wave) * 64 + lane];
  const int row = 16 * (wave / QB) + r, col = 16 * (wave % QB) + 4 * part;
  if (row < rows && col < cols) mx4_store4(a.out, a.out_bf16, (beg + row) * a.N + q0 + col, cols - col, v);
#else
  (void)sums;
#endif
}

int stream_slabs(const Mx4Args& a, const Mx4Stream& c) { return (a.N + 16 * c.q_blocks - 1) / (16 * c.q_blocks); }

template <int PB>
void launch_stream(const Mx4Args& a, const Mx4Stream& c, hipStream_t s) {
  const int slabs = stream_slabs(a, c);
  const dim3 grid = gmm_grid(mx4_stream_grid(a, c));
  if (c.q_blocks == 1) mx4_stream_kernel<PB, 1><<<grid, 64 * W, 0, s>>>(a, slabs);
  else mx4_stream_kernel<PB, 2><<<grid, 64 * W, 0, s>>>(a, slabs);
}

}  // namespace

int64_t mx4_stream_grid(const Mx4Args& a, const Mx4Stream& c) {
  return gmm_row_grid(a.max_rows, a.G, stream_slabs(a, c), 16 * c.p_blocks);
}

hipError_t launch_mx4_stream(const Mx4Args& a, const Mx4Stream& c, hipStream_t s) {
  if (c.p_blocks == 1) launch_stream<1>(a, c, s);
  else if (c.p_blocks == 2) launch_stream<2>(a, c, s);
  else if (c.p_blocks == 3) launch_stream<3>(a, c, s);
  else launch_stream<4>(a, c, s);
  return hipGetLastError();
}

}  // namespace moe

// Grouped product of microscaled 4-bit rows and weights, operands straight from memory to registers:
//   y[r, n] = sum over blocks b of 32: 2^(sx[i, b] + sw[g, n, b] - 254) sum_{k in b} qx[i, k] qw[g, n, k]
// with v_mfma_scale_f32_16x16x128: lane l holds 32 values of row l % 16 of each operand, 16 bytes, which is one
// block and its scale.  Which of the sum's blocks the four lanes of a row hold is free as long as both operands agree, so
// in every window of 512 values lane l takes the four consecutive blocks 4 (l / 16) .. + 3: 64 bytes of codes, and one
// dword with the four scales, of which the t-th product takes byte t.
//
// Work item = up to 16 PB rows of one group x 64 columns; the four waves of a work-group take every fourth window each
// and join their sums in LDS, in a fixed order.  Every weight is read once for its 16 PB rows.
#include "gmm_core.h"
#include "mx4_core.h"

namespace moe {
namespace {

constexpr int kStreamWaves = 4, kStreamQ = 4;  // waves that share a sum; 16-column blocks of an item

template <int NB>
__device__ __forceinline__ void stream_body(const Mx4Args& a, f32x4* sums, int g, int64_t beg, int64_t end, int q0) {
  constexpr int W = kStreamWaves, QB = kStreamQ;
  const int lane = threadIdx.x & 63, wave = gmm_uniform(threadIdx.x >> 6), r = lane & 15, part = lane >> 4;
  const int rows = (int)(end - beg), cols = a.N - q0 < 16 * QB ? a.N - q0 : 16 * QB;
  const uint32_t ld = (uint32_t)(a.K / 2), lds = (uint32_t)mx4_scale_cols(a.K);
  const int windows = (int)(lds / 16);
  const int64_t first = (int64_t)g * a.N + q0;
  const Mx4Rsrc rw = mx4_rsrc(a.w + first * ld, (uint32_t)cols * ld), rws = mx4_rsrc(a.ws + first * lds, (uint32_t)cols * lds);
  const int64_t x0 = a.row_index ? 0 : beg, xn = a.row_index ? a.x_rows : rows;
  const Mx4Rsrc rx = mx4_rsrc(a.x + x0 * ld, (uint32_t)(xn * ld)), rxs = mx4_rsrc(a.xs + x0 * lds, (uint32_t)(xn * lds));
  uint32_t wrow[QB], xrow[NB];  // rows past the end read the last one
#pragma unroll
  for (int j = 0; j < QB; ++j) wrow[j] = (uint32_t)(16 * j + r < cols ? 16 * j + r : cols - 1);
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int rl = 16 * i + r < rows ? 16 * i + r : rows - 1;
    xrow[i] = (uint32_t)(a.row_index ? mx4_gathered(a, beg + rl) : rl);
  }
  f32x4 acc[NB][QB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < QB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int win = wave; win < windows; win += W) {
    const uint32_t kb = (uint32_t)win * 256 + 64 * part, ks = (uint32_t)win * 16 + 4 * part;
    const uint32_t mask = mx4_scale_mask(a.K / 32 - (int)ks);
    gmm_u32x4 w[QB][4], x[NB][4];
    uint32_t sw[QB], sx[NB];
#pragma unroll
    for (int j = 0; j < QB; ++j) {
      sw[j] = mx4_load32(rws, wrow[j] * lds + ks);
#pragma unroll
      for (int t = 0; t < 4; ++t) w[j][t] = mx4_load128(rw, kb + 16 * t < ld ? wrow[j] * ld + kb + 16 * t : kMx4Outside);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      sx[i] = mx4_load32(rxs, xrow[i] * lds + ks);
#pragma unroll
      for (int t = 0; t < 4; ++t) x[i][t] = mx4_load128(rx, kb + 16 * t < ld ? xrow[i] * ld + kb + 16 * t : kMx4Outside);
    }
#pragma unroll
    for (int j = 0; j < QB; ++j) sw[j] &= mask;
#pragma unroll
    for (int i = 0; i < NB; ++i) sx[i] &= mask;
    static_for<4>([&](auto tc) {
      constexpr int t = decltype(tc)::value;
#pragma unroll
      for (int j = 0; j < QB; ++j)
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i][j] = mx4_mfma<t, t>(w[j][t], sw[j], x[i][t], sx[i], acc[i][j]);
    });
  }
  // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
  for (int half = W / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < QB; ++j) sums[(((wave - half) * NB + i) * QB + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < QB; ++j) acc[i][j] += sums[((wave * NB + i) * QB + j) * 64 + lane];
    }
    __syncthreads();
  }
  if (wave) return;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = 16 * i + r;
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < QB; ++j) {
        const int col = 16 * j + 4 * part;
        if (col < cols) mx4_store4(a.out, a.out_bf16, (beg + row) * a.N + q0 + col, cols - col, acc[i][j]);
      }
    }
  }
}

template <int PB>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void mx4_stream_kernel(Mx4Args a, int slabs) {
  __shared__ f32x4 sums[kStreamWaves / 2 * PB * kStreamQ * 64];
  GmmTiles tiles;
  tiles.count(a.group_offsets, a.G, a.max_rows, 16 * PB);
  int t, slab, g;
  if (!gmm_row_item(gmm_block(), tiles, slabs, t, slab)) return;
  int64_t beg, end;
  tiles.find(a.group_offsets, a.G, a.max_rows, 16 * PB, t, g, beg, end);
#if defined(__HIP_DEVICE_COMPILE__)
  const int q0 = slab * 16 * kStreamQ, nb = (int)(end - beg + 15) / 16;
#define MOE_MX4_CASE(N) \
  if constexpr (N <= PB) \
    if (nb == N) return stream_body<N>(a, sums, g, beg, end, q0);
  MOE_MX4_CASE(4)
  MOE_MX4_CASE(3)
  MOE_MX4_CASE(2)
  MOE_MX4_CASE(1)
#undef MOE_MX4_CASE
#else
  (void)sums;
#endif
}

}  // namespace

int64_t mx4_stream_grid(const Mx4Args& a, int p_blocks) {
  return gmm_row_grid(a.max_rows, a.G, (a.N + 16 * kStreamQ - 1) / (16 * kStreamQ), 16 * p_blocks);
}

hipError_t launch_mx4_stream(const Mx4Args& a, int p_blocks, hipStream_t s) {
  const int slabs = (a.N + 16 * kStreamQ - 1) / (16 * kStreamQ);
  const dim3 grid = gmm_grid(mx4_stream_grid(a, p_blocks)), block(64 * kStreamWaves);
  if (p_blocks == 1) mx4_stream_kernel<1><<<grid, block, 0, s>>>(a, slabs);
  else mx4_stream_kernel<4><<<grid, block, 0, s>>>(a, slabs);
  return hipGetLastError();
}

}  // namespace moe

// The root-mean-square norm and its gradients.  A row h (h = x + residual, rounded to its type, or x):
//   m = 1 / sqrt(mean h^2 + eps),  y = h m w
//   g = dy w,  dx = m (g - h m^2 mean(g h)) + dh,  dw = sum over rows of dy h m
// in fp32, each output rounded once.  The 8-bit output quantizes y as it is, before any rounding, like
// moe_quantize_rows (row_core.h).
//
// Bound: HBM, each value moved once.  A row stays in the registers of the lanes that share it (64, 256 or 1024 of
// them, chunks of 8 values a lane; 16 where rows are short), from its one load to its last use; every load of a row
// is issued before the first is waited for.  bf16, 7168 columns, with a residual: 8192 rows 77 us (470 MB, 6.1 TB/s;
// a copy reaches 5.2, reads alone 7.0), in 8 bits 72 (5.7), the gradients of 16384 rows 155 and the join 7 (940 MB,
// 6.1).  Few rows: the latency of a load, two joins over the lanes and a store, 2.8 us for one row, 3.9 for 64.
#include "norm.h"
#include "row_core.h"

namespace moe {
namespace {

__device__ __forceinline__ float widened(float v) { return v; }
__device__ __forceinline__ float widened(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void rounded(float v, float* to) { *to = v; }
__device__ __forceinline__ void rounded(float v, uint16_t* to) { *to = f32_to_bf16(v); }

// The weights of a chunk, of either type (uniform); none: ones.
struct RawWeight {
  Raw8<float> v;
  __device__ __forceinline__ void load(const void* w, bool bf16, int c) {
    if (!w) return;
    if (bf16) __builtin_memcpy(v.u, static_cast<const uint16_t*>(w) + c, 16);
    else v.load(static_cast<const float*>(w) + c);
  }
  __device__ __forceinline__ void widen(const void* w, bool bf16) {
    if (!w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v.u[i] = 0x3f800000u;
    } else if (bf16) {
#pragma unroll
      for (int i = 7; i >= 0; --i) v.u[i] = i & 1 ? v.u[i >> 1] & 0xffff0000u : v.u[i >> 1] << 16;
    }
  }
};
__device__ __forceinline__ float weight_at(const void* w, bool bf16, int c) {
  return !w ? 1.f : bf16 ? bf16_to_f32(static_cast<const uint16_t*>(w)[c]) : static_cast<const float*>(w)[c];
}

constexpr int norm_threads(int lanes) { return lanes < 256 ? 256 : lanes; }

// Every lane's value joined over the kLanes lanes of a row, in a fixed order; part: kLanes / 64 values of LDS that
// nobody else uses until the next barrier.
template <int kLanes, class V, class Join>
__device__ __forceinline__ V join_lanes(V v, V* part, const Join& join) {
#pragma unroll
  for (int d = (kLanes < 64 ? kLanes : 64) / 2; d > 0; d >>= 1) v = join(v, __shfl_xor(v, d, 64));
  if constexpr (kLanes > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < kLanes / 64; ++i) v = join(v, part[i]);
  }
  return v;
}

// Lane l has columns 8 l .. 8 l + 7 of every 8 kLanes, and the l-th of the up to 7 that are left behind the row's last
// whole chunk.
// kNt: 1: x, residual and h with the non-temporal policy, 2: y as well.
template <class T, class Out, int kLanes, int kChunks, int kNt>
__global__ __launch_bounds__(norm_threads(kLanes)) void rms_norm_kernel(NormArgs a) {
  constexpr int kRows = norm_threads(kLanes) / kLanes;  // rows of a work-group
  __shared__ float sums[(kLanes + 63) / 64];
  [[maybe_unused]] __shared__ int tops[(kLanes + 63) / 64];
  const int lane = threadIdx.x % kLanes, whole = a.cols / 8 * 8, last = whole + lane;
  const int64_t r = ((int64_t)blockIdx.y * kGmmGridX + blockIdx.x) * kRows + threadIdx.x / kLanes;
  if (r >= a.rows) return;  // all lanes of a row
  const int64_t at = r * a.cols;
  const T* x = static_cast<const T*>(a.x) + at;
  const T* res = static_cast<const T*>(a.residual) + at;
  const bool has_last = last < a.cols;
  Raw8<T> raw[kChunks], add[kChunks];
  RawWeight w[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = 8 * (j * kLanes + lane);
    if (c < whole) raw[j].template load<(kNt > 0)>(x + c);
  }
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) add[j].template load<(kNt > 0)>(res + c);
    }
  }
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = 8 * (j * kLanes + lane);
    if (c < whole) w[j].load(a.w, a.w_bf16, c);
  }
  float h_last = 0.f, sum = 0.f;
  if (has_last) {
    T v = x[last];
    if (a.residual) {
      rounded(widened(v) + widened(res[last]), &v);
      static_cast<T*>(a.h)[at + last] = v;
    }
    h_last = widened(v);
    sum = h_last * h_last;
  }
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = 8 * (j * kLanes + lane);
    if (c < whole) {
      if (a.residual) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = raw[j][i] + add[j][i];
        raw[j].round(v);
        raw[j].template store<(kNt > 0)>(static_cast<T*>(a.h) + at + c);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += raw[j][i] * raw[j][i];
    }
  }
  sum = join_lanes<kLanes>(sum, sums, [](float p, float q) { return p + q; });
  const float m = 1.f / sqrtf(sum / a.cols + a.eps);
  float y_last = 0.f;
  if (has_last) y_last = h_last * m * weight_at(a.w, a.w_bf16, last);
  if constexpr (sizeof(Out) > 1) {
    Out* out = static_cast<Out*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) {
        w[j].widen(a.w, a.w_bf16);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = raw[j][i] * m * w[j].v[i];
        Raw8<Out> o;
        o.round(y);
        o.template store<(kNt > 1)>(out + c);
      }
    }
    if (has_last) rounded(y_last, out + last);
  } else {
    float y[kChunks][8];
    uint32_t top = __float_as_uint(y_last) & 0x7fffffffu;
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
      if (8 * (j * kLanes + lane) < whole) {
        w[j].widen(a.w, a.w_bf16);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[j][i] = raw[j][i] * m * w[j].v[i];
        top = abs_bits_max(y[j], top);
      }
    top = (uint32_t)join_lanes<kLanes>((int)top, tops, [](int p, int q) { return p > q ? p : q; });
    const bool finite = top < 0x7f800000u;
    if (lane == 0) a.scales[r] = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7fc00000u);
    const RowScale rs = row_scale(finite ? top : 0u);
    int8_t* codes = static_cast<int8_t*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) {
        if (!finite) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[j][i] = 0.f;
        }
        store_codes8(codes + c, 8, y[j], rs);
      }
    }
    if (has_last) {
      const float v[8] = {finite ? y_last : 0.f};
      store_codes8(codes + last, 1, v, rs);
    }
  }
}

// Rows r, r + gridDim.x * kRows, ... of a work-group's kRows sets of kLanes lanes; dw of its rows stays in registers
// and leaves once, as row blockIdx.x of part.  kHold: so do the weights, and dh is read ahead; without, both are read
// where they are used (the weights twice a row, from the cache), for rows that leave no registers for them.  D: the
// type of dy.
template <class T, class D, int kLanes, int kChunks, bool kHold, bool kNt>
__global__ __launch_bounds__(norm_threads(kLanes), 2) void norm_grad_kernel(NormGradArgs a) {
  constexpr int kRows = norm_threads(kLanes) / kLanes;
  struct Two {
    float h2, gh;
  };
  __shared__ Two sums[2][(kLanes + 63) / 64];  // of even and odd turns
  const int lane = threadIdx.x % kLanes, whole = a.cols / 8 * 8, last = whole + lane;
  const bool has_last = last < a.cols;
  RawWeight w[kHold ? kChunks : 1];
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) w[j].load(a.w, a.w_bf16, c);
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
      if (8 * (j * kLanes + lane) < whole) w[j].widen(a.w, a.w_bf16);
  }
  const auto weights = [&](int j, int c) -> const RawWeight& {
    if constexpr (kHold) return w[j];
    w[0].load(a.w, a.w_bf16, c);
    w[0].widen(a.w, a.w_bf16);
    return w[0];
  };
  const float w_last = has_last ? weight_at(a.w, a.w_bf16, last) : 0.f;
  float dw[kChunks][8], dw_last = 0.f;
#pragma unroll
  for (int j = 0; j < kChunks; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes; r < a.rows; r += (int64_t)gridDim.x * kRows) {
    const int64_t at = r * a.cols;
    const D* pdy = static_cast<const D*>(a.dy) + at;
    const T* ph = static_cast<const T*>(a.h) + at;
    const T* pdh = static_cast<const T*>(a.dh) + at;
    Raw8<D> dy[kChunks];
    Raw8<T> h[kChunks];
    [[maybe_unused]] Raw8<T> dh[kHold ? kChunks : 1];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) {
        dy[j].template load<(kNt && sizeof(D) == 2)>(pdy + c);
        h[j].template load<kNt>(ph + c);
      }
    }
    if constexpr (kHold)
      if (a.dh) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          const int c = 8 * (j * kLanes + lane);
          if (c < whole) dh[j].template load<kNt>(pdh + c);
        }
      }
    float h2 = 0.f, gh = 0.f, dy_last = 0.f, h_last = 0.f;
    if (has_last) {
      dy_last = widened(pdy[last]);
      h_last = widened(ph[last]);
      h2 = h_last * h_last;
      gh = dy_last * w_last * h_last;
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) {
        const RawWeight& wj = weights(j, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h2 += h[j][i] * h[j][i];
          gh += dy[j][i] * wj.v[i] * h[j][i];
        }
      }
    }
#pragma unroll
    for (int d = (kLanes < 64 ? kLanes : 64) / 2; d > 0; d >>= 1) {
      h2 += __shfl_xor(h2, d, 64);
      gh += __shfl_xor(gh, d, 64);
    }
    if constexpr (kLanes > 64) {  // the barrier of one turn lies between two uses of the same half
      if ((threadIdx.x & 63) == 0) sums[turn][threadIdx.x >> 6] = Two{h2, gh};
      __syncthreads();
      h2 = gh = 0.f;
#pragma unroll
      for (int i = 0; i < kLanes / 64; ++i) {
        h2 += sums[turn][i].h2;
        gh += sums[turn][i].gh;
      }
      turn ^= 1;
    }
    const float m = 1.f / sqrtf(h2 / a.cols + a.eps), k = gh / a.cols * m * m;
    T* pdx = static_cast<T*>(a.dx) + at;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) {
        const RawWeight& wj = weights(j, c);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = m * (dy[j][i] * wj.v[i] - h[j][i] * k);
          dw[j][i] += dy[j][i] * (h[j][i] * m);
        }
        if (a.dh) {
          Raw8<T>& d = dh[kHold ? j : 0];
          if constexpr (!kHold) d.template load<kNt>(pdh + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += d[i];
        }
        Raw8<T> o;
        o.round(v);
        o.template store<kNt>(pdx + c);
      }
    }
    if (has_last) {
      float v = m * (dy_last * w_last - h_last * k);
      if (a.dh) v += widened(pdh[last]);
      rounded(v, pdx + last);
      dw_last += dy_last * (h_last * m);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * norm_grad_ld(a.cols);
  if constexpr (kRows > 1) {  // the sets' sums, in their order
    __shared__ float all[kRows][kChunks * kLanes * 8 + 8];
    float* mine = all[threadIdx.x / kLanes];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) __builtin_memcpy(mine + c, dw[j], 32);
    }
    if (has_last) mine[last] = dw_last;
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += norm_threads(kLanes)) {
      float v = all[0][c];
#pragma unroll
      for (int i = 1; i < kRows; ++i) v += all[i][c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = 8 * (j * kLanes + lane);
      if (c < whole) __builtin_memcpy(part + c, dw[j], 32);
    }
    if (has_last) part[last] = dw_last;
  }
}

constexpr int kJoinCols = 32, kJoinThreads = 256;

// 32 columns a work-group: 8 lanes of 4 columns, 32 of them over the parts.
__global__ __launch_bounds__(kJoinThreads) void norm_grad_join_kernel(const float* part, int parts, int cols, void* dw,
                                                                      bool bf16) {
  __shared__ f32x4 all[kJoinThreads / 8][8];
  const int q = threadIdx.x % 8, p0 = threadIdx.x / 8;
  const int64_t ld = norm_grad_ld(cols);
  const int c0 = blockIdx.x * kJoinCols + 4 * q;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int p = p0; p < parts; p += kJoinThreads / 8) sum += *reinterpret_cast<const f32x4*>(part + p * ld + c0);
  all[p0][q] = sum;
  __syncthreads();
  if (threadIdx.x >= kJoinCols) return;
  const int c = blockIdx.x * kJoinCols + threadIdx.x;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 8; ++i) v += all[i][threadIdx.x / 4][threadIdx.x % 4];
  if (c < cols) {
    if (bf16) static_cast<uint16_t*>(dw)[c] = f32_to_bf16(v);
    else static_cast<float*>(dw)[c] = v;
  }
}

// Lanes that share a row: few, so that a wave has many loads in flight and no barrier, but enough for a lane to hold
// its share.  The norm of few rows: more lanes, for a shorter way through each (64 rows of 2048: 4.3 us with 64
// lanes, 3.3 with 256; of 7168: 4.5 with 256, 3.9 with 1024; 1024 rows of 7168: 10.8 and 14.3).
int lanes_of(int32_t cols) { return cols <= 2048 ? 64 : cols <= 8192 ? 256 : 1024; }
// Short rows (those of heads, say): 16 lanes, four rows to a wave, where there are many of them (bf16, 262144 rows of
// 128, 16 and 64 lanes: 23.6 us and 64.8, with 8-bit output 27 and 92; of 512: 85 and 111, 66 and 110; fp32 of 512:
// 183 and 183, 118 and 150; 600 rows of 512: 3.5 and 3.1; 4096 of 512 with a residual: 5.6 and 4.8, of 256 4.2 and
// 4.2).
bool short_rows(int64_t rows, int32_t cols) { return cols <= 512 && rows > (cols <= 256 ? 512 : 8192); }
// Gradients, both launches, 16 and 64 lanes, bf16: 262144 rows of 128 45 us and 146, of 512 135 and 193; 8192 of 512
// 13.2 and 14.4; 520 of 512 6.6 and 6.8.  fp32: 262144 rows of 256 147 and 184; 4096 of 512 11.3 and 13.0; 64 where
// both are many: 8192 of 512 18.2 and 17.4, 262144 308 and 293, of 400 250 and 234; of 384 and less either by up to
// 5%.
int grad_lanes(int64_t rows, int32_t cols, bool bf16) {
  const bool narrow = cols <= 512 && rows > 512;
  return narrow && (bf16 || cols <= 384 || rows < 8192) ? 16 : lanes_of(cols);
}
int norm_lanes(int64_t rows, int32_t cols) {
  const int lanes = lanes_of(cols);
  if (short_rows(rows, cols)) return 16;
  return rows > 512 || cols <= 512 ? lanes : lanes == 64 ? 256 : 1024;
}

template <class T, class Out, int kNt>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const int lanes = norm_lanes(a.rows, a.cols), threads = norm_threads(lanes), per = threads / lanes;
  const dim3 grid = gmm_grid((a.rows + per - 1) / per);
  if (lanes == 16) rms_norm_kernel<T, Out, 16, 4, kNt><<<grid, threads, 0, s>>>(a);
  else if (lanes == 64) rms_norm_kernel<T, Out, 64, 4, kNt><<<grid, threads, 0, s>>>(a);
  else if (lanes == 256) rms_norm_kernel<T, Out, 256, 4, kNt><<<grid, threads, 0, s>>>(a);
  else rms_norm_kernel<T, Out, 1024, 4, kNt><<<grid, threads, 0, s>>>(a);
  return hipGetLastError();
}

// y, which what follows reads, with the non-temporal policy only where the cache could not keep most of it.
template <class T, class Out>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const int64_t n = a.rows * a.cols;
  if constexpr (sizeof(T) == 2) {
    if constexpr (sizeof(Out) == 2)
      if (n >= (int64_t)100 << 20) return launch_norm<T, Out, 2>(a, s);
    if (row_streams<T>(n)) return launch_norm<T, Out, 1>(a, s);
  }
  return launch_norm<T, Out, 0>(a, s);
}

template <class T, class D, bool kNt>
hipError_t launch_grad(const NormGradArgs& a, hipStream_t s) {
  const int lanes = grad_lanes(a.rows, a.cols, a.bf16), threads = norm_threads(lanes);
  const int grid = norm_grad_parts(a.rows, a.cols);
  if (lanes == 16) norm_grad_kernel<T, D, 16, 4, true, kNt><<<grid, threads, 0, s>>>(a);
  else if (lanes == 64) norm_grad_kernel<T, D, 64, 4, true, kNt><<<grid, threads, 0, s>>>(a);
  else if (lanes == 256) norm_grad_kernel<T, D, 256, 4, true, kNt><<<grid, threads, 0, s>>>(a);
  else if (a.cols <= 1024 * 8 * 2) norm_grad_kernel<T, D, 1024, 2, true, kNt><<<grid, threads, 0, s>>>(a);
  else norm_grad_kernel<T, D, 1024, 4, false, kNt><<<grid, threads, 0, s>>>(a);
  return hipGetLastError();
}
template <class T, class D>
hipError_t launch_grad(const NormGradArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (row_streams<T>(a.rows * a.cols)) return launch_grad<T, D, true>(a, s);
  return launch_grad<T, D, false>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, NormOut out, hipStream_t s) {
  if (a.bf16)
    return out == NormOut::kI8     ? launch_norm<uint16_t, int8_t>(a, s)
           : out == NormOut::kBf16 ? launch_norm<uint16_t, uint16_t>(a, s)
                                   : launch_norm<uint16_t, float>(a, s);
  return out == NormOut::kI8     ? launch_norm<float, int8_t>(a, s)
         : out == NormOut::kBf16 ? launch_norm<float, uint16_t>(a, s)
                                 : launch_norm<float, float>(a, s);
}

// As many work-groups as run at once, two on a CU or one of 1024 lanes: more write more sums and gain nothing (32768
// rows of 1024: 49 us with 512, 59 with 1024; 2048 of 16384: 79 with 256, 89 with 512).  The same for either type:
// from 8192 rows on 16 lanes to a row make as many of them as 64.
int norm_grad_parts(int64_t rows, int32_t cols) {
  const int lanes = grad_lanes(rows, cols, true), per = norm_threads(lanes) / lanes;
  const int64_t most = lanes == 1024 ? 256 : 512, groups = (rows + per - 1) / per;
  return (int)(groups < most ? groups : most);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (!a.bf16) return launch_grad<float, float>(a, s);
  return a.dy_f32 ? launch_grad<uint16_t, float>(a, s) : launch_grad<uint16_t, uint16_t>(a, s);
}

hipError_t launch_norm_grad_join(const float* part, int parts, int32_t cols, void* dw, bool dw_bf16, hipStream_t s) {
  norm_grad_join_kernel<<<(cols + kJoinCols - 1) / kJoinCols, kJoinThreads, 0, s>>>(part, parts, cols, dw, dw_bf16);
  return hipGetLastError();
}

}  // namespace moe

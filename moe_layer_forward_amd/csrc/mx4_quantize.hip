// Rows to microscaled 4 bits and back (layout: mx4.h).  A block of 32 values with a = max |v| gets the scale
// 2^X, X = max(floor(log2 a) - 2, -127), which brings a into [4, 8); a value's code is the nearest of
// +-{0, 1/2, 1, 3/2, 2, 3, 4, 6} to v 2^-X, ties to the even code, beyond 6 to 6 (v_cvt_scalef32_pk_fp4_f32: exact,
// since the scale is a power of two).  A block with an infinity or a NaN gets the scale 255 (NaN) and codes 0.
//
// Bound: HBM (with SwiGLU of bf16 rows the vector unit as well: 8192 x 7168 in 55 us, 4.8 TB/s).  A wave takes
// windows of 512 values of a row, 8 a lane: four lanes share a block, and its codes and scales leave as 256 and 16
// consecutive bytes.  Large matrices: four windows to a wave, all loaded before the first is used (one at a time: 32
// KB in flight on a CU, 4.1 TB/s of reads and writes; four: 5.8 at 8192 x 7168 bf16, 25.4 us, and 6.3 at 18432 x
// 7168, 53 us; back 22.8 and 48.7).
#include "mx4.h"
#include "row_core.h"
#include "tile_core.h"

namespace moe {
namespace {

constexpr int kMx4Threads = 256, kMx4Window = 512;

// Window number n, counted row by row.
struct Window {
  int64_t row;
  int win;
};
__device__ __forceinline__ Window window_at(int64_t n, int per_row) {
  Window w;
  w.row = n >> 32 ? n / per_row : (uint32_t)n / (uint32_t)per_row;
  w.win = (int)(n - w.row * per_row);
  return w;
}
__device__ __forceinline__ int64_t first_window(int turns) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  return (((int64_t)blockIdx.y * kGmmGridX + blockIdx.x) * (kMx4Threads / 64) + wave) * turns;
}

// max over the four lanes of a block
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true);  // lane ^ 1
  m = o > m ? o : m;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, true);  // lane ^ 2
  return o > m ? o : m;
}

// v = swiglu_f32(gate, up) bit for bit, with a reciprocal in place of its division: the hardware's is off by a unit
// at most, and a step of Newton's method in fused multiply-adds rounds it correctly (compared with the division for
// every fp32 number of [1, 2^126)).  From 2^126 on (gates below -87.3), where it is subnormal, the division itself.
// bf16, 8192 x 7168: 55 us, with the division everywhere 66; 8192 x 2048: 16.8 and 20.5.
template <class In>
__device__ __forceinline__ void swiglu8(const Raw8<In>& gate, const Raw8<In>& up, float (&v)[8]) {
  float d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = 1.f + expf(-gate[i]);
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = __builtin_amdgcn_rcpf(d[i]);
    r[i] = __builtin_fmaf(__builtin_fmaf(-d[i], r[i], 1.f), r[i], r[i]);
  }
  if (__builtin_expect(abs_bits_max(d, 0) >= 0x7e800000u, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 1.f / d[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = gate[i] * r[i] * up[i];
}

// A lane's 8 values of a block (zeros where there are none): the bits of their largest magnitude, at or above those of
// infinity for infinities and NaN, and their codes in units of `unit`.
template <class In, bool kSwiglu>
struct Block8 {
  float v[8];
  __device__ __forceinline__ Block8(const Raw8<In>& x, const Raw8<In>& up, bool some) {
    if constexpr (kSwiglu) {
      swiglu8(x, up, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = some ? v[i] : 0.f;
  }
  __device__ __forceinline__ uint32_t top() const { return abs_bits_max(v, 0); }
  __device__ __forceinline__ uint32_t codes(float unit) const {
    uint32_t q = 0;
    static_for<4>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2 * i], v[2 * i + 1], unit, i);
    });
    return q;
  }
};
template <>  // bf16 as it is, two to a register
struct Block8<uint16_t, false> {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  uint32_t u[4];
  __device__ __forceinline__ Block8(const Raw8<uint16_t>& x, const Raw8<uint16_t>&, bool some) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = some ? x.u[i] : 0;
  }
  __device__ __forceinline__ uint32_t top() const {
    u16x2 m = __builtin_bit_cast(u16x2, u[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, u[i] & 0x7fff7fffu));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
  __device__ __forceinline__ uint32_t codes(float unit) const {
    uint32_t q = 0;
    static_for<4>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, u[i]), unit, i);
    });
    return q;
  }
};

template <class In, bool kSwiglu, int kTurns, bool kNt>
__global__ __launch_bounds__(kMx4Threads) void quantize_mx4_kernel(const In* x, int64_t rows, int cols, int per_row,
                                                                   uint8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 63;
  const int64_t n0 = first_window(kTurns), windows = rows * per_row;
  Raw8<In> raw[kTurns], up[kSwiglu ? kTurns : 1];
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const Window at = window_at(n0 + t, per_row);
    const int c = at.win * kMx4Window + 8 * lane;
    if (n0 + t < windows && c < cols) {
      const In* p = x + at.row * cols * (kSwiglu ? 2 : 1) + c;
      raw[t].template load<kNt>(p);
      if constexpr (kSwiglu) up[t].template load<kNt>(p + cols);
    }
  }
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    if (n0 + t >= windows) return;
    const Window at = window_at(n0 + t, per_row);
    const int c = at.win * kMx4Window + 8 * lane;
    const Block8<In, kSwiglu> v(raw[t], up[kSwiglu ? t : 0], c < cols);
    const uint32_t m = quad_max(v.top());
    const bool finite = m < 0x7f800000u;
    const uint32_t e = m >> 23, s = e > 2 ? e - 2 : 0;
    const uint32_t q = finite ? v.codes(__uint_as_float(s ? s << 23 : 0x00400000u)) : 0;
    if (c < cols) __builtin_memcpy(codes + at.row * (cols / 2) + c / 2, &q, 4);
    if ((lane & 3) == 0) scales[(n0 + t) * 16 + lane / 4] = (uint8_t)(c >= cols ? 0 : finite ? s : 255);
  }
}

// The values of 8 codes of a block with scale s.
template <class Out>
__device__ __forceinline__ void decode8(uint32_t q, uint32_t s, Raw8<Out>& o) {
  const float unit = __uint_as_float(s == 255 ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
  float v[8];  // magnitudes exact in fp32, then times the power of two
  static_for<4>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    const auto two = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, i);
    v[2 * i] = two[0] * unit;
    v[2 * i + 1] = two[1] * unit;
  });
  o.round(v);
}

template <class Out, int kTurns, bool kNt>
__global__ __launch_bounds__(kMx4Threads) void dequantize_mx4_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                     int64_t rows, int cols, int per_row, Out* y) {
  const int lane = threadIdx.x & 63;
  const int64_t n0 = first_window(kTurns), windows = rows * per_row;
  uint32_t codes8[kTurns], scale[kTurns];
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const Window at = window_at(n0 + t, per_row);
    const int c = at.win * kMx4Window + 8 * lane;
    if (n0 + t < windows && c < cols) {
      __builtin_memcpy(&codes8[t], codes + at.row * (cols / 2) + c / 2, 4);
      scale[t] = scales[(n0 + t) * 16 + lane / 4];
    }
  }
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const Window at = window_at(n0 + t, per_row);
    const int c = at.win * kMx4Window + 8 * lane;
    if (n0 + t >= windows || c >= cols) continue;
    Raw8<Out> o;
    decode8(codes8[t], scale[t], o);
    o.template store<kNt>(y + at.row * cols + c);
  }
}

// Rows of up to 8 L values: L lanes to a row, 64 / L rows to a wave.
template <class In, bool kSwiglu, int L>
__global__ __launch_bounds__(kMx4Threads) void quantize_mx4_short_kernel(const In* x, int64_t rows, int cols,
                                                                         uint8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 63, part = lane % L, c = 8 * part;
  const int64_t r = first_window(64 / L) + lane / L;
  const bool some = r < rows && c < cols;
  Raw8<In> raw, up;
  if (some) {
    const In* p = x + r * cols * (kSwiglu ? 2 : 1) + c;
    raw.load(p);
    if constexpr (kSwiglu) up.load(p + cols);
  }
  const Block8<In, kSwiglu> v(raw, up, some);
  const uint32_t m = quad_max(v.top());
  const bool finite = m < 0x7f800000u;
  const uint32_t e = m >> 23, s = e > 2 ? e - 2 : 0;
  const uint32_t q = finite ? v.codes(__uint_as_float(s ? s << 23 : 0x00400000u)) : 0;
  if (some) __builtin_memcpy(codes + r * (cols / 2) + c / 2, &q, 4);
  // the row's scales, up to 8 of its 16 bytes, in its first lane
  const uint32_t byte = !some ? 0 : finite ? s : 255;
  uint32_t all[2] = {part < 16 ? byte << part / 4 * 8 : 0, part < 16 ? 0 : byte << (part / 4 - 4) * 8};
#pragma unroll
  for (int d = 4; d < L; d <<= 1) {
    all[0] |= __shfl_xor(all[0], d, 64);
    if constexpr (L > 16) all[1] |= __shfl_xor(all[1], d, 64);
  }
  if (part == 0 && r < rows) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<u32x4*>(scales + r * 16) = u32x4{all[0], all[1], 0, 0};
  }
}

template <class Out, int L>
__global__ __launch_bounds__(kMx4Threads) void dequantize_mx4_short_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                           int64_t rows, int cols, Out* y) {
  const int lane = threadIdx.x & 63, part = lane % L, c = 8 * part;
  const int64_t r = first_window(64 / L) + lane / L;
  if (r >= rows || c >= cols) return;
  uint32_t q;
  __builtin_memcpy(&q, codes + r * (cols / 2) + c / 2, 4);
  const uint32_t s = scales[r * 16 + part / 4];
  Raw8<Out> o;
  decode8(q, s, o);
  o.template store<false>(y + r * cols + c);
}

// Four windows to a wave where that leaves 16 waves for every SIMD.
struct Mx4Grid {
  int per_row;
  bool four, nt;
  dim3 grid;
  Mx4Grid(int64_t rows, int32_t cols, bool streams) {
    nt = streams;
    per_row = mx4_scale_cols(cols) / 16;
    const int64_t windows = rows * per_row;
    four = nt || windows >= (int64_t)1 << 16;
    const int64_t per = (four ? 4 : 1) * (kMx4Threads / 64);
    grid = gmm_grid((windows + per - 1) / per);
  }
};

// Rows of up to 256 values: several to a wave (bf16, 65536 rows of 64: 12.4 -> 3.6 us, back 11.8 -> 3.9; of 256: 12.4
// -> 9.1, 13.0 -> 8.4; 262144 of 128: 37.6 -> 15.4; with SwiGLU 65536 of 64: 5.6).
constexpr int kMx4Short = 256;
int short_lanes(int32_t cols) { return cols <= 64 ? 8 : cols <= 128 ? 16 : 32; }
dim3 short_grid(int64_t rows, int lanes) {
  const int64_t per = kMx4Threads / lanes;
  return gmm_grid((rows + per - 1) / per);
}

template <class In, bool kSwiglu>
void launch_q(const Mx4Grid& g, const void* x, int64_t rows, int32_t cols, uint8_t* codes, uint8_t* scales,
              hipStream_t s) {
  if (cols <= kMx4Short) {
    const int lanes = short_lanes(cols);
    const auto go = [&](auto kernel) {
      kernel<<<short_grid(rows, lanes), kMx4Threads, 0, s>>>(static_cast<const In*>(x), rows, cols, codes, scales);
    };
    return lanes == 8    ? go(quantize_mx4_short_kernel<In, kSwiglu, 8>)
           : lanes == 16 ? go(quantize_mx4_short_kernel<In, kSwiglu, 16>)
                         : go(quantize_mx4_short_kernel<In, kSwiglu, 32>);
  }
  const auto go = [&](auto kernel) {
    kernel<<<g.grid, kMx4Threads, 0, s>>>(static_cast<const In*>(x), rows, cols, g.per_row, codes, scales);
  };
  if constexpr (sizeof(In) == 2)
    if (g.nt) return go(quantize_mx4_kernel<In, kSwiglu, 4, true>);
  if (g.four) go(quantize_mx4_kernel<In, kSwiglu, 4, false>);
  else go(quantize_mx4_kernel<In, kSwiglu, 1, false>);
}

template <class Out>
void launch_d(const Mx4Grid& g, const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* y,
              hipStream_t s) {
  if (cols <= kMx4Short) {
    const int lanes = short_lanes(cols);
    const auto go = [&](auto kernel) {
      kernel<<<short_grid(rows, lanes), kMx4Threads, 0, s>>>(codes, scales, rows, cols, static_cast<Out*>(y));
    };
    return lanes == 8    ? go(dequantize_mx4_short_kernel<Out, 8>)
           : lanes == 16 ? go(dequantize_mx4_short_kernel<Out, 16>)
                         : go(dequantize_mx4_short_kernel<Out, 32>);
  }
  const auto go = [&](auto kernel) {
    kernel<<<g.grid, kMx4Threads, 0, s>>>(codes, scales, rows, cols, g.per_row, static_cast<Out*>(y));
  };
  if constexpr (sizeof(Out) == 2)
    if (g.nt) return go(dequantize_mx4_kernel<Out, 4, true>);
  if (g.four) go(dequantize_mx4_kernel<Out, 4, false>);
  else go(dequantize_mx4_kernel<Out, 1, false>);
}

}  // namespace

hipError_t launch_quantize_mx4(const void* x, bool x_bf16, int64_t rows, int32_t cols, bool swiglu, uint8_t* codes,
                               uint8_t* scales, hipStream_t s) {
  const Mx4Grid g(rows, cols, x_bf16 && row_streams<uint16_t>(rows * cols * (swiglu ? 2 : 1)));
  if (x_bf16) swiglu ? launch_q<uint16_t, true>(g, x, rows, cols, codes, scales, s)
                     : launch_q<uint16_t, false>(g, x, rows, cols, codes, scales, s);
  else swiglu ? launch_q<float, true>(g, x, rows, cols, codes, scales, s)
              : launch_q<float, false>(g, x, rows, cols, codes, scales, s);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* y,
                                 bool y_bf16, hipStream_t s) {
  const Mx4Grid g(rows, cols, y_bf16 && row_streams<uint16_t>(rows * cols));
  if (y_bf16) launch_d<uint16_t>(g, codes, scales, rows, cols, y, s);
  else launch_d<float>(g, codes, scales, rows, cols, y, s);
  return hipGetLastError();
}

}  // namespace moe

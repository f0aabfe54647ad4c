// Grouped matrix products for any sizes, alignment and type: the plain kernel that every call can take.
//
// Tile 128 x 128, 4 waves in 2 x 2, each 64 x 64 outputs (16 accumulator blocks).  Both operands are
// read into registers one step ahead, 16 bytes a lane at whatever alignment the rows have (odd row
// lengths), with the ends of rows filled with zeros element by element, and stored into one of two
// LDS stages while the other is multiplied.  Contraction indices past the end are zero in both
// operands, so no neighbouring row's values, finite or not, enter a sum.
// Bound: the loads (a 16-byte load of an odd row touches two segments) and their trip through
// registers; see launch_gmm for when the tile kernel takes a call instead.
#include "gmm_core.h"

namespace moe {
namespace {

constexpr int kAnyTile = 128;
constexpr int kAnyThreads = 256;

// nv of the n elements at p (n = 16 bytes of them), zeros after them.
template <class T>
__device__ __forceinline__ gmm_u32x4 load_chunk(const char* p, int nv) {
  constexpr int kN = 16 / T::kBytes;
  gmm_u32x4 v = {0, 0, 0, 0};
  if (nv >= kN) {
    __builtin_memcpy(&v, p, 16);
  } else if (nv > 0) {
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
  return v;
}

// One operand's share of a thread: 4 chunks of a stage (1024 chunks over 256 threads).
// L = GmmAlong: chunk q is chunk q % 8 of tile row q / 8, whose elements run along the contraction.
// L = GmmAcross: chunk q is columns of contraction row q / kChunks.
template <class T, class L>
struct AnyOperand {
  const char* base;         // element [0, 0] of the operand matrix of this tile's group
  int64_t ld;               // bytes between rows
  int64_t first;            // first row (Along) or first column (Across) of the tile
  int64_t outer;            // rows (Along) or columns (Across) that exist
  int64_t depth;            // length of the contraction
  const int32_t* index;     // row gather (rows of the tile, or contraction rows), or null
  int64_t index_rows;       // rows the gathered matrix has

  __device__ __forceinline__ int64_t row_of(int64_t r) const {
    if (!index) return r;
    const int64_t i = index[r];
    return i < 0 ? 0 : i >= index_rows ? index_rows - 1 : i;
  }

  __device__ __forceinline__ void load(int64_t kt, gmm_u32x4 (&v)[4]) const {
    constexpr int kN = 16 / T::kBytes;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = threadIdx.x + kAnyThreads * j;
      const int r = q / L::kChunks, c = q % L::kChunks;
      int64_t row, col, nv;
      if constexpr (L::kAlong) {
        row = first + r;
        col = kt * (kGmmStepBytes / T::kBytes) + c * kN;
        nv = row < outer ? depth - col : 0;
      } else {
        row = kt * L::kRows + r;
        col = first + c * kN;
        nv = row < depth ? outer - col : 0;
      }
      const int n = nv <= 0 ? 0 : nv >= kN ? kN : (int)nv;
      v[j] = gmm_u32x4{0, 0, 0, 0};
      if (n > 0) v[j] = load_chunk<T>(base + row_of(row) * ld + col * T::kBytes, n);
    }
  }
  __device__ static __forceinline__ void store(char* stage, const gmm_u32x4 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = threadIdx.x + kAnyThreads * j;
      *reinterpret_cast<gmm_u32x4*>(stage + L::pos(q / L::kChunks, q % L::kChunks)) = v[j];
    }
  }
};

template <class T>
__device__ __forceinline__ void store_out(const GmmArgs& a, void* out, int64_t row, int64_t col, int64_t ld, float v) {
  if (a.out_bf16)
    static_cast<uint16_t*>(out)[row * ld + col] = f32_to_bf16(v);
  else
    static_cast<float*>(out)[row * ld + col] = v;
}

template <GmmForm F, class T>
__global__ __launch_bounds__(kAnyThreads) void gmm_any_kernel(GmmArgs a) {
  using LP = GmmP<F, T, kAnyTile>;
  using LQ = GmmQ<F, T, kAnyTile>;
  __shared__ __align__(16) char p_lds[2][LP::kStageBytes], q_lds[2][LQ::kStageBytes];

  // which tile: NT / NN a row tile of a group x a column slab, TN a (group, n tile, k tile)
  const int64_t q_len = F == GmmForm::kNT ? a.N : a.K;
  const int64_t q_tiles = (q_len + kAnyTile - 1) / kAnyTile;
  const int64_t t = blockIdx.x / q_tiles;
  const int64_t q0 = (blockIdx.x % q_tiles) * kAnyTile;
  int g;
  int64_t beg, end, p0 = 0;
  if constexpr (F == GmmForm::kTN) {
    const int64_t p_tiles = ((int64_t)a.N + kAnyTile - 1) / kAnyTile;
    g = (int)(t / p_tiles);
    p0 = (t % p_tiles) * kAnyTile;
    gmm_group_rows(a.group_offsets, a.max_rows, g, beg, end);
  } else {
    if (!gmm_find_tile(a.group_offsets, a.G, a.max_rows, kAnyTile, t, g, beg, end)) return;
  }
  const char* w = static_cast<const char*>(a.w);
  if (F != GmmForm::kTN) w += (int64_t)g * a.N * a.K * T::kBytes;

  AnyOperand<T, LP> p;
  AnyOperand<T, LQ> q;
  int64_t depth;
  if constexpr (F == GmmForm::kNT) {
    depth = a.K;
    p = {static_cast<const char*>(a.x), (int64_t)a.K * T::kBytes, beg, end, depth, a.row_index, a.x_rows};
    q = {w, (int64_t)a.K * T::kBytes, q0, a.N, depth, nullptr, 0};
  } else if constexpr (F == GmmForm::kNN) {
    depth = a.N;
    p = {static_cast<const char*>(a.dy), (int64_t)a.N * T::kBytes, beg, end, depth, nullptr, 0};
    q = {w, (int64_t)a.K * T::kBytes, q0, a.K, depth, nullptr, 0};
  } else {
    depth = end - beg;
    const int64_t ldn = (int64_t)a.N * T::kBytes, ldk = (int64_t)a.K * T::kBytes;
    p = {static_cast<const char*>(a.dy) + beg * ldn, ldn, p0, a.N, depth, nullptr, 0};
    q = {static_cast<const char*>(a.x) + (a.row_index ? 0 : beg * ldk), ldk, q0, a.K, depth,
         a.row_index ? a.row_index + beg : nullptr, a.x_rows};
  }

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int pw = (wave >> 1) * 4, qw = (wave & 1) * 4;  // first 16-block of the wave's rows and columns
  const auto lp = LP::lane();
  const auto lq = LQ::lane();
  typename T::Acc acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[i][s] = typename T::Acc{0, 0, 0, 0};

  constexpr int kStep = kGmmStepBytes / T::kBytes;
  const int64_t nk = (depth + kStep - 1) / kStep;
  gmm_u32x4 pv[4], qv[4];
  if (nk > 0) {
    p.load(0, pv);
    q.load(0, qv);
    p.store(p_lds[0], pv);
    q.store(q_lds[0], qv);
  }
  __syncthreads();
  for (int64_t kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    if (kt + 1 < nk) {
      p.load(kt + 1, pv);
      q.load(kt + 1, qv);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      gmm_u32x4 qf[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) qf[s] = LQ::frag(q_lds[cur], lq, qw + s, kk);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const gmm_u32x4 pf = LP::frag(p_lds[cur], lp, pw + i, kk);
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[i][s] = T::mfma(qf[s], pf, acc[i][s]);
      }
    }
    if (kt + 1 < nk) {
      p.store(p_lds[cur ^ 1], pv);
      q.store(q_lds[cur ^ 1], qv);
    }
    __syncthreads();
  }

  // TN: rows are columns of dy, written into dW[g]; otherwise rows [beg, end)
  const int64_t row0 = F == GmmForm::kTN ? p0 : beg, row_end = F == GmmForm::kTN ? (int64_t)a.N : end;
  char* out = static_cast<char*>(a.out);
  if (F == GmmForm::kTN) out += (int64_t)g * a.N * a.K * (a.out_bf16 ? 2 : 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 16 * (pw + i) + (lane & 15);
    if (row >= row_end) continue;
    float sx = 1.f;
    if constexpr (std::is_same_v<T, GmmI8>) sx = a.x_scales[p.row_of(row)];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t col = q0 + 16 * (qw + s) + 4 * (lane >> 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (col + e >= q_len) continue;
        float v = (float)acc[i][s][e];
        if constexpr (std::is_same_v<T, GmmI8>) v = v * sx * a.w_scales[(int64_t)g * a.N + col + e];
        store_out<T>(a, out, row, col + e, q_len, v);
      }
    }
  }
}

template <GmmForm F, class T>
hipError_t launch_any(const GmmArgs& a, hipStream_t s) {
  gmm_any_kernel<F, T><<<dim3((unsigned)gmm_any_grid(a)), dim3(kAnyThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t gmm_any_grid(const GmmArgs& a) {
  const int64_t q_tiles = ((a.form == GmmForm::kNT ? a.N : a.K) + kAnyTile - 1) / kAnyTile;
  const int64_t p_tiles = a.form == GmmForm::kTN ? (int64_t)a.G * ((a.N + kAnyTile - 1) / kAnyTile)
                                                 : gmm_max_tiles(a.max_rows, a.G, kAnyTile);
  return p_tiles * q_tiles;
}

hipError_t launch_gmm_any(const GmmArgs& a, hipStream_t s) {
  switch (a.form) {
    case GmmForm::kNT:
      if (a.type == GmmType::kI8) return launch_any<GmmForm::kNT, GmmI8>(a, s);
      return a.type == GmmType::kBf16 ? launch_any<GmmForm::kNT, GmmBf16>(a, s)
                                      : launch_any<GmmForm::kNT, GmmF32>(a, s);
    case GmmForm::kNN:
      return a.type == GmmType::kBf16 ? launch_any<GmmForm::kNN, GmmBf16>(a, s)
                                      : launch_any<GmmForm::kNN, GmmF32>(a, s);
    default:
      return a.type == GmmType::kBf16 ? launch_any<GmmForm::kTN, GmmBf16>(a, s)
                                      : launch_any<GmmForm::kTN, GmmF32>(a, s);
  }
}

}  // namespace moe

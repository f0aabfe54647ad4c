// Launchers of the root-mean-square norm and of its gradients.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int32_t kMaxNormCols = 32768;  // a row stays in the registers of one work-group

enum class NormOut { kF32, kBf16, kI8 };
struct NormArgs {
  const void* x;
  const void* residual;  // or null
  const void* w;         // or null: ones
  void* h;               // x + residual, where there is one
  void* out;             // y, or its codes
  float* scales;         // kI8
  int64_t rows;
  int32_t cols;
  float eps;
  bool bf16, w_bf16;     // x, residual and h; w
};
hipError_t launch_rms_norm(const NormArgs& a, NormOut out, hipStream_t s);

struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* w;    // or null: ones
  const void* dh;   // or null
  void* dx;
  float* part;      // [norm_grad_parts][norm_grad_ld] partial sums of dw, or null
  int64_t rows;
  int32_t cols;
  float eps;
  bool bf16, w_bf16;   // h, dh and dx; w
  bool dy_f32;         // dy in fp32 over bf16 rows
};
int norm_grad_parts(int64_t rows, int32_t cols);
__host__ __device__ inline int64_t norm_grad_ld(int32_t cols) { return (cols + 31) / 32 * 32; }
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);
// dw = the partial sums' sum, in their order.
hipError_t launch_norm_grad_join(const float* part, int parts, int32_t cols, void* dw, bool dw_bf16, hipStream_t s);

}  // namespace moe

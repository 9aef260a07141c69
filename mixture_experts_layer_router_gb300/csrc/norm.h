// Launchers of the RMS norm kernels (internal interface).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lmoe {

constexpr int kNormMaxWidth = 16384;  // 512 threads of four pieces of 8 elements
constexpr int kNormBlock = 128;       // channels of a scale block

// Types: 0 bf16, 1 fp32. Row strides in elements (codes: bytes).
struct NormArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;
  void* sum;             // or null
  void* y;               // or null
  uint8_t* codes;        // or null
  float* scales;
  float* rstd;           // or null
  long long ld_x, ld_residual, ld_sum, ld_y, ld_codes;
  int x_f32, residual_f32, weight_f32, y_f32;
  int d, blocks;         // blocks: scales of a row (1: one for the whole row)
  int per_block;         // 1: a scale for every kNormBlock channels
  long long T;
  float eps;
};
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s);

struct NormBackwardArgs {
  const void* dy;
  const void* s;
  const void* weight;
  const float* rstd;
  const void* d_sum;  // or null
  void* dx;
  void* dx16;         // or null: dx once more in bf16
  float* dw;          // or null
  float* partial;     // [norm_partials(T, d, sms), d]
  long long ld_dy, ld_s, ld_d_sum, ld_dx, ld_dx16;
  int dy_f32, s_f32, weight_f32;
  int d;
  long long T;
};
// Rows of partial sums of dw that a launch of this size leaves.
int norm_partials(long long T, int d, int sms);
// Two launches (one without dw).
cudaError_t launch_rms_norm_backward(const NormBackwardArgs& a, int sms, cudaStream_t s);

}  // namespace lmoe

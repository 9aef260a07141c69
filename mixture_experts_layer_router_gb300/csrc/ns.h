// Launchers of the Newton-Schulz kernels (internal interface).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "ns_iterate.cuh"

namespace lmoe {

// Update U of each matrix from gradient and momentum, and the partial sums of
// its squares: partial[b * chunks + c] over chunk c of matrix b (n elements a
// matrix), with an eps below kNsPlainEps those of the tiny entries in the batch *
// chunks floats after them. momentum null: U = G. One launch.
constexpr int kNsMaxChunks = 1024;
constexpr int kNsNormThreads = 256;
struct NsUpdate {
  const void* g;
  bool g_f32;
  float* momentum;  // [batch, n] or null
  float mu;
  bool nesterov;
};
cudaError_t launch_ns_norm(const NsUpdate& u, long long batch, long long n, int chunks,
                           long long chunk, float eps, float* partial, cudaStream_t s);

// X_0 = U / (|U|_F + eps) times `scale` in fp32 and in fp16, [batch,
// rows, ld]; the padding columns are zero. U is formed as by launch_ns_norm from
// the momentum that launch updated. Sets the batch * phases counts at `done` and
// the tile counter to zero.
cudaError_t launch_ns_init(const NsUpdate& u, long long batch, long long rows, long long cols,
                           long long ld, int chunks, const float* partial, float eps, float scale,
                           float* x32, __half* x16, int* done, int phases, int* counter,
                           cudaStream_t s);

// All steps in one launch, on tiles of a shape (NsShape).
cudaError_t launch_ns_iterate(int shape, const NsMaps& m, const NsArgs& a, int sms,
                              cudaStream_t s);

// The one-launch kernel for short sides up to kSmallSide (ns_small.cuh).
constexpr int kSmallSide = 128;
constexpr int kSmallW = 256;  // columns a CTA, at most
constexpr int kSmallCluster = 16;
constexpr int kSmallThreads = 256;
struct NsSmallArgs {
  const void* g;
  float* momentum;       // may be null
  int g_f32;
  float mu;
  int nesterov;
  int rows, cols, tall;
  int m, n;              // short and long side
  int width;             // columns of X a CTA, a multiple of 64
  int ctas;              // of a cluster
  int steps;
  float eps, scale0;
  int out_mode;
  void* out;
  float keep, move;
  unsigned* status;
  NsStep step[kNsMaxSteps];
};

// Whether the one-launch kernel takes matrices of this size (short side at most
// 128, long side at most 4096): *ctas CTAs a matrix and *width columns of its
// long side a CTA, or *ctas = 0.
cudaError_t ns_small_plan(long long batch, long long rows, long long cols, int* ctas,
                          int* width);
cudaError_t launch_ns_small(const NsSmallArgs& a, long long batch, cudaStream_t s);

}  // namespace lmoe

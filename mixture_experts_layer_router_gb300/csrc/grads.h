// Launchers of the gradient norm and clipping kernels (internal interface).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lmoe {

// A tile: what a CTA takes at a time, in 16-byte pieces; kGradPieces a thread.
constexpr int kGradThreads = 512;
constexpr int kGradPieces = 8;
constexpr int kGradTile = kGradPieces * kGradThreads;

struct GradEntry {
  const void* g;
  void* out;
  long long n;     // elements
  unsigned first;  // first tile of the tensor in the launch's sequence
  int f32;
};
static_assert(sizeof(GradEntry) == 32, "table entries");

// Tensors of one launch. Their table travels as a kernel argument (32,764 bytes at
// most), so a call has nothing to copy to the device and nothing to keep there. A
// launch of few tensors takes the short form: its arguments are 1 KB and not 32.
constexpr int kGradBatch = 1000;
constexpr int kGradFew = 30;
template <int N>
struct GradTable {
  int count;
  unsigned tiles;
  GradEntry e[N];
};

// Tiles of n elements of `size` bytes at address p: pieces begin on 16-byte
// boundaries of the address.
inline long long grad_tiles(const void* p, long long n, int size) {
  const long long pieces =
      (static_cast<long long>(reinterpret_cast<uintptr_t>(p) & 15u) + n * size + 15) / 16;
  return (pieces + kGradTile - 1) / kGradTile;
}
// CTAs of a launch over this many tiles.
int grad_ctas(unsigned tiles, int sms);

// partial[i] = sum of squares of the tiles of CTA i, i < grad_ctas(tiles, sms).
cudaError_t launch_grad_squares(const GradTable<kGradBatch>& t, double* partial, int sms,
                                cudaStream_t s);
// norm[0] = sqrt of the sum of the partials.
cudaError_t launch_grad_norm(const double* partial, int partials, float* norm, cudaStream_t s);
// out = g min(1, max_norm / (norm + eps)), with the norm formed from the partials by
// every CTA, and written to norm[0] by the first if `norm` is set.
cudaError_t launch_grad_scale(const GradTable<kGradBatch>& t, const double* partial, int partials,
                              double max_norm, double eps, float* norm, int sms, cudaStream_t s);

}  // namespace lmoe

// Global norm of many gradients, and clipping by it (declared in
// include/latentmoe.h):
//
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / (norm + eps))
//
// Two launches whatever the number of tensors (up to kGradBatch): sums of squares
// by CTA, then the scaling, in which every CTA adds up the partial sums for itself.
// The tensors' bytes form one sequence of tiles that CTAs take in turn, so a large
// tensor spreads over the GPU and small ones share it.
//
// A thread's squares are added in fp32, 64 at a time, and from tile to tile with a
// compensated fp32 sum; sums over threads and CTAs are in 64 bits. Squares that
// fp32 cannot hold (a thread's sum of a tile above 2^96 or below 2^-80) are added
// in 64 bits throughout, so the norm is right for any finite numbers. The order of
// the additions depends on the tensors' sizes and alignment alone.
//
// What bounds it: DRAM, the gradients being read twice: 330M bf16 numbers 310 us (2 x 660
// MB read, 660 written: 6.4 TB/s), of which the norm is 98 (6.7 TB/s; 174 while the pieces
// went through local memory). 2M x 3 tensors 12 us, 14 of 450,000 in all 8 us, latency.
// Pieces a thread 4 / 8 (us): 330M 321 / 310, 6M 16 / 12. 64-bit square roots and divisions
// in one thread a CTA and not in all took 6M from 29 to 16.
#include <string.h>

#include "grads.h"
#include "kernels.h"
#include "rows.cuh"

namespace lmoe {

// A tile's tensor and the pieces of it.
struct GradPart {
  const uint8_t* g;    // first byte
  uint8_t* out;
  const uint8_t* end;  // past the last byte
  long long piece;     // first piece of the tile, from the boundary at or before g
  bool f32;
};

template <int N>
__device__ __forceinline__ GradPart grad_part(const GradTable<N>& t, unsigned tile) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= tile) lo = mid; else hi = mid - 1;
  }
  GradPart p;
  p.g = static_cast<const uint8_t*>(t.e[lo].g);
  p.out = static_cast<uint8_t*>(t.e[lo].out);
  p.f32 = t.e[lo].f32 != 0;
  p.end = p.g + t.e[lo].n * (p.f32 ? 4 : 2);
  p.piece = static_cast<long long>(tile - t.e[lo].first) * kGradTile;
  return p;
}

// The piece at `at` (a 16-byte boundary): zeros outside the tensor.
__device__ __forceinline__ uint4 grad_load(const GradPart& p, const uint8_t* at) {
  if (at >= p.g && at + 16 <= p.end) return __ldcg(reinterpret_cast<const uint4*>(at));
  uint32_t w[4] = {0, 0, 0, 0};
  if (at < p.end) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t* b = at + 2 * i;
      if (b >= p.g && b < p.end)  // a half of an fp32 number is inside with the other
        w[i >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(b)) << (16 * (i & 1));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Numbers of a piece; bf16: 8, fp32: 4.
__device__ __forceinline__ float grad_squares(const uint4& v, bool f32) {
  float s = 0.0f;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (f32) {
      const float x = __uint_as_float(w[i]);
      s = fmaf(x, x, s);
    } else {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
      s = fmaf(lo, lo, s);
      s = fmaf(hi, hi, s);
    }
  }
  return s;
}
__device__ __noinline__ double grad_squares64(uint4 v, bool f32) {
  double s = 0.0;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  for (int i = 0; i < 4; ++i) {
    if (f32) {
      const double x = __uint_as_float(w[i]);
      s = fma(x, x, s);
    } else {
      const double lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
      s = fma(lo, lo, s);
      s = fma(hi, hi, s);
    }
  }
  return s;
}

// The CTA's sum, right in thread 0 alone: 64-bit additions are slow here (a few a
// clock an SM), so no thread makes one that it does not need.
__device__ __forceinline__ double block_sum64(double v, double* spare) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_down_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) spare[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kGradThreads / 32 ? spare[threadIdx.x] : 0.0;
#pragma unroll
    for (int off = kGradThreads / 64; off > 0; off >>= 1)
      v += __shfl_down_sync(0xffffffffu, v, off);
  }
  return v;
}

constexpr float kGradTop = 7.922816251426434e28f;    // 2^96: sums of squares below it
constexpr float kGradLow = 8.271806125530277e-25f;   // 2^-80

template <int N>
__global__ void __launch_bounds__(kGradThreads)
    grad_squares_kernel(const __grid_constant__ GradTable<N> t, double* partial) {
  __shared__ double spare[kGradThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  float acc = 0.0f, lost = 0.0f;  // compensated: acc - lost
  double wide = 0.0;
  for (unsigned tile = blockIdx.x; tile < t.tiles; tile += gridDim.x) {
    const GradPart p = grad_part(t, tile);
    const uint8_t* at = p.g - (reinterpret_cast<uintptr_t>(p.g) & 15u) +
                        16 * (p.piece + threadIdx.x);
    uint4 v[kGradPieces];
#pragma unroll
    for (int i = 0; i < kGradPieces; ++i) v[i] = grad_load(p, at + 16 * kGradThreads * i);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kGradPieces; ++i) s += grad_squares(v[i], p.f32);
    if (s >= kGradLow && s < kGradTop) {
      const float y = s - lost, sum = acc + y;
      lost = (sum - acc) - y;
      acc = sum;
    } else {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < kGradPieces; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
      if (any != 0) {
        for (int i = 0; i < kGradPieces; ++i) wide += grad_squares64(v[i], p.f32);
      }
    }
  }
  const double sum = block_sum64(static_cast<double>(acc) - lost + wide, spare);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the partial sums, in thread 0.
__device__ __forceinline__ double grad_norm_of(const double* partial, int partials, double* spare) {
  double v = 0.0;
  for (int i = threadIdx.x; i < partials; i += kGradThreads) v += partial[i];
  v = block_sum64(v, spare);
  return threadIdx.x == 0 ? sqrt(v) : 0.0;
}

__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const double* partial, int partials, float* norm) {
  __shared__ double spare[kGradThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const double n = grad_norm_of(partial, partials, spare);
  if (threadIdx.x == 0) norm[0] = static_cast<float>(n);
}

__device__ __forceinline__ uint4 grad_scaled(const uint4& v, bool f32, float c) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = f32 ? __float_as_uint(__uint_as_float(w[i]) * c)
               : pack_bf16x2(__uint_as_float(w[i] << 16) * c,
                             __uint_as_float(w[i] & 0xffff0000u) * c);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int N>
__global__ void __launch_bounds__(kGradThreads)
    grad_scale_kernel(const __grid_constant__ GradTable<N> t, const double* partial, int partials,
                      double max_norm, double eps, float* norm) {
  __shared__ double spare[kGradThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float factor;
  const double n = grad_norm_of(partial, partials, spare);
  if (threadIdx.x == 0) {
    if (norm != nullptr && blockIdx.x == 0) norm[0] = static_cast<float>(n);
    const double ratio = max_norm / (n + eps);
    factor = ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);  // NaN stays NaN
  }
  __syncthreads();
  const float c = factor;
  // from the last tile back: what the norm's pass read last is still in L2
  for (unsigned i = blockIdx.x; i < t.tiles; i += gridDim.x) {
    const GradPart p = grad_part(t, t.tiles - 1 - i);
    if (c == 1.0f && p.out == p.g) continue;
    const long long off = 16 * (p.piece + threadIdx.x) -
                          static_cast<long long>(reinterpret_cast<uintptr_t>(p.g) & 15u);
    const bool same = ((reinterpret_cast<uintptr_t>(p.g) ^ reinterpret_cast<uintptr_t>(p.out)) & 15u) == 0;
    uint4 v[kGradPieces];
#pragma unroll
    for (int j = 0; j < kGradPieces; ++j) v[j] = grad_load(p, p.g + off + 16 * kGradThreads * j);
#pragma unroll
    for (int j = 0; j < kGradPieces; ++j) {
      const long long o = off + 16 * kGradThreads * j;
      const uint4 x = grad_scaled(v[j], p.f32, c);
      if (same && o >= 0 && p.g + o + 16 <= p.end) {
        __stcs(reinterpret_cast<uint4*>(p.out + o), x);
        continue;
      }
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (o + 2 * q >= 0 && p.g + o + 2 * q < p.end)
          *reinterpret_cast<uint16_t*>(p.out + o + 2 * q) =
              static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
    }
  }
}

int grad_ctas(unsigned tiles, int sms) {
  const unsigned most = 2u * static_cast<unsigned>(sms);
  return static_cast<int>(tiles < 1 ? 1 : tiles < most ? tiles : most);
}

namespace {

GradTable<kGradFew> few(const GradTable<kGradBatch>& t) {
  GradTable<kGradFew> f;
  memset(&f, 0, sizeof(f));
  f.count = t.count;
  f.tiles = t.tiles;
  memcpy(f.e, t.e, sizeof(GradEntry) * static_cast<size_t>(t.count));
  return f;
}

}  // namespace

cudaError_t launch_grad_squares(const GradTable<kGradBatch>& t, double* partial, int sms,
                                cudaStream_t s) {
  const PdlScope pdl(true);
  const dim3 grid(static_cast<unsigned>(grad_ctas(t.tiles, sms)));
  if (t.count <= kGradFew)
    return launch_kernel(grad_squares_kernel<kGradFew>, grid, dim3(kGradThreads), 0, s, 1, false,
                         few(t), partial);
  return launch_kernel(grad_squares_kernel<kGradBatch>, grid, dim3(kGradThreads), 0, s, 1, false, t,
                       partial);
}

cudaError_t launch_grad_norm(const double* partial, int partials, float* norm, cudaStream_t s) {
  const PdlScope pdl(true);
  return launch_kernel(grad_norm_kernel, dim3(1), dim3(kGradThreads), 0, s, 1, false, partial,
                       partials, norm);
}

cudaError_t launch_grad_scale(const GradTable<kGradBatch>& t, const double* partial, int partials,
                              double max_norm, double eps, float* norm, int sms, cudaStream_t s) {
  const PdlScope pdl(true);
  const dim3 grid(static_cast<unsigned>(grad_ctas(t.tiles, sms)));
  if (t.count <= kGradFew)
    return launch_kernel(grad_scale_kernel<kGradFew>, grid, dim3(kGradThreads), 0, s, 1, false,
                         few(t), partial, partials, max_norm, eps, norm);
  return launch_kernel(grad_scale_kernel<kGradBatch>, grid, dim3(kGradThreads), 0, s, 1, false, t,
                       partial, partials, max_norm, eps, norm);
}

}  // namespace lmoe

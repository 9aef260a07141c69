// Elementwise head of the Newton-Schulz orthogonalisation: the momentum
// update, the Frobenius norm and the first iterate.
//
//   m <- mu m + g;  U = g + mu m (Nesterov) or m (or g without momentum)
//   X_0 = U / (|U|_F + eps)
//
// Two passes, because the norm has to be known before an element can be
// scaled: the first reads g (and reads and writes m) and leaves one partial
// sum of squares per block, the second adds the partials in a fixed order in
// every block (the result does not depend on scheduling), forms U again and
// writes X_0 in fp32 and fp16. Both are bound by memory traffic: 8 x 1024 x 2048
// with bf16 g and fp32 m 22 us for 168 MB (norm: g and m read, m written; DRAM 64 %
// busy) and 32 to 36 us for 201 MB (init: 61 to 55 %).
// U is formed with separately rounded products and sums, so that the momentum
// equals m.mul_(mu).add_(g) bit for bit. The sum of squares is held in fp32 (NsSquares):
// a matrix whose norm reaches 1.8e19 has an infinite sum, and X_0 = 0.
#include "kernels.h"
#include "ns.h"

namespace lmoe {

// V consecutive elements of the gradient as floats (V = 8: 16-byte loads, the
// index a multiple of 8).
template <bool F32, int V>
__device__ __forceinline__ void load_g(const void* g, long long i, float (&v)[V]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(g) + i;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 x = reinterpret_cast<const float4*>(p)[q];
        v[4 * q] = x.x;
        v[4 * q + 1] = x.y;
        v[4 * q + 2] = x.z;
        v[4 * q + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = p[j];
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(g) + i;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const uint2 x = reinterpret_cast<const uint2*>(p)[q];
        v[4 * q] = __uint_as_float(x.x << 16);
        v[4 * q + 1] = __uint_as_float(x.x & 0xffff0000u);
        v[4 * q + 2] = __uint_as_float(x.y << 16);
        v[4 * q + 3] = __uint_as_float(x.y & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = __bfloat162float(p[j]);
    }
  }
}

__device__ __forceinline__ float ns_u(float g, float m, float mu, bool nesterov) {
  return nesterov ? __fadd_rn(g, __fmul_rn(mu, m)) : m;
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float ws[kNsNormThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) ws[warp] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kNsNormThreads / 32; ++w) t += ws[w];
  return t;
}

template <bool F32, int V>
__global__ void __launch_bounds__(kNsNormThreads)
    ns_norm_kernel(const void* g, float* mom, float mu, int nesterov,
                   long long n, long long chunk, float eps, float* partial) {
  pdl_wait();
  pdl_launch_dependents();
  const long long base = static_cast<long long>(blockIdx.y) * n;
  const long long lo = blockIdx.x * chunk;
  const long long hi = lo + chunk < n ? lo + chunk : n;
  const bool apart = eps < kNsPlainEps;
  NsSquares sq;
  for (long long i = lo + static_cast<long long>(threadIdx.x) * V; i < hi;
       i += static_cast<long long>(kNsNormThreads) * V) {
    float v[V];
    load_g<F32, V>(g, base + i, v);
    if (mom != nullptr) {
      float m[V];
      load_g<true, V>(mom, base + i, m);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        m[j] = __fadd_rn(__fmul_rn(mu, m[j]), v[j]);
        v[j] = ns_u(v[j], m[j], mu, nesterov != 0);
      }
      float* p = mom + base + i;
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q)
          reinterpret_cast<float4*>(p)[q] =
              make_float4(m[4 * q], m[4 * q + 1], m[4 * q + 2], m[4 * q + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = m[j];
      }
    }
    sq.add(v, apart);
  }
  const float t = block_sum(sq.sum);
  const long long at = static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x;
  if (threadIdx.x == 0) partial[at] = t;
  if (apart) {
    __syncthreads();
    const float tiny = block_sum(sq.tiny);
    if (threadIdx.x == 0) partial[static_cast<long long>(gridDim.y) * gridDim.x + at] = tiny;
  }
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(kNsNormThreads)
    ns_init_kernel(const void* g, const float* mom, float mu,
                   int nesterov, long long rows, long long cols, long long ld, int chunks,
                   const float* partial, float eps, float scale, float* x32, __half* x16,
                   int* done, int phases, int* counter) {
  pdl_wait();
  pdl_launch_dependents();
  const long long b = blockIdx.y;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < phases; i += kNsNormThreads) done[b * phases + i] = 0;
    if (b == 0 && threadIdx.x == 0) *counter = 0;
  }
  NsSquares sq;
  for (int c = threadIdx.x; c < chunks; c += kNsNormThreads) sq.sum += partial[b * chunks + c];
  sq.sum = block_sum(sq.sum);
  if (eps < kNsPlainEps) {
    const float* apart = partial + static_cast<long long>(gridDim.y) * chunks + b * chunks;
    for (int c = threadIdx.x; c < chunks; c += kNsNormThreads) sq.tiny += apart[c];
    __syncthreads();
    sq.tiny = block_sum(sq.tiny);
  }
  const float inv = 1.0f / (sq.norm() + eps);
  const long long base = b * rows * cols;
  const long long per_row = ld / 4;
  const long long total = rows * per_row;
  for (long long i = static_cast<long long>(blockIdx.x) * kNsNormThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kNsNormThreads) {
    const long long r = i / per_row;
    const long long c = (i - r * per_row) * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const long long at = base + r * cols + c;
    if constexpr (VEC) {
      if (c < cols) {
        load_g<F32, 4>(g, at, v);
        if (mom != nullptr) {
          float m[4];
          load_g<true, 4>(mom, at, m);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = ns_u(v[j], m[j], mu, nesterov != 0);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + j < cols) {
          float one[1];
          load_g<F32, 1>(g, at + j, one);
          v[j] = mom != nullptr ? ns_u(one[0], mom[at + j], mu, nesterov != 0) : one[0];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= inv;
    const long long to = (b * rows + r) * ld + c;
    const float4 x = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
    *reinterpret_cast<float4*>(x32 + to) = x;
    const __half2 h01 = __floats2half2_rn(x.x, x.y), h23 = __floats2half2_rn(x.z, x.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&h01);
    w.y = *reinterpret_cast<const uint32_t*>(&h23);
    *reinterpret_cast<uint2*>(x16 + to) = w;
  }
}

cudaError_t launch_ns_norm(const NsUpdate& u, long long batch, long long n, int chunks,
                           long long chunk, float eps, float* partial, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(batch));
  const dim3 block(kNsNormThreads);
  const int nes = u.nesterov ? 1 : 0;
  // 16-byte accesses need every matrix of the stack to start on 8 elements
  const bool vec = n % 8 == 0;
  if (u.g_f32)
    return vec ? launch_kernel(ns_norm_kernel<true, 8>, grid, block, 0, s, 1, false, u.g,
                               u.momentum, u.mu, nes, n, chunk, eps, partial)
               : launch_kernel(ns_norm_kernel<true, 1>, grid, block, 0, s, 1, false, u.g,
                               u.momentum, u.mu, nes, n, chunk, eps, partial);
  return vec ? launch_kernel(ns_norm_kernel<false, 8>, grid, block, 0, s, 1, false, u.g,
                             u.momentum, u.mu, nes, n, chunk, eps, partial)
             : launch_kernel(ns_norm_kernel<false, 1>, grid, block, 0, s, 1, false, u.g,
                             u.momentum, u.mu, nes, n, chunk, eps, partial);
}

cudaError_t launch_ns_init(const NsUpdate& u, long long batch, long long rows, long long cols,
                           long long ld, int chunks, const float* partial, float eps, float scale,
                           float* x32, __half* x16, int* done, int phases, int* counter,
                           cudaStream_t s) {
  long long blocks = (rows * (ld / 4) + 4 * kNsNormThreads - 1) / (4 * kNsNormThreads);
  if (blocks > 4096) blocks = 4096;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(batch));
  const dim3 block(kNsNormThreads);
  const int nes = u.nesterov ? 1 : 0;
  const float* mom = u.momentum;
  const bool vec = cols % 4 == 0;
  if (u.g_f32)
    return vec ? launch_kernel(ns_init_kernel<true, true>, grid, block, 0, s, 1, false, u.g, mom,
                               u.mu, nes, rows, cols, ld, chunks, partial, eps, scale, x32, x16,
                               done, phases, counter)
               : launch_kernel(ns_init_kernel<true, false>, grid, block, 0, s, 1, false, u.g, mom,
                               u.mu, nes, rows, cols, ld, chunks, partial, eps, scale, x32, x16,
                               done, phases, counter);
  return vec ? launch_kernel(ns_init_kernel<false, true>, grid, block, 0, s, 1, false, u.g, mom,
                             u.mu, nes, rows, cols, ld, chunks, partial, eps, scale, x32, x16,
                               done, phases, counter)
             : launch_kernel(ns_init_kernel<false, false>, grid, block, 0, s, 1, false, u.g, mom,
                             u.mu, nes, rows, cols, ld, chunks, partial, eps, scale, x32, x16,
                               done, phases, counter);
}

}  // namespace lmoe

// Rows of bf16 or fp32 numbers spread over the threads of a row group: 8
// elements of every 256-element chunk a thread, in registers as fp32.
//
// A row group is a warp (rows of a few hundred elements: no barrier) or a whole
// CTA. Thread i of the group holds VPT pieces of 8 elements; piece j belongs to
// chunk (j * threads + i) / 32. Two layouts of a chunk's 256 elements:
//   VEC   element 8 * lane + k: one 16-byte access for bf16, two for fp32
//   else  element 32 * k + lane: single elements, 32 neighbours a warp access;
//         for rows that do not begin on a 16-byte boundary or whose length is no
//         multiple of 8
// In both, elements [0, 128) and [128, 256) of a chunk lie in registers of one
// warp: lanes 0..15 and 16..31, or k < 4 and k >= 4.
#pragma once

#include "ptx.cuh"

namespace lmoe {

template <typename T>
struct RowType;
template <>
struct RowType<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct RowType<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

__device__ __forceinline__ void bf16x8_to_float(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 float_to_bf16x8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Elements of chunk `chunk` that this lane holds, as they come from memory; those at
// or past d are zero. load() only starts the accesses.
template <bool VEC, typename T>
struct RowPiece {
  float x[8];
  __device__ __forceinline__ void load(const T* row, int chunk, int lane, int d) {
    const int e = chunk * 256 + lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = e + 32 * k < d ? RowType<T>::get(row[e + 32 * k]) : 0.0f;
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = x[k];
  }
};
template <>
struct RowPiece<true, __nv_bfloat16> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int chunk, int lane, int d) {
    const int e = chunk * 256 + lane * 8;
    x = e < d ? *reinterpret_cast<const uint4*>(row + e) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* v) const { bf16x8_to_float(x, v); }
};
template <>
struct RowPiece<true, float> {
  float4 x[2];
  __device__ __forceinline__ void load(const float* row, int chunk, int lane, int d) {
    const int e = chunk * 256 + lane * 8;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    x[0] = e < d ? reinterpret_cast<const float4*>(row + e)[0] : zero;
    x[1] = e < d ? reinterpret_cast<const float4*>(row + e)[1] : zero;
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = x[0].x; v[1] = x[0].y; v[2] = x[0].z; v[3] = x[0].w;
    v[4] = x[1].x; v[5] = x[1].y; v[6] = x[1].z; v[7] = x[1].w;
  }
};
template <bool VEC, typename T>
__device__ __forceinline__ void row_load(const T* row, int chunk, int lane, int d, float* x) {
  RowPiece<VEC, T> p;
  p.load(row, chunk, lane, d);
  p.get(x);
}

template <bool VEC, typename T>
__device__ __forceinline__ void row_store(T* row, int chunk, int lane, int d, const float* x) {
  if constexpr (VEC) {
    const int e = chunk * 256 + lane * 8;
    if (e < d) {
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(row + e) = float_to_bf16x8(x);
      } else {
        reinterpret_cast<float4*>(row + e)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(row + e)[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  } else {
    const int e = chunk * 256 + lane;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (e + 32 * k < d) row[e + 32 * k] = RowType<T>::put(x[k]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum (or maximum) of v over a row group: blockDim.x threads, one warp or the
// whole CTA (`spare`: 32 floats of shared memory that no thread still reads or
// writes; the call ends with every thread past its writes to it, not its reads).
// The order of the additions depends on blockDim.x alone.
__device__ __forceinline__ float group_sum(float v, float* spare) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) spare[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? spare[lane] : 0.0f);
}
__device__ __forceinline__ float group_max(float v, float* spare) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) spare[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  v = lane < warps ? spare[lane] : 0.0f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

}  // namespace lmoe

// RMS norm with the residual's addition (declared in include/latentmoe.h):
//
//   s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//
// and, for an 8-bit product behind it, y as E4M3 codes with a scale for each
// token or for each 128 channels of a token.
//
// One pass: a row is read once into the registers of its row group (rows.cuh),
// summed, reduced over the group, and everything that leaves is written from
// there. y and rstd come from the sum in fp32, before its rounding to the
// stream's type: the norm is as exact as its inputs, and only `sum` holds the
// rounding.
//
// What bounds it: DRAM, with enough CTAs an SM that some load while others reduce or
// store. 16384 x 6656 in bf16 with a bf16 stream 126 us (6.9 TB/s); to E4M3 by blocks
// 135 us (5.6 TB/s: the issue slots count too, 67 % of them); 8192 x 8192 with an fp32
// stream to E4M3 110 us (6.7 TB/s); 4096 x 2048 12 us; one token of 8704 3.6 us.
#include <math.h>

#include "fp8.cuh"
#include "kernels.h"
#include "norm.h"
#include "rows.cuh"

namespace lmoe {

// 1 / sqrt(mean + eps) of squares that fp32 cannot hold: s scaled by 2^-64.
constexpr float kNormDown = 5.421010862427522e-20f;   // 2^-64
constexpr float kNormDown2 = 2.938735877055719e-39f;  // 2^-128

// The scale of values whose largest magnitude is `top`: top / 448, 1 for zeros
// (as latentmoe_quantize_e4m3), and at least 2^-126, whose reciprocal is still
// an fp32 number.
__device__ __forceinline__ float norm_scale(float top) {
  return top > 0.0f ? fmaxf(top / kE4M3Max, 1.1754943508222875e-38f) : 1.0f;
}

// Pieces a thread, and CTAs an SM that the registers are cut for. 16384 x 6656 to E4M3
// by blocks / to bf16 (us): one piece, 832 threads, 2 CTAs 162 / 149; two pieces, 416
// threads, 2 / 3 / 4 CTAs 165 / 135 / 145 and 146 / 126 / 143; four pieces 192 / 150.
constexpr int norm_threads(int vpt) { return vpt == 1 ? 128 : 512; }
constexpr int norm_ctas(int vpt) { return vpt == 1 ? 12 : vpt == 2 ? 3 : 2; }

template <typename XT, typename RT, bool RES, bool VEC, int VPT>
__global__ void __launch_bounds__(norm_threads(VPT), norm_ctas(VPT)) rms_norm_kernel(const NormArgs a) {
  __shared__ float spare[3][32];
  pdl_wait();
  pdl_launch_dependents();
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.T) return;  // a warp's row; rows of a whole CTA are never past the end
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  const int d = a.d;
  float x[VPT][8];
  {
    const XT* row = static_cast<const XT*>(a.x) + t * a.ld_x;
#pragma unroll
    for (int j = 0; j < VPT; ++j) row_load<VEC>(row, j * warps + warp, lane, d, x[j]);
  }
  if constexpr (RES) {
    const RT* row = static_cast<const RT*>(a.residual) + t * a.ld_residual;
    float r[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) row_load<VEC>(row, j * warps + warp, lane, d, r[j]);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] += r[j][k];
  }
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float part = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) part = fmaf(x[j][k], x[j][k], part);
    ss += part;
  }
  if (RES && a.sum != nullptr) {
    RT* row = static_cast<RT*>(a.sum) + t * a.ld_sum;
#pragma unroll
    for (int j = 0; j < VPT; ++j) row_store<VEC>(row, j * warps + warp, lane, d, x[j]);
  }
  ss = group_sum(ss, spare[0]);
  float rstd = 1.0f / sqrtf(ss / static_cast<float>(d) + a.eps);
  if (isinf(ss)) {
    // numbers above 1.8e19: the same with every s times 2^-64
    float low = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = x[j][k] * kNormDown;
        low = fmaf(v, v, low);
      }
    low = group_sum(low, spare[1]);
    rstd = kNormDown / sqrtf(low / static_cast<float>(d) + a.eps * kNormDown2);
  }
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[t] = rstd;
  if (a.weight_f32) {
    const float* w = static_cast<const float*>(a.weight);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float v[8];
      row_load<VEC>(w, j * warps + warp, lane, d, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] = x[j][k] * rstd * v[k];
    }
  } else {
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(a.weight);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float v[8];
      row_load<VEC>(w, j * warps + warp, lane, d, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] = x[j][k] * rstd * v[k];
    }
  }
  if (a.y != nullptr) {
    if (a.y_f32) {
      float* row = static_cast<float*>(a.y) + t * a.ld_y;
#pragma unroll
      for (int j = 0; j < VPT; ++j) row_store<VEC>(row, j * warps + warp, lane, d, x[j]);
    } else {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(a.y) + t * a.ld_y;
#pragma unroll
      for (int j = 0; j < VPT; ++j) row_store<VEC>(row, j * warps + warp, lane, d, x[j]);
    }
  }
  if (a.codes == nullptr) return;
  // elements past d are 0 * rstd * 0 (NaN where rstd is infinite or NaN; fmaxf
  // passes over a NaN), and are not stored
  float token_scale = 1.0f;
  if (!a.per_block) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[j][k]));
    token_scale = norm_scale(group_max(top, spare[2]));
    if (threadIdx.x == 0) a.scales[t] = token_scale;
  }
  uint8_t* row = a.codes + t * a.ld_codes;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int chunk = j * warps + warp;
    float inv[2];
    inv[0] = inv[1] = inv_scale(token_scale);
    if (a.per_block) {
      // [0]: this lane's block (VEC), or that of k < 4; [1]: of k >= 4
      float top[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        top[VEC ? 0 : k >> 2] = fmaxf(top[VEC ? 0 : k >> 2], fabsf(x[j][k]));
#pragma unroll
      for (int off = VEC ? 8 : 16; off > 0; off >>= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], off));
        if (!VEC) top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], off));
      }
      float scale[2] = {norm_scale(top[0]), norm_scale(top[1])};
      inv[0] = inv_scale(scale[0]);
      inv[1] = VEC ? inv[0] : inv_scale(scale[1]);
      float* to = a.scales + t * a.blocks;
      if (VEC) {
        const int b = 2 * chunk + (lane >> 4);
        if ((lane & 15) == 0 && b < a.blocks) to[b] = scale[0];
      } else if (lane < 2 && 2 * chunk + lane < a.blocks) {
        to[2 * chunk + lane] = lane == 0 ? scale[0] : scale[1];
      }
    }
    if constexpr (VEC) {
      const int e = chunk * 256 + lane * 8;
      if (e < d) {
        const uint32_t lo = quant4_e4m3(x[j][0], x[j][1], x[j][2], x[j][3], inv[0]);
        const uint32_t hi = quant4_e4m3(x[j][4], x[j][5], x[j][6], x[j][7], inv[0]);
        *reinterpret_cast<uint2*>(row + e) = make_uint2(lo, hi);
      }
    } else {
      const int e = chunk * 256 + lane;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (e + 32 * k < d)
          row[e + 32 * k] = static_cast<uint8_t>(quant2_e4m3(x[j][k], 0.0f, inv[k >> 2]));
    }
  }
}

namespace {

bool whole(const void* p, long long ld, int size, int unit) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % unit) == 0 && ld * size % unit == 0);
}

template <typename XT, typename RT, bool RES, bool VEC>
cudaError_t launch_vpt(const NormArgs& a, cudaStream_t s) {
  const PdlScope pdl(true);
  const int chunks = (a.d + 255) / 256;
  // one piece up to 1024 channels (65536 x 256: 22 us, two pieces 28), four where two do
  // not fit 512 threads
  const int vpt = chunks <= 4 ? 1 : chunks <= 32 ? 2 : 4;
  const int warps = (chunks + vpt - 1) / vpt;
  const int rows = warps == 1 ? 4 : 1;
  const dim3 block(32 * warps, rows, 1);
  const long long grid = (a.T + rows - 1) / rows;
  const auto kern = vpt == 1   ? rms_norm_kernel<XT, RT, RES, VEC, 1>
                    : vpt == 2 ? rms_norm_kernel<XT, RT, RES, VEC, 2>
                               : rms_norm_kernel<XT, RT, RES, VEC, 4>;
  return launch_kernel(kern, dim3(static_cast<unsigned>(grid)), block, 0, s, 1, false, a);
}

template <typename XT, typename RT, bool RES>
cudaError_t launch_layout(const NormArgs& a, cudaStream_t s) {
  const bool vec = a.d % 8 == 0 && whole(a.x, a.ld_x, sizeof(XT), 16) &&
                   whole(a.residual, a.ld_residual, sizeof(RT), 16) &&
                   whole(a.sum, a.ld_sum, sizeof(RT), 16) &&
                   whole(a.weight, 0, 1, 16) && whole(a.y, a.ld_y, a.y_f32 ? 4 : 2, 16) &&
                   whole(a.codes, a.ld_codes, 1, 8);
  return vec ? launch_vpt<XT, RT, RES, true>(a, s) : launch_vpt<XT, RT, RES, false>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  if (a.residual == nullptr)
    return a.x_f32 ? launch_layout<float, float, false>(a, s)
                   : launch_layout<__nv_bfloat16, __nv_bfloat16, false>(a, s);
  if (a.x_f32) return launch_layout<float, float, true>(a, s);
  return a.residual_f32 ? launch_layout<__nv_bfloat16, float, true>(a, s)
                        : launch_layout<__nv_bfloat16, __nv_bfloat16, true>(a, s);
}

}  // namespace lmoe

// Gradient of the RMS norm (declared in include/latentmoe.h): with a = dy w and
// n = s rstd,
//
//   dx = d_sum + rstd (a - n mean(a n)),   dw = sum over the tokens of dy n
//
// One pass over dy, s and d_sum: row groups (rows.cuh) take rows t, t + groups,
// ...; a row sits in registers between its one reduction and dx, and each thread
// adds up dw for its own channels over all of its group's rows. A second launch
// adds the groups' partial sums in the order of the groups: results are bitwise
// reproducible. Bound by DRAM.
#include "kernels.h"
#include "norm.h"
#include "rows.cuh"

namespace lmoe {

template <typename YT, typename ST, bool DS, bool VEC, int VPT>
__global__ void __launch_bounds__(512) rms_norm_backward_kernel(const NormBackwardArgs a) {
  __shared__ float spare[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const long long groups = static_cast<long long>(gridDim.x) * blockDim.y;
  const long long group = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  const int d = a.d;
  float dw[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = 0.0f;
  int turn = 0;
  for (long long t = group; t < a.T; t += groups) {
    const YT* dy_row = static_cast<const YT*>(a.dy) + t * a.ld_dy;
    const ST* s_row = static_cast<const ST*>(a.s) + t * a.ld_s;
    float g[VPT][8], n[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) row_load<VEC>(dy_row, j * warps + warp, lane, d, g[j]);
#pragma unroll
    for (int j = 0; j < VPT; ++j) row_load<VEC>(s_row, j * warps + warp, lane, d, n[j]);
    const float rstd = a.rstd[t];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float w[8];
      if (a.weight_f32)
        row_load<VEC>(static_cast<const float*>(a.weight), j * warps + warp, lane, d, w);
      else
        row_load<VEC>(static_cast<const __nv_bfloat16*>(a.weight), j * warps + warp, lane, d, w);
      float part = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        n[j][k] *= rstd;
        dw[j][k] = fmaf(g[j][k], n[j][k], dw[j][k]);
        g[j][k] *= w[k];
        part = fmaf(g[j][k], n[j][k], part);
      }
      dot += part;
    }
    // two barriers' buffers in turn: a row's sums are read before the next row's
    // barrier, so the row after that may write them again
    const float mean = group_sum(dot, spare[turn]) / static_cast<float>(d);
    turn ^= 1;
    ST* to = static_cast<ST*>(a.dx) + t * a.ld_dx;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int chunk = j * warps + warp;
      float o[8];
      if constexpr (DS) {
        row_load<VEC>(static_cast<const ST*>(a.d_sum) + t * a.ld_d_sum, chunk, lane, d, o);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] += rstd * (g[j][k] - n[j][k] * mean);
      row_store<VEC>(to, chunk, lane, d, o);
      if (sizeof(ST) == 4 && a.dx16 != nullptr)
        row_store<VEC>(static_cast<__nv_bfloat16*>(a.dx16) + t * a.ld_dx16, chunk, lane, d, o);
    }
  }
  if (a.dw != nullptr) {
    float* to = a.partial + group * d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      // [groups, d] of the library's own: whole vectors where d allows
      if (d % 8 == 0)
        row_store<VEC>(to, j * warps + warp, lane, d, dw[j]);
      else
        row_store<false>(to, j * warps + warp, lane, d, dw[j]);
    }
  }
}

constexpr int kDwRows = 16;

// dw[c] = sum over the groups of partial[group][c]: 32 columns a CTA, kDwRows
// threads a column.
__global__ void __launch_bounds__(32 * kDwRows)
    rms_norm_dw_kernel(const float* partial, int groups, int d, float* dw) {
  __shared__ float part[kDwRows][33];
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float sum = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int g = threadIdx.y; g < groups; g += kDwRows)
      sum += partial[static_cast<long long>(g) * d + c];
  }
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && c < d) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kDwRows; ++i) sum += part[i][threadIdx.x];
    dw[c] = sum;
  }
}

namespace {

struct Shape {
  int vpt, warps, rows, ctas;
};

Shape shape_of(long long T, int d, int sms) {
  Shape p;
  const int chunks = (d + 255) / 256;
  p.vpt = chunks <= 4 ? 1 : chunks <= 16 ? 2 : 4;
  p.warps = (chunks + p.vpt - 1) / p.vpt;
  p.rows = p.warps == 1 ? 8 : 1;
  // about 32 warps an SM
  int per_sm = 32 / (p.warps * p.rows);
  if (per_sm < 1) per_sm = 1;
  const long long want = (T + p.rows - 1) / p.rows;
  p.ctas = static_cast<int>(want < static_cast<long long>(per_sm) * sms ? want : per_sm * sms);
  return p;
}

bool whole(const void* p, long long ld, int size, int unit) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % unit) == 0 && ld * size % unit == 0);
}

template <typename YT, typename ST, bool DS, bool VEC>
cudaError_t launch_vpt(const NormBackwardArgs& a, const Shape& p, cudaStream_t s) {
  const auto kern = p.vpt == 1   ? rms_norm_backward_kernel<YT, ST, DS, VEC, 1>
                    : p.vpt == 2 ? rms_norm_backward_kernel<YT, ST, DS, VEC, 2>
                                 : rms_norm_backward_kernel<YT, ST, DS, VEC, 4>;
  return launch_kernel(kern, dim3(static_cast<unsigned>(p.ctas)), dim3(32 * p.warps, p.rows), 0, s,
                       1, false, a);
}

template <typename YT, typename ST, bool DS>
cudaError_t launch_layout(const NormBackwardArgs& a, const Shape& p, cudaStream_t s) {
  const bool vec = a.d % 8 == 0 && whole(a.dy, a.ld_dy, sizeof(YT), 16) &&
                   whole(a.s, a.ld_s, sizeof(ST), 16) && whole(a.weight, 0, 1, 16) &&
                   whole(a.d_sum, a.ld_d_sum, sizeof(ST), 16) &&
                   whole(a.dx, a.ld_dx, sizeof(ST), 16) && whole(a.dx16, a.ld_dx16, 2, 16) &&
                   whole(a.partial, 0, 1, 16);
  return vec ? launch_vpt<YT, ST, DS, true>(a, p, s) : launch_vpt<YT, ST, DS, false>(a, p, s);
}

template <typename YT, typename ST>
cudaError_t launch_sum(const NormBackwardArgs& a, const Shape& p, cudaStream_t s) {
  return a.d_sum != nullptr ? launch_layout<YT, ST, true>(a, p, s)
                            : launch_layout<YT, ST, false>(a, p, s);
}

}  // namespace

int norm_partials(long long T, int d, int sms) {
  const Shape p = shape_of(T, d, sms);
  return p.ctas * p.rows;
}

cudaError_t launch_rms_norm_backward(const NormBackwardArgs& a, int sms, cudaStream_t s) {
  const PdlScope pdl(true);
  const Shape p = shape_of(a.T, a.d, sms);
  cudaError_t e;
  if (a.dy_f32)
    e = a.s_f32 ? launch_sum<float, float>(a, p, s) : launch_sum<float, __nv_bfloat16>(a, p, s);
  else
    e = a.s_f32 ? launch_sum<__nv_bfloat16, float>(a, p, s)
                : launch_sum<__nv_bfloat16, __nv_bfloat16>(a, p, s);
  if (e != cudaSuccess || a.dw == nullptr) return e;
  return launch_kernel(rms_norm_dw_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32)),
                       dim3(32, kDwRows), 0, s, 1, false, static_cast<const float*>(a.partial),
                       p.ctas * p.rows, a.d, a.dw);
}

}  // namespace lmoe

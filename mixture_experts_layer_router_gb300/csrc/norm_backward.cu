// Gradient of the RMS norm (declared in include/latentmoe.h): with a = dy w and
// n = s rstd,
//
//   dx = d_sum + rstd (a - n mean(a n)),   dw = sum over the tokens of dy n
//
// One pass over dy, s and d_sum: row groups (rows.cuh) take rows t, t + groups,
// ...; a row sits in registers between its one reduction and dx, and each thread
// adds up dw for its own channels over all of its group's rows. A second launch
// adds the CTAs' partial sums in the order of the CTAs: results are bitwise
// reproducible.
//
// What bounds it: an iteration's latency (loads, one barrier, stores) with the rows that
// the registers let an SM have on their way beside dw. 8192 x 6656, fp32 stream 161 us
// (4.7 TB/s), 16384 x 6656, bf16 161 us (5.4), 16384 x 1024, fp32 44 us (5.3). Also tried:
// rows ahead by asynchronous copies to shared memory (173 / 195), two pieces a thread in two
// CTAs (154 / 220).
#include "kernels.h"
#include "norm.h"
#include "rows.cuh"

namespace lmoe {

// How rows overlap. Narrow and fp32 streams: one piece (8 elements) a thread, about 32 warps
// an SM, and of a bf16 stream two rows at a time (one barrier for both; 65536 x 256 28 us
// either way). Wide bf16 streams: two pieces a thread, 16 warps an SM, and the next row on
// its way in registers while this one is reduced: 16384 x 6656 182 -> 161 us, 4096 x 2048 20 ->
// 17.8 (with the weight in registers too: 245 and 22 without). An fp32 stream's next row does not fit beside dw (8192 x 6656 163 -> 189 us), nor do two
// rows of it (16384 x 1024 44 -> 48).
constexpr int norm_rows(int s_size, int vpt) { return vpt > 1 || s_size > 2 ? 1 : 2; }
constexpr bool norm_ahead(int vpt) { return vpt == 2; }

// R rows of a group, groups rows apart, as they lie in memory: half the registers of their
// fp32 values. A row past the last is zeros.
template <typename YT, typename ST, bool DS, bool VEC, int VPT, int R>
struct NormRows {
  RowPiece<VEC, YT> dy[R][VPT];
  RowPiece<VEC, ST> s[R][VPT], ds[R][VPT];
  float rstd[R];
  __device__ __forceinline__ void load(const NormBackwardArgs& a, long long t0, long long groups,
                                       int warp, int warps, int lane) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long t = t0 + r * groups;
      const int width = t < a.T ? a.d : 0;
      rstd[r] = t < a.T ? a.rstd[t] : 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int chunk = j * warps + warp;
        dy[r][j].load(static_cast<const YT*>(a.dy) + t * a.ld_dy, chunk, lane, width);
        s[r][j].load(static_cast<const ST*>(a.s) + t * a.ld_s, chunk, lane, width);
        if (DS)
          ds[r][j].load(static_cast<const ST*>(a.d_sum) + t * a.ld_d_sum, chunk, lane, width);
      }
    }
  }
};

template <typename YT, typename ST, bool DS, bool VEC, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) rms_norm_backward_kernel(const NormBackwardArgs a) {
  constexpr int R = norm_rows(sizeof(ST), VPT);
  __shared__ float spare[2][R][32];
  __shared__ float join[8][256];  // dw of the warps of a CTA that has a row a warp
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
  // 8 elements of the weight: in registers beside rows that are on their way, else in L1
  // after the first row
  auto load_weight = [&](int j, float* w) {
    if (a.weight_f32)
      row_load<VEC>(static_cast<const float*>(a.weight), j * warps + warp, lane, d, w);
    else
      row_load<VEC>(static_cast<const __nv_bfloat16*>(a.weight), j * warps + warp, lane, d, w);
  };
  float held[VPT][8];
  if (norm_ahead(VPT)) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) load_weight(j, held[j]);
  }
  auto weight = [&](int j, float* w) {
    if (norm_ahead(VPT)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = held[j][k];
    } else {
      load_weight(j, w);
    }
  };
  int turn = 0;
  NormRows<YT, ST, DS, VEC, VPT, R> next;
  if (norm_ahead(VPT)) next.load(a, group, groups, warp, warps, lane);
  for (long long t0 = group; t0 < a.T; t0 += R * groups) {
    if (!norm_ahead(VPT)) next.load(a, t0, groups, warp, warps, lane);
    const NormRows<YT, ST, DS, VEC, VPT, R> now = next;
    if (norm_ahead(VPT)) next.load(a, t0 + groups, groups, warp, warps, lane);
    float dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float w[8];
      weight(j, w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float g[8], n[8];
        now.dy[r][j].get(g);
        now.s[r][j].get(n);
        float part = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          n[k] *= now.rstd[r];
          dw[j][k] = fmaf(g[k], n[k], dw[j][k]);
          part = fmaf(g[k] * w[k], n[k], part);
        }
        dot[r] += part;
      }
    }
    // sums over the group; two buffers in turn: an iteration's sums are read before the
    // next one's barrier, so the one after that may write them again
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = warp_sum(dot[r]);
    if (warps > 1) {
      if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) spare[turn][r][warp] = dot[r];
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) dot[r] = warp_sum(lane < warps ? spare[turn][r][lane] : 0.0f);
      turn ^= 1;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int chunk = j * warps + warp;
      float w[8];
      weight(j, w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long t = t0 + r * groups;
        if (t >= a.T) break;
        const float back = now.rstd[r] * (dot[r] / static_cast<float>(d));
        float g[8], n[8], o[8];
        now.dy[r][j].get(g);
        now.s[r][j].get(n);
        if constexpr (DS) {
          now.ds[r][j].get(o);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += now.rstd[r] * (g[k] * w[k] - n[k] * back);
        row_store<VEC>(static_cast<ST*>(a.dx) + t * a.ld_dx, chunk, lane, d, o);
        if (sizeof(ST) == 4 && a.dx16 != nullptr)
          row_store<VEC>(static_cast<__nv_bfloat16*>(a.dx16) + t * a.ld_dx16, chunk, lane, d, o);
      }
    }
  }
  if (a.dw == nullptr) return;
  if (VPT == 1 && blockDim.y > 1) {
    // one row of partial sums a CTA: its warps' in their order
#pragma unroll
    for (int k = 0; k < 8; ++k) join[threadIdx.y][(VEC ? 8 * lane + k : 32 * k + lane)] = dw[0][k];
    __syncthreads();
    const int c = threadIdx.y * 32 + lane;  // eight warps: 256 channels
    if (c < d) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += join[i][c];
      a.partial[static_cast<long long>(blockIdx.x) * d + c] = sum;
    }
    return;
  }
  float* to = a.partial + static_cast<long long>(blockIdx.x) * d;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    // [CTAs, d] of the library's own: whole vectors where d allows
    if (d % 8 == 0)
      row_store<VEC>(to, j * warps + warp, lane, d, dw[j]);
    else
      row_store<false>(to, j * warps + warp, lane, d, dw[j]);
  }
}

constexpr int kDwRows = 32;

// dw[c] = sum over the CTAs of partial[CTA][c]: 32 columns a CTA, kDwRows threads
// a column.
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

Shape shape_of(long long T, int d, int sms, bool s_f32) {
  Shape p;
  const int chunks = (d + 255) / 256;
  p.vpt = chunks > 32 ? 4 : !s_f32 && chunks > 4 ? 2 : 1;
  p.warps = (chunks + p.vpt - 1) / p.vpt;
  p.rows = p.warps == 1 ? 8 : 1;  // eight: what the kernel joins
  // warps an SM: one piece a thread, 24 / 32 / 40: 22 / 20 / 22 us for 4096 x 2048 in bf16
  int per_sm = (p.vpt == 2 ? 16 : 32) / (p.warps * p.rows);
  if (per_sm < 1) per_sm = 1;
  const long long want = (T + p.rows - 1) / p.rows, most = static_cast<long long>(per_sm) * sms;
  p.ctas = static_cast<int>(want < most ? want : most);
  return p;
}

bool whole(const void* p, long long ld, int size, int unit) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % unit) == 0 && ld * size % unit == 0);
}

template <typename YT, typename ST, bool DS, bool VEC>
cudaError_t launch_vpt(const NormBackwardArgs& a, const Shape& p, cudaStream_t s) {
  auto kern = rms_norm_backward_kernel<YT, ST, DS, VEC, 1>;
  if (p.vpt == 4) kern = rms_norm_backward_kernel<YT, ST, DS, VEC, 4>;
  if constexpr (sizeof(ST) == 2) {
    if (p.vpt == 2) kern = rms_norm_backward_kernel<YT, ST, DS, VEC, 2>;
  }
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
  const int a = shape_of(T, d, sms, false).ctas, b = shape_of(T, d, sms, true).ctas;
  return a > b ? a : b;
}

cudaError_t launch_rms_norm_backward(const NormBackwardArgs& a, int sms, cudaStream_t s) {
  const PdlScope pdl(true);
  const Shape p = shape_of(a.T, a.d, sms, a.s_f32 != 0);
  cudaError_t e;
  if (a.dy_f32)
    e = a.s_f32 ? launch_sum<float, float>(a, p, s) : launch_sum<float, __nv_bfloat16>(a, p, s);
  else
    e = a.s_f32 ? launch_sum<__nv_bfloat16, float>(a, p, s)
                : launch_sum<__nv_bfloat16, __nv_bfloat16>(a, p, s);
  if (e != cudaSuccess || a.dw == nullptr) return e;
  return launch_kernel(rms_norm_dw_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32)),
                       dim3(32, kDwRows), 0, s, 1, false, static_cast<const float*>(a.partial),
                       p.ctas, a.d, a.dw);
}

}  // namespace lmoe

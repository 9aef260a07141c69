// Launcher of the gated block's products.
#include "ffn_gemm.cuh"
#include "kernels.h"

namespace lmoe {

template <int EPI, int SHAPE>
static cudaError_t launch_ffn_impl(const FfnArgs& a, int sms, cudaStream_t s) {
  constexpr bool PAIR = SHAPE == kFfnPair;
  static int units_of[kMaxDevices] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  int& most = units_of[dev];
  if (most == 0) {
    cudaError_t e = cudaFuncSetAttribute(ffn_gemm_kernel<EPI, SHAPE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         ffn_smem_bytes(EPI));
    if (e != cudaSuccess) return e;
    int n = sms;
    if (PAIR) {
      // pairs that can be resident at once
      cudaLaunchConfig_t cfg;
      memset(&cfg, 0, sizeof(cfg));
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(static_cast<unsigned>(2 * (sms / 2)), 1, 1);
      cfg.blockDim = dim3(kFfnThreads, 1, 1);
      cfg.dynamicSmemBytes = ffn_smem_bytes(EPI);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n, ffn_gemm_kernel<EPI, SHAPE>, &cfg);
      if (e != cudaSuccess) return e;
      if (n > sms / 2) n = sms / 2;
    }
    if (n < 1) return cudaErrorInvalidConfiguration;
    most = n;
  }
  const int units = a.tiles < most ? a.tiles : most;
  return launch_kernel(ffn_gemm_kernel<EPI, SHAPE>,
                       dim3(static_cast<unsigned>(PAIR ? 2 * units : units)), dim3(kFfnThreads),
                       ffn_smem_bytes(EPI), s, PAIR ? 2 : 1, false, a);
}

// A CTA a row, 8 channels a thread at a time.
__global__ void __launch_bounds__(256)
    ffn_pad_kernel(const __nv_bfloat16* x, long long ld_x, const __nv_bfloat16* dy, long long ld_dy,
                   int tokens, int d, int F, __nv_bfloat16* xs, __nv_bfloat16* dys,
                   __nv_bfloat16* h, __nv_bfloat16* dg, __nv_bfloat16* du) {
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.x;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c = threadIdx.x * 8; c < d; c += 256 * 8) {
    const long long to = static_cast<long long>(row) * d + c;
    *reinterpret_cast<uint4*>(dys + to) =
        row < tokens ? *reinterpret_cast<const uint4*>(dy + row * ld_dy + c) : zero;
    if (x != nullptr)
      *reinterpret_cast<uint4*>(xs + to) =
          row < tokens ? *reinterpret_cast<const uint4*>(x + row * ld_x + c) : zero;
  }
  if (row < tokens) return;
  for (int c = threadIdx.x * 8; c < F; c += 256 * 8) {
    const long long to = static_cast<long long>(row) * F + c;
    *reinterpret_cast<uint4*>(h + to) = zero;
    *reinterpret_cast<uint4*>(dg + to) = zero;
    *reinterpret_cast<uint4*>(du + to) = zero;
  }
}

cudaError_t launch_ffn_pad(const __nv_bfloat16* x, long long ld_x, const __nv_bfloat16* dy,
                           long long ld_dy, int tokens, int d, int F, __nv_bfloat16* xs,
                           __nv_bfloat16* dys, __nv_bfloat16* h, __nv_bfloat16* dg,
                           __nv_bfloat16* du, cudaStream_t s) {
  return launch_kernel(ffn_pad_kernel, dim3(kFfnLeastRows), dim3(256), 0, s, 1, false, x, ld_x, dy,
                       ld_dy, tokens, d, F, xs, dys, h, dg, du);
}

cudaError_t launch_ffn(int epi, int shape, const FfnArgs& a, int sms, cudaStream_t s) {
  if (epi == kFfnGateUp)
    return shape == kFfnPair ? launch_ffn_impl<kFfnGateUp, kFfnPair>(a, sms, s)
                             : launch_ffn_impl<kFfnGateUp, kFfnSingle>(a, sms, s);
  if (epi == kFfnDGate)
    return shape == kFfnPair ? launch_ffn_impl<kFfnDGate, kFfnPair>(a, sms, s)
                             : launch_ffn_impl<kFfnDGate, kFfnSingle>(a, sms, s);
  return shape == kFfnPair ? launch_ffn_impl<kFfnPlain, kFfnPair>(a, sms, s)
                           : launch_ffn_impl<kFfnPlain, kFfnSingle>(a, sms, s);
}

}  // namespace lmoe

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

// Instantiations and launcher of the Newton-Schulz products.
#include "kernels.h"
#include "ns.h"

namespace lmoe {

template <bool PAIR, bool AMN, bool BMN, int EPI>
static cudaError_t launch_ns_impl(const CUtensorMap& ma, const CUtensorMap& mb, const NsArgs& a,
                                  int sms, cudaStream_t s) {
  static int units_of[kMaxDevices] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  int& most = units_of[dev];
  if (most == 0) {
    cudaError_t e = cudaFuncSetAttribute(ns_gemm_kernel<PAIR, AMN, BMN, EPI>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmemBytes);
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
      cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
      cfg.blockDim = dim3(kNsThreads, 1, 1);
      cfg.dynamicSmemBytes = kNsSmemBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n, ns_gemm_kernel<PAIR, AMN, BMN, EPI>, &cfg);
      if (e != cudaSuccess) return e;
      if (n > sms / 2) n = sms / 2;
    }
    if (n < 1) return cudaErrorInvalidConfiguration;
    most = n;
  }
  const long long total = static_cast<long long>(a.tiles) * a.batch;
  const int units = static_cast<int>(total < most ? total : most);
  return launch_kernel(ns_gemm_kernel<PAIR, AMN, BMN, EPI>,
                       dim3(static_cast<unsigned>(PAIR ? 2 * units : units)), dim3(kNsThreads),
                       kNsSmemBytes, s, PAIR ? 2 : 1, false, ma, mb, a);
}

template <bool PAIR>
static cudaError_t launch_ns_pick(int epi, bool tall, const CUtensorMap& ma, const CUtensorMap& mb,
                                  const NsArgs& a, int sms, cudaStream_t s) {
  switch (epi) {
    case kNsGram:
      return tall ? launch_ns_impl<PAIR, true, true, kNsGram>(ma, mb, a, sms, s)
                  : launch_ns_impl<PAIR, false, false, kNsGram>(ma, mb, a, sms, s);
    case kNsPoly:
      return launch_ns_impl<PAIR, false, false, kNsPoly>(ma, mb, a, sms, s);
    default:
      return tall ? launch_ns_impl<PAIR, false, false, kNsApply>(ma, mb, a, sms, s)
                  : launch_ns_impl<PAIR, false, true, kNsApply>(ma, mb, a, sms, s);
  }
}

cudaError_t launch_ns_gemm(int epi, bool tall, bool pair, const CUtensorMap& ma,
                           const CUtensorMap& mb, const NsArgs& a, int sms, cudaStream_t s) {
  return pair ? launch_ns_pick<true>(epi, tall, ma, mb, a, sms, s)
              : launch_ns_pick<false>(epi, tall, ma, mb, a, sms, s);
}

}  // namespace lmoe

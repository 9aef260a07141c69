// Launcher of the Newton-Schulz iteration.
#include "kernels.h"
#include "ns.h"

namespace lmoe {

template <int SHAPE, bool SPLIT>
static cudaError_t launch_ns_impl(const NsMaps& m, const NsArgs& a, int sms, cudaStream_t s) {
  constexpr bool PAIR = SHAPE == kNsPair;
  static int units_of[kMaxDevices] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  int& most = units_of[dev];
  if (most == 0) {
    cudaError_t e = cudaFuncSetAttribute(
        ns_iterate_kernel<SHAPE, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        ns_smem_bytes(SHAPE));
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
      cfg.dynamicSmemBytes = ns_smem_bytes(SHAPE);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n, ns_iterate_kernel<SHAPE, SPLIT>, &cfg);
      if (e != cudaSuccess) return e;
      if (n > sms / 2) n = sms / 2;
    }
    if (n < 1) return cudaErrorInvalidConfiguration;
    most = n;
  }
  // no more units than the widest phase of all matrices in flight has tiles
  const long long sym = static_cast<long long>(a.sym_tiles) * a.split;
  const long long wide = (sym > a.apply_tiles ? sym : a.apply_tiles) * a.batch;
  const int units = static_cast<int>(wide < most ? wide : most);
  return launch_kernel(ns_iterate_kernel<SHAPE, SPLIT>,
                       dim3(static_cast<unsigned>(PAIR ? 2 * units : units)), dim3(kNsThreads),
                       ns_smem_bytes(SHAPE), s, PAIR ? 2 : 1, false, m, a);
}

cudaError_t launch_ns_iterate(int shape, const NsMaps& m, const NsArgs& a, int sms,
                              cudaStream_t s) {
  if (shape == kNsPair) return launch_ns_impl<kNsPair, false>(m, a, sms, s);
  if (shape == kNsSingle)
    return a.split > 1 ? launch_ns_impl<kNsSingle, true>(m, a, sms, s)
                       : launch_ns_impl<kNsSingle, false>(m, a, sms, s);
  return a.split > 1 ? launch_ns_impl<kNsNarrow, true>(m, a, sms, s)
                     : launch_ns_impl<kNsNarrow, false>(m, a, sms, s);
}

}  // namespace lmoe

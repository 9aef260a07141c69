// Launcher of the one-launch Newton-Schulz iteration for short sides up to 128.
#include "kernels.h"
#include "ns.h"
#include "ns_small.cuh"

namespace lmoe {

// Attributes once per device; the clusters of `ctas` CTAs that fit, 0 if none.
static cudaError_t small_prepare(int ctas, int* clusters) {
  static bool set[kMaxDevices] = {};
  static int fit[kMaxDevices][kSmallCluster + 1] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(ns_small_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(ns_small_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  if (fit[dev][ctas] == 0) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kSmallThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmallBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, ns_small_kernel, &cfg);
    if (e != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    fit[dev][ctas] = n > 0 ? n : -1;
  }
  *clusters = fit[dev][ctas] > 0 ? fit[dev][ctas] : 0;
  return cudaSuccess;
}

cudaError_t ns_small_plan(long long rows, long long cols, int* ctas, int* width) {
  *ctas = 0;
  const long long m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (m > kSmallSide || n > kSmallCluster * kSmallW) return cudaSuccess;
  // one CTA up to 256 columns (no exchange); then 128 columns a CTA while eight
  // CTAs hold them, then up to 256, then up to 16 CTAs
  long long c = n <= kSmallW ? 1 : (n + 127) / 128;
  if (c > 8) c = n <= 8 * kSmallW ? 8 : (n + kSmallW - 1) / kSmallW;
  const long long w = ((n + c - 1) / c + 63) / 64 * 64;
  c = (n + w - 1) / w;
  int clusters = 0;
  const cudaError_t e = small_prepare(static_cast<int>(c), &clusters);
  if (e != cudaSuccess) return e;
  if (clusters > 0) {
    *ctas = static_cast<int>(c);
    *width = static_cast<int>(w);
  }
  return cudaSuccess;
}

cudaError_t launch_ns_small(const NsSmallArgs& a, long long batch, cudaStream_t s) {
  return launch_kernel(ns_small_kernel,
                       dim3(static_cast<unsigned>(batch) * static_cast<unsigned>(a.ctas)),
                       dim3(kSmallThreads), kSmallBytes, s, a.ctas, false, a);
}

}  // namespace lmoe

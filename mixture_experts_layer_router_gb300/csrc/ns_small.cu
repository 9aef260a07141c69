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

// Rounds of clusters that the GPU holds at once decide the width: a matrix on
// fewer, wider CTAs takes longer alone, but more of them run at a time (clusters
// of eight leave the most SMs over). Measured, a matrix of 128 rows alone with 256 /
// 192 / 128 columns a CTA: 512 columns 52.6 / 47.3 / 41.5 us, 1024 columns 47.6 /
// 46.8 / 42.0; 64 matrices of 128 x 512 53.8 / 94.9 / 84.5, of 128 x 1024 97.6 /
// 145 / 213, 512 of 128 x 512 385 / 578 / 627. 64 columns a CTA change a single
// matrix by -6 to +3 % and double the rest. One CTA takes 256 columns without any
// exchange: 22.0 against 25.9 us on two.
cudaError_t ns_small_plan(long long batch, long long rows, long long cols, int* ctas,
                          int* width) {
  *ctas = 0;
  const long long m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (m > kSmallSide || n > kSmallCluster * kSmallW) return cudaSuccess;
  long long best = 0;
  for (long long w = kSmallW; w >= 128; w -= 64) {
    const long long c = (n + w - 1) / w;
    if (c > kSmallCluster) break;
    const long long even = ((n + c - 1) / c + 63) / 64 * 64;  // the same width in all CTAs
    int clusters = 0;
    const cudaError_t e = small_prepare(static_cast<int>(c), &clusters);
    if (e != cudaSuccess) return e;
    if (clusters == 0) continue;
    const long long cost = (batch + clusters - 1) / clusters * (380 + even);
    if (best == 0 || cost < best) {
      best = cost;
      *ctas = static_cast<int>(c);
      *width = static_cast<int>(even);
    }
    if (c == 1) break;
  }
  return cudaSuccess;
}

cudaError_t launch_ns_small(const NsSmallArgs& a, long long batch, cudaStream_t s) {
  return launch_kernel(ns_small_kernel,
                       dim3(static_cast<unsigned>(batch) * static_cast<unsigned>(a.ctas)),
                       dim3(kSmallThreads), kSmallBytes, s, a.ctas, false, a);
}

}  // namespace lmoe

// Launcher of the gated block's products for few tokens.
#include "ffn_few.cuh"
#include "kernels.h"

namespace lmoe {

int few_ctas(int tiles, int k_blocks, int sms) {
  const long long units = static_cast<long long>(tiles) * k_blocks;
  const int least = k_blocks < kFewLeast ? k_blocks : kFewLeast;
  const long long most = units / least;
  return static_cast<int>(most < 1 ? 1 : most < sms ? most : sms);
}

template <int EPI, int NT, bool MN>
static cudaError_t launch_few_impl(const FewArgs& a, int sms, cudaStream_t s) {
  static bool smem_set[kMaxDevices] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!smem_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(ffn_few_kernel<EPI, NT, MN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             few_smem_bytes(NT));
    if (e != cudaSuccess) return e;
    smem_set[dev] = true;
  }
  return launch_kernel(ffn_few_kernel<EPI, NT, MN>,
                       dim3(static_cast<unsigned>(few_ctas(a.tiles, a.k_blocks, sms))),
                       dim3(kFewThreads), few_smem_bytes(NT), s, 1, false, a);
}

template <int EPI, bool MN>
static cudaError_t launch_few_tokens(const FewArgs& a, int sms, cudaStream_t s) {
  switch (few_tokens(a.tokens)) {
    case 16: return launch_few_impl<EPI, 16, MN>(a, sms, s);
    case 32: return launch_few_impl<EPI, 32, MN>(a, sms, s);
    case 64: return launch_few_impl<EPI, 64, MN>(a, sms, s);
    default: return launch_few_impl<EPI, 128, MN>(a, sms, s);
  }
}

cudaError_t launch_ffn_few(int epi, bool transposed, const FewArgs& a, int sms, cudaStream_t s) {
  if (epi == kFfnGateUp) return launch_few_tokens<kFfnGateUp, false>(a, sms, s);
  if (epi == kFfnDGate) return launch_few_tokens<kFfnDGate, true>(a, sms, s);
  return transposed ? launch_few_tokens<kFfnPlain, true>(a, sms, s)
                    : launch_few_tokens<kFfnPlain, false>(a, sms, s);
}

}  // namespace lmoe

// C ABI of the RMS norm and of gradient clipping (declared in
// include/latentmoe.h): argument checks and launches. No handle; scratch is the
// caller's, so calls on different streams do not meet.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "grads.h"
#include "kernels.h"
#include "latentmoe.h"
#include "norm.h"

namespace {

bool known(int64_t dtype) { return dtype == LATENTMOE_BF16 || dtype == LATENTMOE_FP32; }
int size_of(int64_t dtype) { return dtype == LATENTMOE_FP32 ? 4 : 2; }
bool aligned_to(const void* p, int size) {
  return (reinterpret_cast<uintptr_t>(p) % static_cast<unsigned>(size)) == 0;
}

// SMs of the current device; 0 on a CUDA error.
int device_sms() {
  static int sms_of[lmoe::kMaxDevices] = {};
  const int dev = lmoe::current_device_index();
  if (dev < 0) return 0;
  if (sms_of[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    sms_of[dev] = n;
  }
  return sms_of[dev];
}

// The SMs that workspace sizes are made for, whatever device is current or
// whether there is one: as many CTAs as any launch may take.
constexpr int kMostSms = 256;

int check_rows(int64_t T, int64_t d) {
  if (T < 1 || d < 1) return LATENTMOE_ERR_INVALID_ARG;
  if (d > lmoe::kNormMaxWidth || T > INT32_MAX) return LATENTMOE_ERR_UNSUPPORTED;
  return LATENTMOE_OK;
}

// A row stride: 0 means d.
bool stride(int64_t* ld, int64_t d) {
  if (*ld == 0) *ld = d;
  return *ld >= d;
}

// ---- gradients

struct Span {
  uintptr_t begin, end;
  int64_t of;
};

// Whether every out is apart from every other tensor's g and out, and from its own
// g unless it is that.
bool outs_apart(const latentmoe_gradient* g, int64_t count) {
  std::vector<Span> outs;
  outs.reserve(static_cast<size_t>(count));
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(g[i].out);
    outs.push_back({p, p + static_cast<uintptr_t>(g[i].n) * size_of(g[i].dtype), i});
  }
  std::sort(outs.begin(), outs.end(),
            [](const Span& a, const Span& b) { return a.begin < b.begin; });
  for (size_t i = 1; i < outs.size(); ++i)
    if (outs[i].begin < outs[i - 1].end) return false;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(g[i].g);
    const uintptr_t end = p + static_cast<uintptr_t>(g[i].n) * size_of(g[i].dtype);
    // the outs do not overlap, so their ends are in order too: the first that ends past p
    auto it = std::upper_bound(outs.begin(), outs.end(), p,
                               [](uintptr_t v, const Span& s) { return v < s.end; });
    for (; it != outs.end() && it->begin < end; ++it)
      if (it->of != i || g[i].out != g[i].g) return false;
  }
  return true;
}

int check_grads(const latentmoe_gradient* g, int64_t count, bool clip, const float* norm,
                const void* ws, size_t bytes) {
  if (count < 0 || (count > 0 && g == nullptr) || norm == nullptr || ws == nullptr)
    return LATENTMOE_ERR_INVALID_ARG;
  if (count > (1ll << 24)) return LATENTMOE_ERR_UNSUPPORTED;
  if (bytes < latentmoe_grad_workspace(count)) return LATENTMOE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n < 0 || !known(g[i].dtype)) return LATENTMOE_ERR_INVALID_ARG;
    if (g[i].n == 0) continue;
    if (g[i].g == nullptr || (clip && g[i].out == nullptr)) return LATENTMOE_ERR_INVALID_ARG;
    if (g[i].n > (1ll << 44)) return LATENTMOE_ERR_UNSUPPORTED;
  }
  if (!aligned_to(ws, 16) || !aligned_to(norm, 4)) return LATENTMOE_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const int size = size_of(g[i].dtype);
    if (!aligned_to(g[i].g, size) || (clip && !aligned_to(g[i].out, size)))
      return LATENTMOE_ERR_UNSUPPORTED;
  }
  return LATENTMOE_OK;
}

// The tensors from *next on that fit a launch; false if their tiles do not count.
bool next_table(const latentmoe_gradient* g, int64_t count, int64_t* next,
                lmoe::GradTable<lmoe::kGradBatch>* t) {
  t->count = 0;
  long long tiles = 0;
  for (; *next < count && t->count < lmoe::kGradBatch; ++*next) {
    const latentmoe_gradient& x = g[*next];
    if (x.n == 0) continue;
    lmoe::GradEntry& e = t->e[t->count++];
    e.g = x.g;
    e.out = x.out;
    e.n = x.n;
    e.first = static_cast<unsigned>(tiles);
    e.f32 = x.dtype == LATENTMOE_FP32;
    tiles += lmoe::grad_tiles(x.g, x.n, size_of(x.dtype));
    if (tiles > INT32_MAX) return false;
  }
  t->tiles = static_cast<unsigned>(tiles);
  return true;
}

// Both entries; max_norm < 0: the norm alone.
int grads(const latentmoe_gradient* g, int64_t count, double max_norm, double eps, float* norm,
          void* ws, cudaStream_t s) {
  const bool clip = max_norm >= 0.0;
  const int sms = device_sms();
  if (sms < 1 || sms > kMostSms) return LATENTMOE_ERR_CUDA;
  double* partial = static_cast<double*>(ws);
  auto* table = new (std::nothrow) lmoe::GradTable<lmoe::kGradBatch>;
  if (table == nullptr) return LATENTMOE_ERR_OUT_OF_MEMORY;
  int partials = 0;
  bool fits = true;
  for (int64_t next = 0; next < count && fits;) fits = next_table(g, count, &next, table);
  cudaError_t e = cudaSuccess;
  for (int64_t next = 0; next < count && fits && e == cudaSuccess;) {
    next_table(g, count, &next, table);
    if (table->count == 0) continue;
    e = lmoe::launch_grad_squares(*table, partial + partials, sms, s);
    partials += lmoe::grad_ctas(table->tiles, sms);
  }
  if (fits && e == cudaSuccess && (!clip || partials == 0))
    e = lmoe::launch_grad_norm(partial, partials, norm, s);
  if (fits && e == cudaSuccess && clip) {
    float* to = partials == 0 ? nullptr : norm;
    for (int64_t next = 0; next < count && e == cudaSuccess;) {
      // a single table is still at hand
      if (next != 0 || count > lmoe::kGradBatch) next_table(g, count, &next, table);
      else next = count;
      if (table->count == 0) continue;
      e = lmoe::launch_grad_scale(*table, partial, partials, max_norm, eps, to, sms, s);
      to = nullptr;
    }
  }
  delete table;
  if (!fits) return LATENTMOE_ERR_UNSUPPORTED;
  return e == cudaSuccess ? LATENTMOE_OK : LATENTMOE_ERR_CUDA;
}

}  // namespace

extern "C" {

int latentmoe_rms_norm(const latentmoe_norm* n, int64_t T, int64_t d, latentmoe_stream_t st) {
  if (n == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  latentmoe_norm p = *n;
  if (p.x == nullptr || p.weight == nullptr || (p.y == nullptr && p.codes == nullptr) ||
      (p.codes != nullptr && p.scales == nullptr) || (p.sum != nullptr && p.residual == nullptr))
    return LATENTMOE_ERR_INVALID_ARG;
  if (!known(p.x_dtype) || !known(p.weight_dtype) ||
      (p.residual != nullptr && !known(p.residual_dtype)) || (p.y != nullptr && !known(p.y_dtype)))
    return LATENTMOE_ERR_INVALID_ARG;
  if (p.codes != nullptr && p.scale_block != 0 && p.scale_block != lmoe::kNormBlock)
    return LATENTMOE_ERR_INVALID_ARG;
  if (!(p.eps >= 1e-30f) || !isfinite(p.eps)) return LATENTMOE_ERR_INVALID_ARG;
  const int rc = check_rows(T, d);
  if (rc != LATENTMOE_OK) return rc;
  if (!stride(&p.ld_x, d) || !stride(&p.ld_residual, d) || !stride(&p.ld_sum, d) ||
      !stride(&p.ld_y, d) || !stride(&p.ld_codes, d))
    return LATENTMOE_ERR_INVALID_ARG;
  if (p.x_dtype == LATENTMOE_FP32 && p.residual != nullptr && p.residual_dtype == LATENTMOE_BF16)
    return LATENTMOE_ERR_UNSUPPORTED;
  if (!aligned_to(p.x, size_of(p.x_dtype)) || !aligned_to(p.weight, size_of(p.weight_dtype)) ||
      !aligned_to(p.residual, size_of(p.residual_dtype)) ||
      !aligned_to(p.sum, size_of(p.residual_dtype)) || !aligned_to(p.y, size_of(p.y_dtype)) ||
      !aligned_to(p.scales, 4) || !aligned_to(p.rstd, 4))
    return LATENTMOE_ERR_UNSUPPORTED;
  lmoe::NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = p.x;
  a.residual = p.residual;
  a.weight = p.weight;
  a.sum = p.sum;
  a.y = p.y;
  a.codes = p.codes;
  a.scales = p.scales;
  a.rstd = p.rstd;
  a.ld_x = p.ld_x;
  a.ld_residual = p.ld_residual;
  a.ld_sum = p.ld_sum;
  a.ld_y = p.ld_y;
  a.ld_codes = p.ld_codes;
  a.x_f32 = p.x_dtype == LATENTMOE_FP32;
  a.residual_f32 = p.residual_dtype == LATENTMOE_FP32;
  a.weight_f32 = p.weight_dtype == LATENTMOE_FP32;
  a.y_f32 = p.y_dtype == LATENTMOE_FP32;
  a.d = static_cast<int>(d);
  a.per_block = p.scale_block != 0;
  a.blocks = a.per_block ? static_cast<int>((d + lmoe::kNormBlock - 1) / lmoe::kNormBlock) : 1;
  a.T = T;
  a.eps = p.eps;
  const cudaError_t e = lmoe::launch_rms_norm(a, reinterpret_cast<cudaStream_t>(st));
  return e == cudaSuccess ? LATENTMOE_OK : LATENTMOE_ERR_CUDA;
}

size_t latentmoe_rms_norm_backward_workspace(int64_t T, int64_t d) {
  if (check_rows(T, d) != LATENTMOE_OK) return 0;
  return static_cast<size_t>(lmoe::norm_partials(T, static_cast<int>(d), kMostSms)) *
         static_cast<size_t>(d) * 4;
}

int latentmoe_rms_norm_backward(const latentmoe_norm_grad* n, int64_t T, int64_t d,
                                void* workspace, size_t workspace_bytes, latentmoe_stream_t st) {
  if (n == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  latentmoe_norm_grad p = *n;
  if (p.dy == nullptr || p.s == nullptr || p.weight == nullptr || p.rstd == nullptr ||
      p.dx == nullptr)
    return LATENTMOE_ERR_INVALID_ARG;
  if (!known(p.dy_dtype) || !known(p.s_dtype) || !known(p.weight_dtype))
    return LATENTMOE_ERR_INVALID_ARG;
  if (p.dx16 != nullptr && p.s_dtype != LATENTMOE_FP32) return LATENTMOE_ERR_INVALID_ARG;
  const int rc = check_rows(T, d);
  if (rc != LATENTMOE_OK) return rc;
  if (!stride(&p.ld_dy, d) || !stride(&p.ld_s, d) || !stride(&p.ld_d_sum, d) ||
      !stride(&p.ld_dx, d) || !stride(&p.ld_dx16, d))
    return LATENTMOE_ERR_INVALID_ARG;
  if (p.dw != nullptr && (workspace == nullptr ||
                          workspace_bytes < latentmoe_rms_norm_backward_workspace(T, d)))
    return LATENTMOE_ERR_INVALID_ARG;
  const int s_size = size_of(p.s_dtype);
  if (!aligned_to(p.dy, size_of(p.dy_dtype)) || !aligned_to(p.s, s_size) ||
      !aligned_to(p.weight, size_of(p.weight_dtype)) || !aligned_to(p.rstd, 4) ||
      !aligned_to(p.d_sum, s_size) || !aligned_to(p.dx, s_size) || !aligned_to(p.dx16, 2) ||
      !aligned_to(p.dw, 4) || (p.dw != nullptr && !aligned_to(workspace, 16)))
    return LATENTMOE_ERR_UNSUPPORTED;
  const int sms = device_sms();
  if (sms < 1 || sms > kMostSms) return LATENTMOE_ERR_CUDA;
  lmoe::NormBackwardArgs a;
  memset(&a, 0, sizeof(a));
  a.dy = p.dy;
  a.s = p.s;
  a.weight = p.weight;
  a.rstd = p.rstd;
  a.d_sum = p.d_sum;
  a.dx = p.dx;
  a.dx16 = p.dx16;
  a.dw = p.dw;
  a.partial = static_cast<float*>(workspace);
  a.ld_dy = p.ld_dy;
  a.ld_s = p.ld_s;
  a.ld_d_sum = p.ld_d_sum;
  a.ld_dx = p.ld_dx;
  a.ld_dx16 = p.ld_dx16;
  a.dy_f32 = p.dy_dtype == LATENTMOE_FP32;
  a.s_f32 = p.s_dtype == LATENTMOE_FP32;
  a.weight_f32 = p.weight_dtype == LATENTMOE_FP32;
  a.d = static_cast<int>(d);
  a.T = T;
  const cudaError_t e =
      lmoe::launch_rms_norm_backward(a, sms, reinterpret_cast<cudaStream_t>(st));
  return e == cudaSuccess ? LATENTMOE_OK : LATENTMOE_ERR_CUDA;
}

size_t latentmoe_grad_workspace(int64_t count) {
  if (count < 0) return 0;
  const size_t launches = static_cast<size_t>((count + lmoe::kGradBatch - 1) / lmoe::kGradBatch);
  return (launches < 1 ? 1 : launches) *
         static_cast<size_t>(lmoe::grad_ctas(~0u, kMostSms)) * sizeof(double);
}

int latentmoe_grad_norm(const latentmoe_gradient* g, int64_t count, float* norm, void* workspace,
                        size_t workspace_bytes, latentmoe_stream_t st) {
  const int rc = check_grads(g, count, false, norm, workspace, workspace_bytes);
  if (rc != LATENTMOE_OK) return rc;
  return grads(g, count, -1.0, 0.0, norm, workspace, reinterpret_cast<cudaStream_t>(st));
}

int latentmoe_grad_clip(const latentmoe_gradient* g, int64_t count, double max_norm, double eps,
                        float* norm, void* workspace, size_t workspace_bytes,
                        latentmoe_stream_t st) {
  if (!(max_norm >= 0.0) || !(eps >= 0.0) || !isfinite(eps)) return LATENTMOE_ERR_INVALID_ARG;
  const int rc = check_grads(g, count, true, norm, workspace, workspace_bytes);
  if (rc != LATENTMOE_OK) return rc;
  try {
    if (!outs_apart(g, count)) return LATENTMOE_ERR_INVALID_ARG;
  } catch (...) {
    return LATENTMOE_ERR_OUT_OF_MEMORY;
  }
  return grads(g, count, max_norm, eps, norm, workspace, reinterpret_cast<cudaStream_t>(st));
}

}  // extern "C"

// C ABI of the Newton-Schulz orthogonalisation (declared in
// include/latentmoe.h): handle, workspace, scales, launch sequence.
//
// Muon with Newton-Schulz products is named for these models in "Frontier
// Pre-training at Microsoft AI" (optimiser section) and "MAI-Base-2:
// Microsoft's 2.8T base model, and whether its compute numbers add up"; the
// iteration is the published quintic one.
//
// Launches of one call: norm, init, then gram, poly, apply for every step;
// the last apply writes the caller's output or weights.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "kernels.h"
#include "latentmoe.h"
#include "ns.h"
#include "tensor_map.h"

using lmoe::NsArgs;

namespace {

constexpr int kMaxSteps = 32;
constexpr long long kMaxSide = 65536;
// fp16 entries are kept at or below 2^14, a quarter of the format's range
constexpr double kHalfTop = 16384.0;

// Per step: coefficients and the power-of-two scales of the fp16 X, A and
// P = b A + c A^2.
struct Step {
  float a, b, c;
  float sx, sa, sp;
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

float pow2_scale(double bound) {
  if (!(bound > 0.0)) return 1.0f;
  int e = static_cast<int>(floor(log2(kHalfTop / bound)));
  if (e > 60) e = 60;
  if (e < -60) e = -60;
  return static_cast<float>(ldexp(1.0, e));
}

// 3-D fp16 map (cols, rows, batch) with row stride ld, boxes of 64 x 64 x 1,
// 128-byte swizzle, zeros outside.
bool make_ns_map(CUtensorMap* map, const void* p, long long batch, long long rows, long long cols,
                 long long ld) {
  const lmoe::EncodeTiledFn fn = lmoe::tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2,
                                 static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(rows) * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

struct latentmoe_muon {
  long long batch = 0, rows = 0, cols = 0;
  long long side = 0;   // min(rows, cols): A and P are side x side
  bool tall = false;
  int steps = 0;
  float eps = 0.0f;
  Step step[kMaxSteps];
  int device = 0;
  int sms = 1;
  long long ldx = 0, lda = 0;
  int chunks = 1;
  long long chunk = 0;
  void* ws = nullptr;
  float* x32 = nullptr;
  __half* x16[2] = {nullptr, nullptr};
  __half* gram = nullptr;
  __half* poly = nullptr;
  float* partial = nullptr;
  unsigned* status = nullptr;
  CUtensorMap m_x[2], m_gram, m_poly;
  int pairs = 2;  // 0 single SMs, 1 SM pairs, 2 by the number of tiles
  int64_t launches = 0;
  int last_cuda = 0;
};

namespace {

int fail(latentmoe_muon* h, cudaError_t e) {
  h->last_cuda = static_cast<int>(e);
  return e == cudaErrorMemoryAllocation ? LATENTMOE_ERR_OUT_OF_MEMORY : LATENTMOE_ERR_CUDA;
}

#define NS_CK(h, call)                          \
  do {                                          \
    const cudaError_t e_ = (call);              \
    if (e_ != cudaSuccess) return fail(h, e_);  \
  } while (0)

long long tiles_of(long long M, long long N, long long bt, bool sym) {
  const long long mt = (M + bt - 1) / bt, nt = (N + bt - 1) / bt;
  return sym ? mt * (mt + 1) / 2 : mt * nt;
}

// SM pairs (256 x 256 tiles) or single SMs (128 x 128): whichever needs fewer
// rounds of tiles, a pair tile being two single tiles' work per SM.
bool use_pairs(const latentmoe_muon* h, long long M, long long N, bool sym) {
  if (h->pairs != 2) return h->pairs == 1;
  const long long tp = tiles_of(M, N, 256, sym) * h->batch;
  const long long ts = tiles_of(M, N, 128, sym) * h->batch;
  const long long np = h->sms / 2 > 0 ? h->sms / 2 : 1;
  const long long rounds_p = (tp + np - 1) / np, rounds_s = (ts + h->sms - 1) / h->sms;
  return 2 * rounds_p <= rounds_s;
}

int product(latentmoe_muon* h, int epi, const CUtensorMap& ma, const CUtensorMap& mb, long long M,
            long long N, long long K, NsArgs a, cudaStream_t s) {
  const bool sym = epi != lmoe::kNsApply;
  const bool pair = use_pairs(h, M, N, sym);
  const long long bt = pair ? 256 : 128;
  a.batch = static_cast<int>(h->batch);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.k_blocks = static_cast<int>((K + lmoe::kNsBK - 1) / lmoe::kNsBK);
  a.m_tiles = static_cast<int>((M + bt - 1) / bt);
  a.n_tiles = static_cast<int>((N + bt - 1) / bt);
  a.tiles = static_cast<int>(tiles_of(M, N, bt, sym));
  a.status = h->status;
  NS_CK(h, lmoe::launch_ns_gemm(epi, h->tall, pair, ma, mb, a, h->sms, s));
  h->launches += 1;
  return LATENTMOE_OK;
}

// The whole iteration on U; the last product writes `out` as out_mode says.
int iterate(latentmoe_muon* h, const lmoe::NsUpdate& u, int out_mode, void* out, float keep,
            float move, cudaStream_t s) {
  const lmoe::PdlScope pdl(true);
  const long long n = h->rows * h->cols;
  NS_CK(h, lmoe::launch_ns_norm(u, h->batch, n, h->chunks, h->chunk, h->partial, s));
  NS_CK(h, lmoe::launch_ns_init(u, h->batch, h->rows, h->cols, h->ldx, h->chunks, h->partial,
                                h->eps, h->step[0].sx, h->x32, h->x16[0], s));
  h->launches += 2;
  const long long m = h->side;
  for (int i = 0; i < h->steps; ++i) {
    const Step& st = h->step[i];
    const bool last = i + 1 == h->steps;
    const CUtensorMap& mx = h->m_x[i & 1];
    NsArgs a;
    memset(&a, 0, sizeof(a));
    a.ld = h->lda;
    a.bstride = m * h->lda;
    // A, scaled by sa, from X scaled by sx
    a.alpha = st.sa / (st.sx * st.sx);
    a.out16 = h->gram;
    int r = product(h, lmoe::kNsGram, mx, mx, m, m, h->tall ? h->rows : h->cols, a, s);
    if (r != LATENTMOE_OK) return r;
    // P = b A + c A^2, scaled by sp
    a.alpha = st.c * st.sp / (st.sa * st.sa);
    a.beta = st.b * st.sp / st.sa;
    a.out16 = h->poly;
    a.old16 = h->gram;
    r = product(h, lmoe::kNsPoly, h->m_gram, h->m_gram, m, m, m, a, s);
    if (r != LATENTMOE_OK) return r;
    // X <- a X + P X (wide) or a X + X P (tall)
    a.alpha = 1.0f / (st.sp * st.sx);
    a.beta = st.a;
    a.scale = last ? 1.0f : h->step[i + 1].sx;
    a.out16 = h->x16[(i + 1) & 1];
    a.old16 = nullptr;
    a.x32 = h->x32;
    a.ld = h->ldx;
    a.bstride = h->rows * h->ldx;
    a.out_mode = last ? out_mode : static_cast<int>(lmoe::kNsOutNext);
    a.out = out;
    a.keep = keep;
    a.move = move;
    r = product(h, lmoe::kNsApply, h->tall ? mx : h->m_poly, h->tall ? h->m_poly : mx, h->rows,
                h->cols, m, a, s);
    if (r != LATENTMOE_OK) return r;
  }
  return LATENTMOE_OK;
}

}  // namespace

extern "C" {

int latentmoe_muon_create(const latentmoe_muon_dims* dims, latentmoe_muon_t* out) {
  if (out == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (dims == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  const latentmoe_muon_dims d = *dims;
  if (d.batch < 1 || d.rows < 1 || d.cols < 1 || d.steps < 1) return LATENTMOE_ERR_INVALID_ARG;
  if (!(d.eps >= 1e-30f) || !isfinite(d.eps)) return LATENTMOE_ERR_INVALID_ARG;
  if (d.rows > kMaxSide || d.cols > kMaxSide || d.batch > 65535 || d.steps > kMaxSteps)
    return LATENTMOE_ERR_UNSUPPORTED;
  Step step[kMaxSteps];
  // bound on the spectral norm of X before the step: 1 after the division by
  // the Frobenius norm, then the largest value of |a s + b s^3 + c s^5| on
  // [0, bound], each a little more for rounding (the scales leave a factor of
  // 4; a wide margin here would leave the interval that the usual coefficients
  // keep to, and grow)
  double u = 1.001;
  for (int i = 0; i < d.steps; ++i) {
    Step& st = step[i];
    st.a = d.coefs ? d.coefs[3 * i] : 3.4445f;
    st.b = d.coefs ? d.coefs[3 * i + 1] : -4.7750f;
    st.c = d.coefs ? d.coefs[3 * i + 2] : 2.0315f;
    if (!isfinite(st.a) || !isfinite(st.b) || !isfinite(st.c)) return LATENTMOE_ERR_INVALID_ARG;
    double next = 0.0, poly = 0.0;
    for (int j = 0; j <= 1024; ++j) {
      const double x = u * j / 1024.0, x2 = x * x;
      const double p = st.b * x2 + st.c * x2 * x2;
      poly = fmax(poly, fabs(p));
      next = fmax(next, fabs((st.a + p) * x));
    }
    st.sx = pow2_scale(u);
    st.sa = pow2_scale(u * u);
    st.sp = pow2_scale(poly);
    u = 1.002 * next;
    if (!(u < 1e6)) return LATENTMOE_ERR_INVALID_ARG;  // the coefficients diverge
    if (u < 1e-6) u = 1e-6;
  }
  const long long B = d.batch, R = d.rows, C = d.cols;
  const long long side = R < C ? R : C;
  const long long ldx = (C + 7) / 8 * 8, lda = (side + 7) / 8 * 8;
  // tile counts stay in int
  const long long t128 = ((R + 127) / 128) * ((C + 127) / 128);
  if (t128 * B > (1ll << 30)) return LATENTMOE_ERR_UNSUPPORTED;

  latentmoe_muon* h = new (std::nothrow) latentmoe_muon();
  if (h == nullptr) return LATENTMOE_ERR_OUT_OF_MEMORY;
  h->batch = B;
  h->rows = R;
  h->cols = C;
  h->side = side;
  h->tall = R > C;
  h->steps = static_cast<int>(d.steps);
  h->eps = d.eps;
  memcpy(h->step, step, sizeof(step));
  h->ldx = ldx;
  h->lda = lda;
  // blocks of the norm pass: 16 elements a thread or more, whole vectors
  const long long n = R * C;
  const long long unit = 8ll * lmoe::kNsNormThreads;
  long long chunk = 2 * unit;
  const long long need = (n + lmoe::kNsMaxChunks - 1) / lmoe::kNsMaxChunks;
  if (chunk < need) chunk = (need + unit - 1) / unit * unit;
  h->chunk = chunk;
  h->chunks = static_cast<int>((n + chunk - 1) / chunk);

  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    delete h;
    return LATENTMOE_ERR_CUDA;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 1023) / 1024 * 1024;
    return o;
  };
  const size_t xn = static_cast<size_t>(B) * R * ldx, an = static_cast<size_t>(B) * side * lda;
  const size_t o_x32 = take(xn * 4), o_x0 = take(xn * 2);
  const size_t o_x1 = h->steps > 1 ? take(xn * 2) : o_x0;
  const size_t o_gram = take(an * 2), o_poly = take(an * 2);
  const size_t o_partial = take(static_cast<size_t>(B) * h->chunks * 4), o_status = take(16);
  e = cudaMalloc(&h->ws, off);
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return e == cudaErrorMemoryAllocation ? LATENTMOE_ERR_OUT_OF_MEMORY : LATENTMOE_ERR_CUDA;
  }
  char* base = static_cast<char*>(h->ws);
  h->x32 = reinterpret_cast<float*>(base + o_x32);
  h->x16[0] = reinterpret_cast<__half*>(base + o_x0);
  h->x16[1] = reinterpret_cast<__half*>(base + o_x1);
  h->gram = reinterpret_cast<__half*>(base + o_gram);
  h->poly = reinterpret_cast<__half*>(base + o_poly);
  h->partial = reinterpret_cast<float*>(base + o_partial);
  h->status = reinterpret_cast<unsigned*>(base + o_status);
  e = cudaMemset(h->status, 0, 16);
  if (e != cudaSuccess || !make_ns_map(&h->m_x[0], h->x16[0], B, R, C, ldx) ||
      !make_ns_map(&h->m_x[1], h->x16[1], B, R, C, ldx) ||
      !make_ns_map(&h->m_gram, h->gram, B, side, side, lda) ||
      !make_ns_map(&h->m_poly, h->poly, B, side, side, lda)) {
    cudaFree(h->ws);
    delete h;
    return LATENTMOE_ERR_CUDA;
  }
  *out = h;
  return LATENTMOE_OK;
}

int latentmoe_muon_destroy(latentmoe_muon_t h) {
  if (h == nullptr) return LATENTMOE_OK;
  if (h->ws) cudaFree(h->ws);
  delete h;
  return LATENTMOE_OK;
}

int latentmoe_muon_orthogonalize(latentmoe_muon_t h, const void* g, int g_dtype, void* out,
                                 latentmoe_stream_t st) {
  if (h == nullptr || g == nullptr || out == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  if (g_dtype != LATENTMOE_BF16 && g_dtype != LATENTMOE_FP32) return LATENTMOE_ERR_INVALID_ARG;
  if (!aligned16(g) || !aligned16(out)) return LATENTMOE_ERR_UNSUPPORTED;
  NS_CK(h, cudaSetDevice(h->device));
  const lmoe::NsUpdate u = {g, g_dtype == LATENTMOE_FP32, nullptr, 0.0f, false};
  return iterate(h, u, lmoe::kNsOutBf16, out, 0.0f, 0.0f, reinterpret_cast<cudaStream_t>(st));
}

int latentmoe_muon_step(latentmoe_muon_t h, const latentmoe_muon_update* p,
                        latentmoe_stream_t st) {
  if (h == nullptr || p == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  if (p->g == nullptr || p->momentum == nullptr || p->w == nullptr)
    return LATENTMOE_ERR_INVALID_ARG;
  if ((p->g_dtype != LATENTMOE_BF16 && p->g_dtype != LATENTMOE_FP32) ||
      (p->w_dtype != LATENTMOE_BF16 && p->w_dtype != LATENTMOE_FP32))
    return LATENTMOE_ERR_INVALID_ARG;
  if (!isfinite(p->lr) || !isfinite(p->momentum_coef) || !isfinite(p->weight_decay) ||
      !isfinite(p->scale))
    return LATENTMOE_ERR_INVALID_ARG;
  if (!aligned16(p->g) || !aligned16(p->momentum) || !aligned16(p->w))
    return LATENTMOE_ERR_UNSUPPORTED;
  NS_CK(h, cudaSetDevice(h->device));
  const lmoe::NsUpdate u = {p->g, p->g_dtype == LATENTMOE_FP32, p->momentum, p->momentum_coef,
                            p->nesterov != 0};
  const double lr = p->lr;
  return iterate(h, u,
                 p->w_dtype == LATENTMOE_BF16 ? lmoe::kNsOutWeightBf16 : lmoe::kNsOutWeightF32,
                 p->w, static_cast<float>(1.0 - lr * p->weight_decay),
                 static_cast<float>(lr * p->scale), reinterpret_cast<cudaStream_t>(st));
}

int latentmoe_muon_set_sm_pairs(latentmoe_muon_t h, int mode) {
  if (h == nullptr || mode < 0 || mode > 2) return LATENTMOE_ERR_INVALID_ARG;
  h->pairs = mode;
  return LATENTMOE_OK;
}

int latentmoe_muon_get_status(latentmoe_muon_t h, uint32_t* device_status) {
  if (h == nullptr || device_status == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  NS_CK(h, cudaSetDevice(h->device));
  NS_CK(h, cudaDeviceSynchronize());
  unsigned v = 0;
  NS_CK(h, cudaMemcpy(&v, h->status, 4, cudaMemcpyDeviceToHost));
  NS_CK(h, cudaMemset(h->status, 0, 4));
  *device_status = v;
  if (v & LATENTMOE_STATUS_TIMEOUT) return LATENTMOE_ERR_TIMEOUT;
  return v != 0 ? LATENTMOE_ERR_DEVICE_STATUS : LATENTMOE_OK;
}

int latentmoe_muon_get_launch_count(latentmoe_muon_t h, int64_t* launches) {
  if (h == nullptr || launches == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  *launches = h->launches;
  return LATENTMOE_OK;
}

int latentmoe_muon_last_cuda_error(latentmoe_muon_t h) { return h ? h->last_cuda : 0; }

}  // extern "C"

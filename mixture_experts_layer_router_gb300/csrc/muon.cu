// C ABI of the Newton-Schulz orthogonalisation (declared in
// include/latentmoe.h): handle, workspace, scales, launch sequence.
//
// Muon with Newton-Schulz products is named for these models in "Frontier
// Pre-training at Microsoft AI" (optimiser section) and "MAI-Base-2:
// Microsoft's 2.8T base model, and whether its compute numbers add up"; the
// iteration is the published quintic one.
//
// Launches of one call: norm, init, and the iteration, whose last product
// writes the caller's output or weights; or, for short sides up to 128, one
// launch for everything.
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

using lmoe::kNsMaxSteps;
constexpr long long kMaxSide = 65536;
// fp16 entries are kept at or below 2^14, a quarter of the format's range
constexpr double kHalfTop = 16384.0;
// Matrices in flight at once: their X (fp32 and fp16 twice), A and P. Few leave
// SMs waiting between a matrix's phases, many leave L2 (129 MB) before they come
// round again; a phase's tiles touch only a part of the bytes, so the best size is
// above L2's. Measured, pairs: 64 x 2048 x 1024 (20 MB each) with 1 / 4 / 8 / 16 /
// 32 / 64 in flight 11.8 / 4.1 / 2.97 / 2.80 / 2.85 / 2.91 ms, 12 x 4096 x 2048
// (84 MB) with 1 / 2 / 3 / 6 / 12 5.15 / 3.31 / 3.15 / 3.20 / 3.26 ms, 1000 x 256 x
// 256 with 100 / 200 / 400 / 1000 1.81 / 1.73 / 1.73 / 1.77 ms.
constexpr long long kGroupBytes = 320ll << 20;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

float pow2_scale(double bound) {
  if (!(bound > 0.0)) return 1.0f;
  int e = static_cast<int>(floor(log2(kHalfTop / bound)));
  if (e > 60) e = 60;
  if (e < -60) e = -60;
  return static_cast<float>(ldexp(1.0, e));
}

// 3-D fp16 (or fp32) map (cols, rows, batch) with row stride ld, zeros outside;
// boxes of `box` columns x `box` rows. Swizzle: as wide as a box row, 64 or 128
// bytes.
bool make_ns_map(CUtensorMap* map, const void* p, long long batch, long long rows, long long cols,
                 long long ld, int box, bool f32 = false) {
  const lmoe::EncodeTiledFn fn = lmoe::tensor_map_encoder();
  if (fn == nullptr) return false;
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {
      static_cast<cuuint64_t>(ld) * size,
      static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(rows) * size};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(box), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(p), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

struct latentmoe_muon {
  long long batch = 0, rows = 0, cols = 0;
  long long side = 0;   // min(rows, cols): A and P are side x side
  bool tall = false;
  int steps = 0;
  float eps = 0.0f;
  float scale0 = 1.0f;  // of the first X
  int device = 0;
  int sms = 1;
  int group = 1;        // matrices in flight
  int chunks = 1;
  long long chunk = 0;
  void* ws = nullptr;
  float* partial = nullptr;
  float* x32 = nullptr;   // [batch, rows, ld_x]
  __half* x16 = nullptr;  // the first X
  NsArgs args;  // everything but the output and the tile shape
  lmoe::NsMaps maps;
  int pairs = 2;  // 0 single, 1 pair, 2 by the number of tiles, 3 narrow
  int small_ctas = 0, small_width = 0;  // the one-launch kernel's plan, 0: not for this size
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

// Tiles of a symmetric m x m result (on and below the diagonal) and of an M x N one.
long long sym_tiles(long long m, int shape) {
  const long long t = (m + lmoe::ns_bm(shape) - 1) / lmoe::ns_bm(shape);
  return t * (t + 1) / 2 * (lmoe::ns_bm(shape) / lmoe::ns_bn(shape));
}
long long tiles(long long M, long long N, int shape) {
  const long long bm = lmoe::ns_bm(shape), bn = lmoe::ns_bn(shape);
  return ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

// Into how many parts gram's k-blocks are split: a few tiles with a long K (the
// gradient of a router or a projection to a small latent) would leave most SMs
// idle. Joining the parts, through L2, costs about as much as 12 k-blocks, so a
// part has 8 or more and the split has to save more than those: 64 x 8704 (136
// k-blocks, 8 parts) 253 -> 110 us, 200 x 2000 (32, 4 parts) 118 -> 104, but 1024 x
// 1024 (16) in two parts 146 -> 158.
constexpr int kJoinBlocks = 12;
int gram_split(long long batch, long long side, int k_gram, int sms, int shape) {
  if (shape == lmoe::kNsPair) return 1;
  const long long free_sms = sms / (batch * sym_tiles(side, shape));
  long long split = free_sms < k_gram / 8 ? free_sms : k_gram / 8;
  if (split > 8) split = 8;
  if (split < 2 || (k_gram + split - 1) / split + kJoinBlocks >= k_gram) return 1;
  return static_cast<int>(split);
}

// apply takes the tiles that hold the first three quarters of A's rows first, so
// that the SMs that its last round leaves idle can begin with the gram tiles of
// those rows. Without / with, in turn: 4096 x 8704 2095 / 2005 us, 8704 x 4096 2227 /
// 2168, 4096 x 4096 1155 / 1136, 6 of 640 x 640 154 / 148; one or two quarters first
// gain less (4096 x 8704 1 % and nothing), stacks of many matrices take the same
// time either way.
long long apply_cut(long long side) {
  const long long cut = side * 3 / 4 / 256 * 256;  // whole tiles of every shape
  return cut > 0 ? cut : side;
}

// Rounds of tiles decide the shape: a round takes its k-blocks and, once a phase,
// the hand-over of the results to the next phase. In ns, measured: a k-block 270
// (narrow), 320 (single), 310 (pair): an SM takes in about 64 bytes a clock, which
// bounds the first two; a hand-over 4200, 5400, 8400. Whole calls in us, narrow /
// single / pair: 512 x 512 103 / 124 / 162, 1024 x 1024 147 / 163 / 202, 3 x 777 x
// 1333 220 / 213 / 238, 2048 x 2048 471 / 314 / 298, 8 x 1024 x 2048 732 / 470 / 394.
int pick_shape(const latentmoe_muon* h) {
  if (h->pairs != 2)
    return h->pairs == 0 ? lmoe::kNsSingle : h->pairs == 1 ? lmoe::kNsPair : lmoe::kNsNarrow;
  const NsArgs& a = h->args;
  const auto cost = [&](int shape, long long units, long long block, long long hand_over) {
    const long long sym = (sym_tiles(h->side, shape) * h->batch + units - 1) / units;
    const int split = gram_split(h->batch, h->side, a.k_gram, h->sms, shape);
    const long long gram = (a.k_gram + split - 1) / split + (split > 1 ? kJoinBlocks : 0);
    const long long app = (tiles(h->rows, h->cols, shape) * h->batch + units - 1) / units;
    return (sym * (gram + a.k_side) + app * a.k_side) * block + 3 * hand_over;
  };
  const long long narrow = cost(lmoe::kNsNarrow, h->sms, 270, 4200);
  const long long single = cost(lmoe::kNsSingle, h->sms, 320, 5400);
  const long long pair =
      h->sms >= 2 ? cost(lmoe::kNsPair, h->sms / 2, 310, 8400) : single + narrow;
  if (pair < single && pair < narrow) return lmoe::kNsPair;
  return narrow < single ? lmoe::kNsNarrow : lmoe::kNsSingle;
}

// The whole iteration on U; the last product writes `out` as out_mode says.
int iterate(latentmoe_muon* h, const lmoe::NsUpdate& u, int out_mode, void* out, float keep,
            float move, cudaStream_t s) {
  const lmoe::PdlScope pdl(true);
  const long long n = h->rows * h->cols;
  NsArgs& a = h->args;
  if (h->small_ctas > 0 && h->pairs == 2) {
    lmoe::NsSmallArgs t;
    memset(&t, 0, sizeof(t));
    t.g = u.g;
    t.momentum = u.momentum;
    t.g_f32 = u.g_f32 ? 1 : 0;
    t.mu = u.mu;
    t.nesterov = u.nesterov ? 1 : 0;
    t.rows = a.rows;
    t.cols = a.cols;
    t.tall = a.tall;
    t.m = a.side;
    t.n = static_cast<int>(h->tall ? h->rows : h->cols);
    t.width = h->small_width;
    t.ctas = h->small_ctas;
    t.steps = a.steps;
    t.eps = h->eps;
    t.scale0 = h->scale0;
    t.out_mode = out_mode;
    t.out = out;
    t.keep = keep;
    t.move = move;
    t.status = a.status;
    memcpy(t.step, a.step, sizeof(t.step));
    NS_CK(h, lmoe::launch_ns_small(t, h->batch, s));
    h->launches += 1;
    return LATENTMOE_OK;
  }
  NS_CK(h, lmoe::launch_ns_norm(u, h->batch, n, h->chunks, h->chunk, h->eps, h->partial, s));
  NS_CK(h, lmoe::launch_ns_init(u, h->batch, h->rows, h->cols, a.ld_x, h->chunks, h->partial,
                                h->eps, h->scale0, h->x32, h->x16, a.done, a.done_ld, a.counter, s));
  h->launches += 2;
  const int shape = pick_shape(h);
  const long long bm = lmoe::ns_bm(shape);
  a.sym_tiles = static_cast<int>(sym_tiles(h->side, shape));
  a.m_tiles = static_cast<int>((h->rows + bm - 1) / bm);
  a.apply_tiles = static_cast<int>(tiles(h->rows, h->cols, shape));
  const long long cut = apply_cut(h->side);
  a.cut = static_cast<int>(cut);
  a.lower = static_cast<int>(cut == h->side ? a.apply_tiles
                             : h->tall      ? cut / lmoe::ns_bn(shape) * a.m_tiles
                                            : cut / bm * (a.apply_tiles / a.m_tiles));
  a.split = gram_split(h->batch, h->side, a.k_gram, h->sms, shape);
  a.group = h->group;
  a.out_mode = out_mode;
  a.out = out;
  a.keep = keep;
  a.move = move;
  NS_CK(h, lmoe::launch_ns_iterate(shape, h->maps, a, h->sms, s));
  h->launches += 1;
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
  if (d.rows > kMaxSide || d.cols > kMaxSide || d.batch > 65535 || d.steps > kNsMaxSteps)
    return LATENTMOE_ERR_UNSUPPORTED;
  lmoe::NsStep step[kNsMaxSteps];
  memset(step, 0, sizeof(step));
  // bound on the spectral norm of X before the step: 1 after the division by
  // the Frobenius norm, then the largest value of |a s + b s^3 + c s^5| on
  // [0, bound], each a little more for rounding (the scales leave a factor of
  // 4; a wide margin here would leave the interval that the usual coefficients
  // keep to, and grow)
  double u = 1.001;
  float scale0 = 1.0f;
  for (int i = 0; i < d.steps; ++i) {
    const float ca = d.coefs ? d.coefs[3 * i] : 3.4445f;
    const float cb = d.coefs ? d.coefs[3 * i + 1] : -4.7750f;
    const float cc = d.coefs ? d.coefs[3 * i + 2] : 2.0315f;
    if (!isfinite(ca) || !isfinite(cb) || !isfinite(cc)) return LATENTMOE_ERR_INVALID_ARG;
    // the scales come from the largest possible singular value: directions far
    // below it, whose A^2 underflows, are right only through their a X
    if (!(fabsf(ca) * 64.0f >= fabsf(cb) + fabsf(cc))) return LATENTMOE_ERR_INVALID_ARG;
    double next = 0.0, poly = 0.0;
    for (int j = 0; j <= 1024; ++j) {
      const double x = u * j / 1024.0, x2 = x * x;
      const double p = cb * x2 + cc * x2 * x2;
      poly = fmax(poly, fabs(p));
      next = fmax(next, fabs((ca + p) * x));
    }
    const float sx = pow2_scale(u), sa = pow2_scale(u * u), sp = pow2_scale(poly);
    lmoe::NsStep& f = step[i];
    f.gram_diag = 1.0f / sx / sx;
    f.gram_off = sa * f.gram_diag;
    f.poly_b = cb * (sp / sa);
    f.poly_c = cc * (sp / sa);
    f.poly_acc = f.poly_c / sa;
    f.diag_acc = cc / sa / sa;
    f.b = cb;
    f.c = cc;
    f.s_p = sp;
    f.d_x = 1.0f / sx;
    if (i == 0) scale0 = sx;
    else step[i - 1].d_x *= sx;  // the step before leaves X with this step's scale
    u = 1.002 * next;
    if (!(u < 1e6)) return LATENTMOE_ERR_INVALID_ARG;  // the coefficients diverge
    if (u < 1e-6) u = 1e-6;
  }
  for (int i = 0; i < d.steps; ++i) {
    step[i].a_x = (d.coefs ? d.coefs[3 * i] : 3.4445f) * step[i].d_x;
    step[i].apply_acc = step[i].d_x / step[i].s_p;
  }
  const long long B = d.batch, R = d.rows, C = d.cols;
  const long long side = R < C ? R : C;
  const long long ldx = (C + 7) / 8 * 8, lda = (side + 7) / 8 * 8;
  // positions in the tile sequence stay in int
  if ((2 * sym_tiles(side, lmoe::kNsNarrow) + tiles(R, C, lmoe::kNsNarrow)) * B * d.steps >
      (1ll << 30))
    return LATENTMOE_ERR_UNSUPPORTED;

  latentmoe_muon* h = new (std::nothrow) latentmoe_muon();
  if (h == nullptr) return LATENTMOE_ERR_OUT_OF_MEMORY;
  h->batch = B;
  h->rows = R;
  h->cols = C;
  h->side = side;
  h->tall = R > C;
  h->steps = static_cast<int>(d.steps);
  h->eps = d.eps;
  h->scale0 = scale0;
  memset(&h->args, 0, sizeof(h->args));
  NsArgs& a = h->args;
  a.batch = static_cast<int>(B);
  a.rows = static_cast<int>(R);
  a.cols = static_cast<int>(C);
  a.side = static_cast<int>(side);
  a.tall = h->tall ? 1 : 0;
  a.steps = h->steps;
  a.k_gram = static_cast<int>(((R > C ? R : C) + lmoe::kNsBK - 1) / lmoe::kNsBK);
  a.k_side = static_cast<int>((side + lmoe::kNsBK - 1) / lmoe::kNsBK);
  a.ld_x = ldx;
  a.ld_a = lda;
  memcpy(a.step, step, sizeof(step));
  // matrices in flight: what stays in L2
  const long long bytes = 8 * R * ldx + 4 * side * lda;
  long long group = kGroupBytes / bytes;
  h->group = static_cast<int>(group < 1 ? 1 : group > B ? B : group);
  // blocks of the norm pass: 16 elements a thread or more, whole vectors
  const long long n = R * C;
  const long long unit = 8ll * lmoe::kNsNormThreads;
  long long chunk = 2 * unit;
  const long long need = (n + lmoe::kNsMaxChunks - 1) / lmoe::kNsMaxChunks;
  if (chunk < need) chunk = (need + unit - 1) / unit * unit;
  h->chunk = chunk;
  h->chunks = static_cast<int>((n + chunk - 1) / chunk);

  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = lmoe::ns_small_plan(B, R, C, &h->small_ctas, &h->small_width);
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
  const size_t o_da = take(static_cast<size_t>(B) * lda * 4);
  const size_t o_dp = take(static_cast<size_t>(B) * lda * 4);
  // the parts of a split gram product, in either shape that may be asked for
  size_t parts = 0;
  a.done_ld = 4 * h->steps;
  for (int shape : {lmoe::kNsSingle, lmoe::kNsNarrow}) {
    const long long split = gram_split(B, side, a.k_gram, h->sms, shape);
    if (split == 1) continue;
    const long long n_tiles = sym_tiles(side, shape);
    const size_t need = static_cast<size_t>(B * n_tiles * split) * lmoe::ns_bm(shape) *
                        lmoe::ns_bn(shape) * 4;
    if (need > parts) parts = need;
    const long long ld = 4 * h->steps + n_tiles * lmoe::kNsEpiWarps;
    if (ld > a.done_ld) a.done_ld = static_cast<int>(ld);
  }
  const size_t o_parts = take(parts);
  const size_t o_done = take(static_cast<size_t>(B) * a.done_ld * 4), o_counter = take(16);
  const size_t o_partial = take(static_cast<size_t>(B) * h->chunks * 8), o_status = take(16);
  e = cudaMalloc(&h->ws, off);
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return e == cudaErrorMemoryAllocation ? LATENTMOE_ERR_OUT_OF_MEMORY : LATENTMOE_ERR_CUDA;
  }
  char* base = static_cast<char*>(h->ws);
  h->x32 = reinterpret_cast<float*>(base + o_x32);
  h->x16 = reinterpret_cast<__half*>(base + o_x0);
  void* x1 = base + o_x1;
  void* gram = base + o_gram;
  void* poly = base + o_poly;
  a.diag_a = reinterpret_cast<float*>(base + o_da);
  a.diag_p = reinterpret_cast<float*>(base + o_dp);
  a.parts = reinterpret_cast<float*>(base + o_parts);
  a.done = reinterpret_cast<int*>(base + o_done);
  a.counter = reinterpret_cast<int*>(base + o_counter);
  a.status = reinterpret_cast<unsigned*>(base + o_status);
  h->partial = reinterpret_cast<float*>(base + o_partial);
  e = cudaMemset(a.status, 0, 16);
  lmoe::NsMaps& t = h->maps;
  if (e != cudaSuccess || !make_ns_map(&t.x[0], h->x16, B, R, C, ldx, 64) ||
      !make_ns_map(&t.x[1], x1, B, R, C, ldx, 64) ||
      !make_ns_map(&t.gram, gram, B, side, side, lda, 64) ||
      !make_ns_map(&t.poly, poly, B, side, side, lda, 64) ||
      !make_ns_map(&t.chunk_h[0], h->x16, B, R, C, ldx, 32) ||
      !make_ns_map(&t.chunk_h[1], x1, B, R, C, ldx, 32) ||
      !make_ns_map(&t.chunk_x, h->x32, B, R, C, ldx, 32, true) ||
      !make_ns_map(&t.chunk_gram, gram, B, side, side, lda, 32) ||
      !make_ns_map(&t.chunk_poly, poly, B, side, side, lda, 32)) {
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
  if (h == nullptr || mode < 0 || mode > 3) return LATENTMOE_ERR_INVALID_ARG;
  h->pairs = mode;
  return LATENTMOE_OK;
}

int latentmoe_muon_get_status(latentmoe_muon_t h, uint32_t* device_status) {
  if (h == nullptr || device_status == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  NS_CK(h, cudaSetDevice(h->device));
  NS_CK(h, cudaDeviceSynchronize());
  unsigned v = 0;
  NS_CK(h, cudaMemcpy(&v, h->args.status, 4, cudaMemcpyDeviceToHost));
  NS_CK(h, cudaMemset(h->args.status, 0, 4));
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

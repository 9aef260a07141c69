// C ABI of the gated feed-forward block (declared in include/latentmoe.h): handle,
// workspace, tensor maps, launches.
//
// The block is the shared expert of "MAI-Base-2: Microsoft's 2.8T base model, and
// whether its compute numbers add up", section "The model", as an operator on the
// caller's own weights, with the gradient that the layer's forward lacks.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "ffn.h"
#include "kernels.h"
#include "latentmoe.h"
#include "tensor_map.h"

using lmoe::FfnArgs;
using lmoe::FfnProduct;

struct latentmoe_ffn {
  long long d = 0, F = 0, max_tokens = 0;
  bool training = false;
  int device = 0;
  int sms = 1;
  int mode = 2;  // 0 single, 1 pair, 2 by the expected time, 3 the kernel for few tokens
  void* ws = nullptr;
  __nv_bfloat16* h = nullptr;   // [max_tokens, F]
  __nv_bfloat16* dg = nullptr;  // training only
  __nv_bfloat16* du = nullptr;
  __nv_bfloat16* xs = nullptr;  // [8, d]: x and dy of fewer tokens than that
  __nv_bfloat16* dys = nullptr;
  unsigned* status = nullptr;
  float* parts = nullptr;   // of the kernel for few tokens
  int* arrived = nullptr;
  size_t arrived_bytes = 0;
  int* counter = nullptr;   // of the plain products' tiles
  int64_t launches = 0;
  int last_cuda = 0;
};

namespace {

constexpr long long kMaxWidth = 65536;
constexpr long long kMaxTokens = 1ll << 22;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int fail(latentmoe_ffn* h, cudaError_t e) {
  h->last_cuda = static_cast<int>(e);
  return e == cudaErrorMemoryAllocation ? LATENTMOE_ERR_OUT_OF_MEMORY : LATENTMOE_ERR_CUDA;
}

#define FFN_CK(h, call)                         \
  do {                                          \
    const cudaError_t e_ = (call);              \
    if (e_ != cudaSuccess) return fail(h, e_);  \
  } while (0)

// 2-D map of a row-major matrix [rows, cols] with row stride ld (elements).
bool encode(CUtensorMap* map, const void* p, long long rows, long long cols, long long ld, int box,
            int box_rows, bool f32) {
  const lmoe::EncodeTiledFn fn = lmoe::tensor_map_encoder();
  if (fn == nullptr) return false;
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * size};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box),
                               static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(p), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix in memory.
struct Mat {
  const void* p;
  long long rows, cols, ld;
};
bool operand(CUtensorMap* map, const Mat& m) {
  return encode(map, m.p, m.rows, m.cols, m.ld, 64, 64, false);
}
bool chunk(CUtensorMap* map, const Mat& m, bool f32 = false) {
  return encode(map, m.p, m.rows, m.cols, m.ld, 32, 32, f32);
}

// Collects a launch's products; `ok` turns false where a map cannot be made.
struct Launch {
  FfnArgs a;
  bool ok = true;
  explicit Launch(const latentmoe_ffn* h) {
    memset(&a, 0, sizeof(a));
    a.status = h->status;
    a.counter = h->counter;
  }
  // D [M, N] = A B^T over K: a_mn / b_mn say that the operand lies as [K, M] / [K, N].
  FfnProduct& add(const Mat& A, bool a_mn, const Mat& B, bool b_mn, long long M, long long N,
                  long long K) {
    FfnProduct& p = a.p[a.products++];
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.k_blocks = static_cast<int>((K + lmoe::kFfnBK - 1) / lmoe::kFfnBK);
    p.segments = 1;
    p.a_mn = a_mn;
    p.b_mn = b_mn;
    p.save = 0;
    p.out_mode = lmoe::kFfnBf16;
    ok = ok && operand(&p.a[0], A) && operand(&p.b[0], B);
    return p;
  }
};

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Tiles for a shape, in the order of the products; the expected time of the launch in
// ns: whole rounds for one product, else the work spread evenly and half of the longest
// tile for the end. A k-block takes 320 (single) or 310 (pair; measured for the
// Newton-Schulz products, whose main loop is the same: single tiles are bound by the 64
// bytes a clock that an SM takes in), a tile at least its epilogue, and the last tile's
// epilogue is seen in full. us, single / pair: 128 x 256 x 256 forward 9.3 / 12.3, backward 12.9 /
// 18.5; 1024 x 1024 x 1024 forward 16.4 / 19.5; 300 x 4096 x 4096 dx 64.5 / 76, forward 67 / 55;
// 777 x 1336 x 2040 forward 42 / 33; 4096 x 2048 x 2048 113 / 77.
double plan(FfnArgs& a, int epi, int shape, int sms) {
  const bool pair = shape == lmoe::kFfnPair;
  const int cols = epi == lmoe::kFfnGateUp ? lmoe::ffn_bn(shape) / 2 : lmoe::ffn_bn(shape);
  const long long units = pair ? sms / 2 : sms;
  const double block = pair ? 310.0 : 320.0, least = pair ? 1850.0 : 1300.0;
  const double end = !pair ? 0.0 : epi == lmoe::kFfnDGate ? 4000.0 : 1500.0;
  long long tiles = 0;
  double work = 0.0, longest = 0.0;
  for (int i = 0; i < a.products; ++i) {
    FfnProduct& p = a.p[i];
    p.first = static_cast<int>(tiles);
    p.m_tiles = static_cast<int>(ceil_div(p.M, lmoe::ffn_bm(shape)));
    p.n_tiles = static_cast<int>(ceil_div(p.N, cols));
    const long long n = static_cast<long long>(p.m_tiles) * p.n_tiles;
    double one = block * p.k_blocks * p.segments;
    if (one < least) one = least;
    tiles += n;
    work += n * one;
    if (one > longest) longest = one;
  }
  a.tiles = static_cast<int>(tiles);
  a.band = pair ? 8 : 16;
  if (units < 1) return 1e30;
  if (a.products == 1) return ceil_div(tiles, units) * longest + end;
  const double even = work / units + (tiles > units ? 0.5 * longest : 0.0);
  return (even > longest ? even : longest) + end;
}

int run(latentmoe_ffn* h, Launch& l, int epi, cudaStream_t s) {
  if (!l.ok) return LATENTMOE_ERR_CUDA;
  const lmoe::PdlScope pdl(true);
  int shape = h->mode;
  if (shape > lmoe::kFfnPair) {
    const double single = plan(l.a, epi, lmoe::kFfnSingle, h->sms);
    const double pair = plan(l.a, epi, lmoe::kFfnPair, h->sms);
    shape = pair <= single ? lmoe::kFfnPair : lmoe::kFfnSingle;
  }
  plan(l.a, epi, shape, h->sms);
  FFN_CK(h, lmoe::launch_ffn(epi, shape, l.a, h->sms, s));
  h->launches += 1;
  return LATENTMOE_OK;
}

// The time of a launch of one product in ns, on whichever tiles take less: whole rounds
// of tiles, each its k-blocks.
double tile_time(long long M, long long N, long long K, int epi, int sms) {
  FfnArgs a;
  memset(&a, 0, sizeof(a));
  a.products = 1;
  a.p[0].M = static_cast<int>(M);
  a.p[0].N = static_cast<int>(N);
  a.p[0].k_blocks = static_cast<int>(ceil_div(K, lmoe::kFfnBK));
  a.p[0].segments = 1;
  const double single = plan(a, epi, lmoe::kFfnSingle, sms);
  const double pair = plan(a, epi, lmoe::kFfnPair, sms);
  return single < pair ? single : pair;
}

// Whether the forward of T tokens takes the kernel for few: the weights at 6.2 TB/s, and
// 0.25 us a token for the parts' way through memory, against whole rounds of tiles. In us,
// few / tiles: 8704 x 10240 1 token 89 / 451, 27 tokens 97 / 152, 128 tokens 128 / 154;
// 4096 x 2048 16 tokens 20 / 39, 64 tokens 34 / 36, 96 tokens 44 / 36; 2048 x 2048 48 tokens
// 23 / 26, 96 tokens 34 / 26.
bool few_wins(const latentmoe_ffn* h, long long T) {
  if (T > lmoe::kFewMost) return false;
  if (T < lmoe::kFfnLeastRows) return true;  // tiles are slow with operands of few rows
  const double few = 6.0 * h->d * h->F / 6200.0 + 250.0 * T;
  const double tiles = tile_time(T, h->F, h->d, lmoe::kFfnGateUp, h->sms) +
                       tile_time(T, h->d, h->F, lmoe::kFfnPlain, h->sms);
  return few < tiles;
}

// Whether the gradient of T tokens takes it for dgate and dx (dW then goes alone): up to 24
// tokens, for weights that take longer to read than the launch that it adds. us, few /
// tiles, with dx alone and with everything: 8704 x 10240 8 tokens 93 / 137 and 214 / 235, 64
// tokens 120 / 140 and 262 / 236; 4096 x 2048 16 tokens 28 / 53 and 44 / 61, 32 tokens 38 / 44
// and 60 / 50; 2048 x 2048 17 tokens 25 / 34 and 35 / 39, 32 tokens 30 / 34 and 42 / 35; 1024 x
// 1024 8 tokens 14 / 20 and 20 / 21; 256 x 256 8 tokens 11 / 12 and 15 / 12.
bool dgate_few_wins(const latentmoe_ffn* h, long long T) {
  return T <= 24 && h->d * h->F >= (1ll << 21);
}

// What the products for few tokens have in common; x is their one operand or first one.
bool few_args(lmoe::FewArgs* a, const latentmoe_ffn* h, int epi, const Mat& x, long long rows,
              long long k_blocks) {
  memset(a, 0, sizeof(*a));
  a->tokens = static_cast<int>(x.rows);
  a->rows = static_cast<int>(rows);
  a->tiles = static_cast<int>(ceil_div(rows, epi == lmoe::kFfnGateUp ? 64 : 128));
  a->k_blocks = static_cast<int>(k_blocks);
  a->cut = a->k_blocks;
  a->parts = h->parts;
  a->arrived = h->arrived;
  a->status = h->status;
  return encode(&a->x[0], x.p, x.rows, x.cols, x.ld, 64, lmoe::few_tokens(a->tokens), false);
}

int run_few(latentmoe_ffn* h, int epi, bool transposed, const lmoe::FewArgs& a, cudaStream_t s) {
  const lmoe::PdlScope pdl(true);
  FFN_CK(h, lmoe::launch_ffn_few(epi, transposed, a, h->sms, s));
  h->launches += 1;
  return LATENTMOE_OK;
}

// The forward for few tokens.
int forward_few(latentmoe_ffn* h, const latentmoe_ffn_weights* w, const Mat& x, void* y,
                long long ld_y, void* gate, void* up, cudaStream_t s) {
  const long long d = h->d, F = h->F, T = x.rows;
  lmoe::FewArgs a;
  if (!few_args(&a, h, lmoe::kFfnGateUp, x, F, ceil_div(d, lmoe::kFfnBK)) ||
      !operand(&a.w[0], {w->w_g, F, d, d}) || !operand(&a.w[1], {w->w_u, F, d, d}))
    return LATENTMOE_ERR_CUDA;
  a.out = h->h;
  a.ld = F;
  a.gate = static_cast<__nv_bfloat16*>(gate);
  a.up = static_cast<__nv_bfloat16*>(up);
  const int rc = run_few(h, lmoe::kFfnGateUp, false, a, s);
  if (rc != LATENTMOE_OK) return rc;
  if (!few_args(&a, h, lmoe::kFfnPlain, {h->h, T, F, F}, d, ceil_div(F, lmoe::kFfnBK)) ||
      !operand(&a.w[0], {w->w_d, d, F, F}))
    return LATENTMOE_ERR_CUDA;
  a.early = 1;
  a.out = static_cast<__nv_bfloat16*>(y);
  a.ld = ld_y;
  return run_few(h, lmoe::kFfnPlain, false, a, s);
}

// dg, du and h for few tokens.
int dgate_few(latentmoe_ffn* h, const void* w_d, const Mat& dy, const void* gate, const void* up,
              cudaStream_t s) {
  const long long d = h->d, F = h->F;
  lmoe::FewArgs a;
  if (!few_args(&a, h, lmoe::kFfnDGate, dy, F, ceil_div(d, lmoe::kFfnBK)) ||
      !operand(&a.w[0], {w_d, d, F, F}))
    return LATENTMOE_ERR_CUDA;
  a.out = h->dg;
  a.du = h->du;
  a.h = h->h;
  a.ld = F;
  a.gate = static_cast<__nv_bfloat16*>(const_cast<void*>(gate));
  a.up = static_cast<__nv_bfloat16*>(const_cast<void*>(up));
  return run_few(h, lmoe::kFfnDGate, true, a, s);
}

// dx for few tokens, after the launch that leaves dg and du.
int dx_few(latentmoe_ffn* h, const latentmoe_ffn_weights* w, long long T, void* dx, long long ld_dx,
           cudaStream_t s) {
  const long long d = h->d, F = h->F, blocks = ceil_div(F, lmoe::kFfnBK);
  lmoe::FewArgs a;
  if (!few_args(&a, h, lmoe::kFfnPlain, {h->dg, T, F, F}, d, 2 * blocks) ||
      !encode(&a.x[1], h->du, T, F, F, 64, lmoe::few_tokens(static_cast<int>(T)), false) ||
      !operand(&a.w[0], {w->w_g, F, d, d}) || !operand(&a.w[1], {w->w_u, F, d, d}))
    return LATENTMOE_ERR_CUDA;
  a.cut = static_cast<int>(blocks);
  a.early = 1;
  a.out = static_cast<__nv_bfloat16*>(dx);
  a.ld = ld_dx;
  return run_few(h, lmoe::kFfnPlain, true, a, s);
}

bool stride(int64_t* ld, int64_t width) {
  if (*ld == 0) *ld = width;
  return *ld >= width;
}

}  // namespace

extern "C" {

int latentmoe_ffn_create(const latentmoe_ffn_dims* dims, latentmoe_ffn_t* out) {
  if (out == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (dims == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  const latentmoe_ffn_dims p = *dims;
  if (p.hidden < 1 || p.ffn < 1 || p.max_tokens < 1) return LATENTMOE_ERR_INVALID_ARG;
  if (p.hidden % 8 != 0 || p.ffn % 8 != 0 || p.hidden > kMaxWidth || p.ffn > kMaxWidth ||
      p.max_tokens > kMaxTokens)
    return LATENTMOE_ERR_UNSUPPORTED;
  latentmoe_ffn* h = new (std::nothrow) latentmoe_ffn();
  if (h == nullptr) return LATENTMOE_ERR_OUT_OF_MEMORY;
  h->d = p.hidden;
  h->F = p.ffn;
  h->max_tokens = p.max_tokens;
  h->training = p.training != 0;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    delete h;
    return LATENTMOE_ERR_CUDA;
  }
  const long long most = p.max_tokens < lmoe::kFfnLeastRows ? lmoe::kFfnLeastRows : p.max_tokens;
  const size_t rows = (static_cast<size_t>(most) * p.ffn * 2 + 1023) / 1024 * 1024;
  const size_t pad = (static_cast<size_t>(lmoe::kFfnLeastRows) * p.hidden * 2 + 1023) / 1024 * 1024;
  const long long few = p.max_tokens < lmoe::kFewMost ? p.max_tokens : lmoe::kFewMost;
  const size_t parts = static_cast<size_t>(h->sms) * 2 * 128 * 4 *
                       static_cast<size_t>(lmoe::few_tokens(static_cast<int>(few)));
  const long long tiles = ceil_div(p.ffn, 64) > ceil_div(p.hidden, 128) ? ceil_div(p.ffn, 64)
                                                                        : ceil_div(p.hidden, 128);
  // status word and arrival counts, parts, h (dg, du)
  h->arrived_bytes = static_cast<size_t>(tiles) * 4;
  const size_t head = (1024 + h->arrived_bytes + 1023) / 1024 * 1024;
  const size_t bytes = head + parts + (h->training ? 3 * rows + 2 * pad : rows);
  e = cudaMalloc(&h->ws, bytes);
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return e == cudaErrorMemoryAllocation ? LATENTMOE_ERR_OUT_OF_MEMORY : LATENTMOE_ERR_CUDA;
  }
  char* base = static_cast<char*>(h->ws);
  h->status = reinterpret_cast<unsigned*>(base);
  h->counter = reinterpret_cast<int*>(base + 512);
  h->arrived = reinterpret_cast<int*>(base + 1024);
  h->parts = reinterpret_cast<float*>(base + head);
  base += head + parts;
  h->h = reinterpret_cast<__nv_bfloat16*>(base);
  if (h->training) {
    h->dg = reinterpret_cast<__nv_bfloat16*>(base + rows);
    h->du = reinterpret_cast<__nv_bfloat16*>(base + 2 * rows);
    h->xs = reinterpret_cast<__nv_bfloat16*>(base + 3 * rows);
    h->dys = reinterpret_cast<__nv_bfloat16*>(base + 3 * rows + pad);
  }
  e = cudaMemset(h->status, 0, head);
  if (e != cudaSuccess) {
    cudaFree(h->ws);
    delete h;
    return LATENTMOE_ERR_CUDA;
  }
  *out = h;
  return LATENTMOE_OK;
}

int latentmoe_ffn_destroy(latentmoe_ffn_t h) {
  if (h == nullptr) return LATENTMOE_OK;
  if (h->ws) cudaFree(h->ws);
  delete h;
  return LATENTMOE_OK;
}

int latentmoe_ffn_forward(latentmoe_ffn_t h, const latentmoe_ffn_weights* w, const void* x,
                          int64_t ld_x, void* y, int64_t ld_y, void* gate, void* up, int64_t T,
                          latentmoe_stream_t st) {
  if (h == nullptr || w == nullptr || x == nullptr || y == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  if (w->w_g == nullptr || w->w_u == nullptr || w->w_d == nullptr)
    return LATENTMOE_ERR_INVALID_ARG;
  if ((gate == nullptr) != (up == nullptr) || T < 1 || T > h->max_tokens)
    return LATENTMOE_ERR_INVALID_ARG;
  if (!stride(&ld_x, h->d) || !stride(&ld_y, h->d)) return LATENTMOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(w->w_g) || !aligned16(w->w_u) ||
      !aligned16(w->w_d) || !aligned16(gate) || !aligned16(up) || ld_x % 8 != 0 || ld_y % 8 != 0)
    return LATENTMOE_ERR_UNSUPPORTED;
  FFN_CK(h, cudaSetDevice(h->device));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
  const long long d = h->d, F = h->F;
  if (h->mode == 3 ? T <= lmoe::kFewMost : h->mode == 2 && few_wins(h, T)) {
    return forward_few(h, w, {x, T, d, ld_x}, y, ld_y, gate, up, s);
  }
  Launch l(h);
  FfnProduct& p = l.add({x, T, d, ld_x}, false, {w->w_g, F, d, d}, false, T, F, d);
  l.ok = l.ok && operand(&p.b[1], {w->w_u, F, d, d}) && chunk(&p.out[0], {h->h, T, F, F});
  if (gate != nullptr) {
    p.save = 1;
    l.ok = l.ok && chunk(&p.out[1], {gate, T, F, F}) && chunk(&p.out[2], {up, T, F, F});
  }
  const int rc = run(h, l, lmoe::kFfnGateUp, s);
  if (rc != LATENTMOE_OK) return rc;
  Launch m(h);
  FfnProduct& q = m.add({h->h, T, F, F}, false, {w->w_d, d, F, F}, false, T, d, F);
  m.ok = m.ok && chunk(&q.out[0], {y, T, d, ld_y});
  return run(h, m, lmoe::kFfnPlain, s);
}

int latentmoe_ffn_backward(latentmoe_ffn_t h, const latentmoe_ffn_weights* w,
                           const latentmoe_ffn_grad* grad, int64_t T, latentmoe_stream_t st) {
  if (h == nullptr || w == nullptr || grad == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  latentmoe_ffn_grad g = *grad;
  if (w->w_d == nullptr || g.dy == nullptr || g.gate == nullptr || g.up == nullptr)
    return LATENTMOE_ERR_INVALID_ARG;
  if (g.dx == nullptr && g.dw_g == nullptr && g.dw_u == nullptr && g.dw_d == nullptr)
    return LATENTMOE_ERR_INVALID_ARG;
  if (g.dx != nullptr && (w->w_g == nullptr || w->w_u == nullptr)) return LATENTMOE_ERR_INVALID_ARG;
  if ((g.dw_g != nullptr || g.dw_u != nullptr) && g.x == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  if (g.dw_dtype != LATENTMOE_BF16 && g.dw_dtype != LATENTMOE_FP32)
    return LATENTMOE_ERR_INVALID_ARG;
  if (g.accumulate != 0 && g.dw_dtype != LATENTMOE_FP32) return LATENTMOE_ERR_UNSUPPORTED;
  if (T < 1 || T > h->max_tokens || !h->training) return LATENTMOE_ERR_INVALID_ARG;
  if (!stride(&g.ld_dy, h->d) || !stride(&g.ld_x, h->d) || !stride(&g.ld_dx, h->d))
    return LATENTMOE_ERR_INVALID_ARG;
  if (!aligned16(g.dy) || !aligned16(g.x) || !aligned16(g.gate) || !aligned16(g.up) ||
      !aligned16(g.dx) || !aligned16(g.dw_g) || !aligned16(g.dw_u) || !aligned16(g.dw_d) ||
      !aligned16(w->w_g) || !aligned16(w->w_u) || !aligned16(w->w_d) || g.ld_dy % 8 != 0 ||
      g.ld_x % 8 != 0 || g.ld_dx % 8 != 0)
    return LATENTMOE_ERR_UNSUPPORTED;
  FFN_CK(h, cudaSetDevice(h->device));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
  const long long d = h->d, F = h->F;
  // rows of the operands: those past T are zeros
  const long long R = T < lmoe::kFfnLeastRows ? lmoe::kFfnLeastRows : T;
  Mat dy = {g.dy, T, d, g.ld_dy}, x = {g.x, T, d, g.ld_x};
  if (R > T) {
    const lmoe::PdlScope pdl(true);
    FFN_CK(h, lmoe::launch_ffn_pad(static_cast<const __nv_bfloat16*>(g.x), g.ld_x,
                                   static_cast<const __nv_bfloat16*>(g.dy), g.ld_dy,
                                   static_cast<int>(T), static_cast<int>(d), static_cast<int>(F),
                                   h->xs, h->dys, h->h, h->dg, h->du, s));
    h->launches += 1;
    dy = {h->dys, R, d, d};
    x = {h->xs, R, d, d};
  }
  const Mat hm = {h->h, R, F, F}, dg = {h->dg, R, F, F}, du = {h->du, R, F, F};
  const bool few = h->mode == 3 ? T <= lmoe::kFewMost : h->mode == 2 && dgate_few_wins(h, T);
  int rc;
  if (few) {
    rc = dgate_few(h, w->w_d, {dy.p, T, d, dy.ld}, g.gate, g.up, s);
  } else {
    Launch l(h);
    FfnProduct& p = l.add(dy, false, {w->w_d, d, F, F}, true, T, F, d);
    l.ok = l.ok && chunk(&l.a.gate, {g.gate, T, F, F}) && chunk(&l.a.up, {g.up, T, F, F}) &&
           chunk(&p.out[0], {h->dg, T, F, F}) && chunk(&p.out[1], {h->du, T, F, F}) &&
           chunk(&p.out[2], {h->h, T, F, F});
    rc = run(h, l, lmoe::kFfnDGate, s);
  }
  if (rc != LATENTMOE_OK) return rc;
  const bool dx_apart = g.dx != nullptr && few;
  if (dx_apart) {
    rc = dx_few(h, w, T, g.dx, g.ld_dx, s);
    if (rc != LATENTMOE_OK || (g.dw_g == nullptr && g.dw_u == nullptr && g.dw_d == nullptr))
      return rc;
  }
  Launch m(h);
  const bool f32 = g.dw_dtype == LATENTMOE_FP32;
  const int out_mode = !f32             ? lmoe::kFfnBf16
                       : g.accumulate ? lmoe::kFfnF32Add
                                      : lmoe::kFfnF32;
  auto add_dx = [&]() {
    if (g.dx == nullptr || dx_apart) return;
    FfnProduct& q = m.add(dg, false, {w->w_g, F, d, d}, true, T, d, F);
    q.segments = 2;
    m.ok = m.ok && operand(&q.a[1], du) && operand(&q.b[1], {w->w_u, F, d, d}) &&
           chunk(&q.out[0], {g.dx, T, d, g.ld_dx});
  };
  // the longest tiles first
  const bool dx_first = 2 * F > T;
  if (dx_first) add_dx();
  auto add_dw = [&](const Mat& A, const Mat& B, void* to) {
    if (to == nullptr) return;
    FfnProduct& q = m.add(A, true, B, true, A.cols, B.cols, T);
    q.out_mode = out_mode;
    m.ok = m.ok && chunk(&q.out[0], {to, A.cols, B.cols, B.cols}, f32);
  };
  add_dw(dg, x, g.dw_g);
  add_dw(du, x, g.dw_u);
  add_dw(dy, hm, g.dw_d);
  if (!dx_first) add_dx();
  return run(h, m, lmoe::kFfnPlain, s);
}

int latentmoe_ffn_set_sm_pairs(latentmoe_ffn_t h, int mode) {
  if (h == nullptr || mode < 0 || mode > 3) return LATENTMOE_ERR_INVALID_ARG;
  h->mode = mode;
  return LATENTMOE_OK;
}

int latentmoe_ffn_get_status(latentmoe_ffn_t h, uint32_t* device_status) {
  if (h == nullptr || device_status == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  FFN_CK(h, cudaSetDevice(h->device));
  FFN_CK(h, cudaDeviceSynchronize());
  unsigned v = 0;
  FFN_CK(h, cudaMemcpy(&v, h->status, 4, cudaMemcpyDeviceToHost));
  FFN_CK(h, cudaMemset(h->status, 0, 4));
  // a launch that gave up may have left arrivals and tiles taken
  if (v != 0) {
    FFN_CK(h, cudaMemset(h->arrived, 0, h->arrived_bytes));
    FFN_CK(h, cudaMemset(h->counter, 0, 8));
  }
  *device_status = v;
  if (v & LATENTMOE_STATUS_TIMEOUT) return LATENTMOE_ERR_TIMEOUT;
  return v != 0 ? LATENTMOE_ERR_DEVICE_STATUS : LATENTMOE_OK;
}

int latentmoe_ffn_get_launch_count(latentmoe_ffn_t h, int64_t* launches) {
  if (h == nullptr || launches == nullptr) return LATENTMOE_ERR_INVALID_ARG;
  *launches = h->launches;
  return LATENTMOE_OK;
}

int latentmoe_ffn_last_cuda_error(latentmoe_ffn_t h) { return h ? h->last_cuda : 0; }

}  // extern "C"

// Launchers of the gated feed-forward block's kernels (internal interface).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lmoe {

// What the epilogue of a launch does with its products' accumulators.
enum FfnEpi : int {
  kFfnGateUp = 0,  // B: gate rows and up rows of the same features; h, gate, up
  kFfnDGate = 1,   // the accumulator is dh; reads gate and up, leaves dg, du, h
  kFfnPlain = 2    // the product, in bf16 or fp32
};
enum FfnShape : int { kFfnSingle = 0, kFfnPair = 1 };
enum FfnOut : int { kFfnBf16 = 0, kFfnF32 = 1, kFfnF32Add = 2 };

constexpr int kFfnBK = 64;
__host__ __device__ constexpr int ffn_bm(int shape) { return shape == kFfnPair ? 256 : 128; }
__host__ __device__ constexpr int ffn_bn(int shape) { return shape == kFfnPair ? 256 : 128; }

// D [M, N] = A B^T summed over `segments` pairs of operands, K each. Operand maps:
// boxes of 64 x 64 bf16, 128-byte swizzle; (columns, rows) of the matrix in memory.
// An operand is K-major (rows of M or N, columns of K) or MN-major (rows of K).
struct FfnProduct {
  CUtensorMap a[2], b[2];
  CUtensorMap out[3];  // boxes of 32 x 32: plain: [0]; gate+up: h, gate, up; dgate: dg, du, h
  int M, N;            // gate+up: N output features
  int k_blocks;        // of a segment
  int segments;
  int a_mn, b_mn;
  int m_tiles, n_tiles;
  int first;           // first tile in the launch's sequence
  int out_mode;        // FfnOut
  int save;            // gate+up: gate and up are stored
};
constexpr int kFfnProducts = 4;
struct FfnArgs {
  FfnProduct p[kFfnProducts];
  CUtensorMap gate, up;  // dgate: boxes of 32 x 32
  int products;
  int tiles;
  int band;  // m-tiles of a band of the raster
  int* counter;  // plain: {next tile, units that have ended}, zero; left zero
  unsigned* status;
};
cudaError_t launch_ffn(int epi, int shape, const FfnArgs& a, int sms, cudaStream_t s);

// Operands of fewer than kFfnLeastRows rows, padded: a TMA load of a box of a matrix
// with fewer than 8 rows (the height of a swizzle pattern) takes several times as long
// as of one with 8, most of them outside alike. 8704 x 10240 forward on single tiles, 4
// tokens 407 us, seen as 8 rows 159; 8 tokens 158. xs, dys [8, d] = x and dy [tokens, d]
// (x null: none), rows of h, dg and du from `tokens` to 8: zeros.
constexpr int kFfnLeastRows = 8;
cudaError_t launch_ffn_pad(const __nv_bfloat16* x, long long ld_x, const __nv_bfloat16* dy,
                           long long ld_dy, int tokens, int d, int F, __nv_bfloat16* xs,
                           __nv_bfloat16* dys, __nv_bfloat16* h, __nv_bfloat16* dg,
                           __nv_bfloat16* du, cudaStream_t s);

// Few tokens: D^T = W x^T with 128 rows of W by up to 128 tokens a tile (ffn_few.cuh).
//   kFfnGateUp  W = Wg and Wu, 64 rows of each a tile: h, gate, up
//   kFfnPlain   W = Wd: y; or, from the transposes, W = Wg^T and then Wu^T with x = dg and
//               then du: dx
//   kFfnDGate   W = Wd^T, x = dy: dg, du, h
constexpr int kFewMost = 128;      // tokens
constexpr int kFewLeast = 8;       // k-blocks of a part, unless a tile has fewer
struct FewArgs {
  CUtensorMap w[2];  // boxes of 64 x 64 of the matrix in memory
  CUtensorMap x[2];  // [tokens, K]; boxes of 64 columns x few_tokens(tokens) rows
  int tokens;
  int rows;          // output features
  int tiles, k_blocks;
  int cut;           // k-blocks of w[0] and x[0] (transposed; else k_blocks)
  int early;         // weights may be loaded before the kernel ahead has finished
  float* parts;      // [CTAs, 2, few_tokens, 128]
  int* arrived;      // [tiles], zero; left zero
  __nv_bfloat16* out;   // [tokens, ld]: h, y, dx or dg
  __nv_bfloat16* du;    // kFfnDGate: [tokens, ld], and h
  __nv_bfloat16* h;
  __nv_bfloat16* gate;  // [tokens, rows]; kFfnGateUp: written, or null; kFfnDGate: read
  __nv_bfloat16* up;
  long long ld;
  unsigned* status;
};
inline int few_tokens(int tokens) {
  return tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
}
// CTAs of a launch: one an SM, fewer where parts would get too short.
int few_ctas(int tiles, int k_blocks, int sms);
// transposed: W lies as [K, rows] in memory (kFfnPlain, kFfnDGate).
cudaError_t launch_ffn_few(int epi, bool transposed, const FewArgs& a, int sms, cudaStream_t s);

}  // namespace lmoe

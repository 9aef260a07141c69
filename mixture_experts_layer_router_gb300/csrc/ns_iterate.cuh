// The whole Newton-Schulz iteration X <- a X + (b A + c A^2) X, A = X X^T
// (X wide) or X <- a X + X (b A + c A^2), A = X^T X (X tall) of a stack of
// matrices in one persistent launch on tcgen05 tensor cores. A step has three
// products ("phases"):
//
//   gram   A = X X^T or X^T X     symmetric: tiles on and below the diagonal,
//   poly   P = b A + c A A        the tiles below stored a second time, mirrored
//   apply  X' = a X + P X or a X + X P
//
// Number formats. Operands are fp16 with a power-of-two scale per kind and step
// (the host derives it from a bound on X's spectral norm, so that no entry
// overflows and entries 2^-28 below the largest possible one are still normal
// numbers), accumulators fp32. fp16 and not bf16: 11 bits against 8 at the same
// MMA rate. Two things keep 11 bits enough:
// - X lives in fp32 beside its fp16 operand copy, and a X is taken from it. The
//   small singular directions, which the iteration amplifies up to a^steps = 485
//   times, pass through the a X term alone; with X in fp16 only, the rounding of
//   the large directions drowns them (matrices of low rank plus noise: error
//   2e-2 of the result's norm; with the fp32 X 2e-4 to 9e-4).
// - A and P are fp16 off their diagonals; the diagonals, by far their largest
//   entries once X's singular values draw together, are fp32 vectors that the
//   epilogues apply (A A = A' A' + (d_i + d_j) A' + d d, with A' = A less its
//   diagonal d). That takes the error from 1.2e-3..2.0e-3 to 2e-4..7e-4. In the
//   first two steps P keeps its diagonal in fp16 (the vector holds what the
//   rounding left): there it has to cancel against the off-diagonal part in the
//   directions where P X is small (low rank: 1.2e-3..3e-3 with the whole
//   diagonal apart, 2e-4..9e-4 so).
//
// X keeps the caller's orientation. Where the contracted index is X's row
// index, X is read as an MN-major operand (TMA boxes of 64 contiguous columns x
// 64 rows, the transpose bits of the instruction descriptor), so nothing is
// transposed in memory:
//   wide: gram K-major x K-major, apply: P K-major, X MN-major
//   tall: gram MN-major x MN-major, apply: X K-major, P K-major (symmetric)
// Sizes that no tile divides need no padding: TMA fills what lies outside a
// matrix with zeros (the batch is the maps' third dimension, so a box never
// reaches into the next matrix) and the epilogue stores what lies inside.
//
// One launch instead of three a step: the tiles of all phases form one sequence
// that running CTAs take from a counter (groups of matrices; in a group: steps,
// phases, matrices, tiles), and a tile waits until every tile of its matrix's
// preceding phase has been stored (a count per matrix and phase; apply has two, for
// the rows of A below a cut, whose tiles come first, and for the others, and a gram
// tile below the cut waits for the first alone). While one matrix waits, tiles of
// the others run. Progress: tiles are taken in sequence order by running CTAs alone
// and wait only for earlier ones, so the earliest unfinished tile can always
// proceed. No buffer is overwritten early: a phase's inputs were read by phases that
// its own predecessor has waited for (gram writes A and its diagonal, which no apply
// reads; poly waits for all of gram, and with that for all of the apply before).
//
// Tiles (NsShape):
//   pair    256 x 256 on two SMs (cta_group::2, each CTA holds 128 rows of A and
//           128 of B): half the operand bytes of the others per product, for
//           products that fill the GPU
//   single  128 x 128 on one SM, 32 KB a k-block as in a pair's CTA
//   narrow  128 x 64 on one SM, for products with so few tiles that latency
//           decides: 24 KB a k-block (an SM takes in about 64 bytes a clock,
//           which is what the mainloops of single tiles are bound by) and half
//           as many results to store
// SPLIT (single and narrow): gram's k-blocks in `split` parts, each a tile of its
// own, for few tiles with a long K (a router's gradient). The parts' fp32 sums go
// to memory, and the warp that comes last for its 32 rows adds them in the order
// of the parts. 64 x 8704 253 -> 110 us, 200 x 2000 118 -> 104 us. An
// instantiation of its own: as a branch it cost the others 4 %.
//
// What bounds it. Pairs: the MMA rate at the clock the power cap leaves (about
// 1.46 GHz under this load) and, in apply, the operands and the fp32 X that come
// through L2 at 13 TB/s in all; 8 x 1024 x 2048: 392 us, 575 MB read
// and 578 MB written in DRAM, tensor pipe busy 36 % of the time; 64 x 2048 x 1024:
// 2.82 ms, 0.85 PFLOP/s of the 2.41 TFLOP that the symmetric form needs;
// 4096 x 8704 2.0 ms, 1.26 PFLOP/s. Single
// and narrow: the hand-over between phases (4 to 5 us: last store, count, first
// load, ring, epilogue) and the 64 bytes a clock that an SM takes in:
// 3 x 777 x 1333 213 us, 1024 x 1024 147 us, 512 x 512 103 us.
//
//   warp 0      TMA producer (one lane), takes and publishes the tiles
//   warp 1      TMEM allocator, MMA issuer (one lane; pair: the leader's)
//   warps 2..9  epilogue (TMEM lane quarter warp % 4, alternate 32-column chunks)
#pragma once

#include <cuda_fp16.h>

#include "ptx_pair.cuh"

namespace lmoe {

enum NsPhase : int { kNsGram = 0, kNsPoly = 1, kNsApply = 2 };
enum NsOut : int { kNsOutBf16 = 0, kNsOutWeightBf16 = 1, kNsOutWeightF32 = 2 };

enum NsShape : int { kNsNarrow = 0, kNsSingle = 1, kNsPair = 2 };

constexpr int kNsMaxSteps = 32;
constexpr int kNsBK = 64;
constexpr int kNsTileBytes = 128 * kNsBK * 2;  // 16 KB: 128 rows of one operand
__host__ __device__ constexpr int ns_bm(int shape) { return shape == kNsPair ? 256 : 128; }
__host__ __device__ constexpr int ns_bn(int shape) {
  return shape == kNsPair ? 256 : shape == kNsSingle ? 128 : 64;
}
__host__ __device__ constexpr int ns_stages(int shape) { return shape == kNsNarrow ? 7 : 4; }
__host__ __device__ constexpr int ns_stage_bytes(int shape) {
  return shape == kNsNarrow ? kNsTileBytes * 3 / 2 : kNsTileBytes * 2;
}
// epilogue slots of a warp: a narrow tile has one chunk a warp
__host__ __device__ constexpr int ns_slots(int shape) { return shape == kNsNarrow ? 1 : 2; }
constexpr int kNsEpiWarps = 8;
constexpr int kNsThreads = 64 + 32 * kNsEpiWarps;
// An epilogue slot: a 32 x 32 chunk of X in fp32 (128-byte rows, the
// 128-byte swizzle), brought in by TMA ahead of the accumulators, changed in
// place and stored by TMA, and the chunk's next fp16 copy (64-byte rows, 64-byte
// swizzle). poly keeps A' and gram and poly their result and its mirror image in
// the halves of the first. A thread owns a row; the swizzles put 16-byte accesses
// of 8 neighbouring rows into different banks.
constexpr int kNsX = 32 * 128;
constexpr int kNsH = 32 * 64;
constexpr int kNsCoefBytes = kNsEpiWarps * 32 * 4;
constexpr int kNsRing = 4;  // published tiles
constexpr int kNsLooks = 64;
__host__ __device__ constexpr int ns_smem_bytes(int shape) {
  return 1024 + ns_stages(shape) * ns_stage_bytes(shape) +
         kNsEpiWarps * ns_slots(shape) * (kNsX + kNsH) + kNsCoefBytes +
         8 * (2 * ns_stages(shape) + 2 + 2 + 1 + 2 * kNsRing + kNsEpiWarps * ns_slots(shape)) +
         4 * kNsRing + 16;
}
static_assert(ns_smem_bytes(kNsNarrow) <= 232448 && ns_smem_bytes(kNsSingle) <= 232448 &&
                  ns_smem_bytes(kNsPair) <= 232448,
              "Newton-Schulz shared memory");
constexpr int kNsEarly = 2;  // steps in which P keeps its diagonal

// Factors of one step; s_x, s_a, s_p: the scales of the fp16 X, A', P'.
struct NsStep {
  float gram_off;   // s_a / s_x^2
  float gram_diag;  // 1 / s_x^2
  float poly_acc;   // c s_p / s_a^2
  float poly_b;     // b s_p / s_a
  float poly_c;     // c s_p / s_a
  float diag_acc;   // c / s_a^2
  float b, c;
  float s_p;
  // apply; s: the scale of the next X over s_x (last step: 1 / s_x)
  float a_x;        // a s
  float d_x;        // s
  float apply_acc;  // s / s_p
};

// Tensor maps. Operands: boxes of 64 columns x 64 rows, 128-byte swizzle;
// chunks: boxes of 32 x 32, 64-byte (fp16) or 128-byte (X in fp32) swizzle.
struct NsMaps {
  CUtensorMap x[2], gram, poly;
  CUtensorMap chunk_h[2], chunk_x, chunk_gram, chunk_poly;
};

struct NsArgs {
  int batch, group;    // matrices; matrices of a group
  int rows, cols, side, tall, steps;
  int sym_tiles;       // of gram and poly
  int m_tiles, apply_tiles;
  int cut, lower;      // rows of A up to which apply goes first, and its tiles for them
  int k_gram, k_side;  // k-blocks of gram, of poly and apply
  int split;           // parts of gram's k-blocks, each a tile of its own
  long long ld_x, ld_a;
  float* diag_a;       // [batch, ld_a]
  float* diag_p;
  float* parts;        // [batch, sym_tiles, split, tile] gram's partial sums (split > 1)
  int* done;           // a matrix: [4 steps] epilogue warps that have stored gram, poly
                       // and the lower and upper part of apply, then
                       // [sym_tiles, kNsEpiWarps] warps that have left partial sums
  int done_ld;
  int* counter;        // next tile of the sequence
  int out_mode;
  void* out;           // [batch, rows, cols] contiguous
  float keep, move;    // weights: W <- keep W - move X
  unsigned* status;
  NsStep step[kNsMaxSteps];
};

// Shared-memory descriptor of an MN-major fp16 tile, 128-byte swizzle: boxes of
// 64 contiguous MN elements (128 bytes) x 64 k rows, 8 KB a box. Leading
// offset: from one 64-element column of the tile to the next (one box);
// stride offset: from 8 k rows to the next 8 (1024 bytes).
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(const void* tile) {
  const uint64_t addr = smem_addr(tile);
  return ((addr & 0x3FFFFull) >> 4) | (512ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// Instruction descriptor, kind::f16, fp16 operands (format code 0), fp32
// accumulator; a_mn / b_mn: the operand is MN-major (bits 15, 16).
__host__ __device__ constexpr uint32_t instr_desc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Arrive on a barrier of this or the peer CTA without ordering this thread's
// memory accesses: what the arrival announces, TMEM reads, is complete and
// ordered by the tcgen05 fence before it. (The release form waits for the
// thread's outstanding accesses: 0.8 us here.)
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// mbarrier tests that do not suspend the thread.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool mbar_test_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Sum of squares for the Frobenius norm, added up in fp32. Squares below 2^-126 lose
// bits and those below 2^-149 are gone, which for n elements takes at most sqrt(n 2^-149)
// from the norm, 2.6e-18 at the largest size: nothing beside an eps of 1e-12. Below
// that, entries under 2^-40 are added apart, times 2^80, so that norms down to the
// smallest eps are right. (A matrix of ordinary entries has the same sum either way.)
constexpr float kNsPlainEps = 1e-12f;
struct NsSquares {
  static constexpr float kTiny = 9.094947017729282e-13f;  // 2^-40
  static constexpr float kUp = 1.2089258196146292e24f;    // 2^80
  static constexpr float kDown = 8.271806125530277e-25f;  // 2^-80
  float sum = 0.0f, tiny = 0.0f;
  template <int V>
  __device__ __forceinline__ void add(const float (&v)[V], bool apart) {
    if (apart) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool low = fabsf(v[j]) < kTiny;
        const float t = low ? v[j] * kUp : 0.0f, x = low ? 0.0f : v[j];
        tiny = fmaf(t, t, tiny);
        sum = fmaf(x, x, sum);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
    }
  }
  __device__ __forceinline__ float norm() const {
    return sum == 0.0f ? sqrtf(tiny) * kDown : sqrtf(fmaf(tiny * kDown, kDown, sum));
  }
};

struct NsTile {
  int b;           // matrix
  int step, phase;
  int row0, col0;  // of the result
  bool mirror;     // symmetric result, tile below the diagonal
  bool upper;      // apply: past the cut
  int tile, part;  // gram: of the matrix, of its k-blocks
  int kb0, kbs;    // first k-block and how many
};

template <int SHAPE, bool SPLIT>
__device__ __forceinline__ NsTile ns_decode(int t, const NsArgs& a) {
  NsTile c;
  const int split = SPLIT ? a.split : 1;
  const int per_step = (split + 1) * a.sym_tiles + a.apply_tiles;  // of one matrix
  const int per_group = a.group * a.steps * per_step;
  const int g = t / per_group;
  const int first = g * a.group;
  const int n = min(a.group, a.batch - first);
  int r = t - g * per_group;
  c.step = r / (n * per_step);
  r -= c.step * n * per_step;
  int tiles = split * a.sym_tiles;
  c.phase = kNsGram;
  if (r >= n * tiles) {
    r -= n * tiles;
    c.phase = kNsPoly;
    tiles = a.sym_tiles;
    if (r >= n * tiles) {
      r -= n * tiles;
      c.phase = kNsApply;
      tiles = a.apply_tiles;
    }
  }
  const int mi = r / tiles;
  c.b = first + mi;
  int local = r - mi * tiles;
  c.part = 0;
  c.kb0 = 0;
  c.kbs = c.phase == kNsGram ? a.k_gram : a.k_side;
  if (SPLIT && c.phase == kNsGram) {
    c.part = local % split;
    local /= split;
    c.kb0 = c.part * a.k_gram / split;
    c.kbs = (c.part + 1) * a.k_gram / split - c.kb0;
  }
  c.tile = local;
  c.upper = false;
  constexpr int BM = ns_bm(SHAPE), BN = ns_bn(SHAPE);
  constexpr int R = BM / BN;  // tiles across a square of the diagonal
  int i, j;
  if (c.phase != kNsApply) {
    // row i of the lower triangle has R (i + 1) tiles and starts at R i (i + 1) / 2
    const float x = static_cast<float>(local) * (8.0f / R) + 1.0f;
    i = static_cast<int>((sqrtf(x) - 1.0f) * 0.5f);
    while (i > 0 && R * (i * (i + 1) / 2) > local) --i;
    while (R * ((i + 1) * (i + 2) / 2) <= local) ++i;
    j = local - R * (i * (i + 1) / 2);
    c.mirror = j < R * i;
  } else {
    c.upper = local >= a.lower;
    int m = a.m_tiles, i0 = 0;
    if (!a.tall) {
      const int low = (a.cut + BM - 1) / BM;
      if (c.upper) local -= a.lower;
      i0 = c.upper ? low : 0;
      m = c.upper ? m - low : low;
    }
    j = local / m;
    i = i0 + local - j * m;
    c.mirror = false;
  }
  c.row0 = i * BM;
  c.col0 = j * BN;
  return c;
}

// One operand's ROWS x 64 tile: rows / columns mn0.. of matrix b, from k0 on.
template <bool PAIR, int ROWS>
__device__ __forceinline__ void ns_load(const CUtensorMap* map, bool mn, uint64_t* bar,
                                        uint32_t bar_cluster, uint8_t* dst, int mn0, int k0, int b,
                                        uint64_t pol) {
#pragma unroll
  for (int h = 0; h < ROWS / 64; ++h) {
    const int c0 = mn ? mn0 + 64 * h : k0;
    const int c1 = mn ? k0 : mn0 + 64 * h;
    uint8_t* d = dst + h * (kNsTileBytes / 2);
    if constexpr (PAIR)
      tma_load_3d_pair(map, bar_cluster, d, c0, c1, b, pol);
    else
      tma_load_3d(map, bar, d, c0, c1, b, pol);
  }
}

// Eight fp16 numbers as floats, and back.
__device__ __forceinline__ void half8_to_float(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 float_to_half8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 16-byte piece k of a row: 8 halves (64-byte rows) or 4 floats (128-byte rows).
__device__ __forceinline__ uint4* half_at(uint8_t* part, int row, int k) {
  return reinterpret_cast<uint4*>(part + row * 64 + ((k ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ float4* float_at(uint8_t* part, int row, int k) {
  return reinterpret_cast<float4*>(part + row * 128 + ((k ^ (row & 7)) << 4));
}

// gram and poly: one chunk, thread = row. Leaves the fp16 chunk in the first
// half of x (poly: over A') and, for a tile below the diagonal, its mirror image
// in the second. di: d of the thread's row; coef[j]: poly_c d of column j.
__device__ __forceinline__ void ns_sym_chunk(const NsArgs& a, const NsStep& f, const NsTile& c,
                                             uint8_t* slot, const float* coef,
                                             const uint32_t (&v)[32], int row, int col, float di) {
  const int lane = threadIdx.x & 31;
  const bool poly = c.phase == kNsPoly;
  const float scale = poly ? f.poly_acc : f.gram_off;
  const float base = fmaf(f.poly_c, di, f.poly_b);
  uint4 before[4];
  if (poly) {
#pragma unroll
    for (int k = 0; k < 4; ++k) before[k] = *half_at(slot, lane, k);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = scale * __uint_as_float(v[8 * k + i]);
    if (poly) {
      float old[8];
      half8_to_float(before[k], old);
      const float4 c0 = reinterpret_cast<const float4*>(coef)[2 * k];
      const float4 c1 = reinterpret_cast<const float4*>(coef)[2 * k + 1];
      x[0] = fmaf(old[0], base + c0.x, x[0]);
      x[1] = fmaf(old[1], base + c0.y, x[1]);
      x[2] = fmaf(old[2], base + c0.z, x[2]);
      x[3] = fmaf(old[3], base + c0.w, x[3]);
      x[4] = fmaf(old[4], base + c1.x, x[4]);
      x[5] = fmaf(old[5], base + c1.y, x[5]);
      x[6] = fmaf(old[6], base + c1.z, x[6]);
      x[7] = fmaf(old[7], base + c1.w, x[7]);
    }
    const uint4 h = float_to_half8(x);
    *half_at(slot, lane, k) = h;
    if (c.mirror) {
      const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint8_t* to = reinterpret_cast<uint8_t*>(half_at(slot + kNsH, 8 * k + i, lane >> 3));
        *reinterpret_cast<uint16_t*>(to + (lane & 7) * 2) =
            static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
  if (row == col && row + lane < a.side) {
    // this thread's diagonal entry
    float acc = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) acc = lane == j ? __uint_as_float(v[j]) : acc;
    float d = poly ? fmaf(f.diag_acc, acc, di * fmaf(f.c, di, f.b)) : f.gram_diag * acc;
    __half h = __float2half_rn(0.0f);
    if (poly && c.step < kNsEarly) {
      h = __float2half_rn(d * f.s_p);
      d -= __half2float(h) / f.s_p;  // what the rounding left
    }
    reinterpret_cast<__half*>(half_at(slot, lane, lane >> 3))[lane & 7] = h;
    (poly ? a.diag_p : a.diag_a)[c.b * a.ld_a + row + lane] = d;
  }
}

// apply: X' = a X + diag(P) X + P' X of one chunk, thread = row, in place; the
// fp16 copy goes to h (not in the last step). TALL: coef[j] is the factor of X in
// column j; else `by_row`.
template <bool TALL, bool LAST>
__device__ __forceinline__ void ns_apply_chunk(float acc_scale, float by_row, const float* coef,
                                               uint8_t* x, uint8_t* h, const uint32_t (&v)[32]) {
  const int lane = threadIdx.x & 31;
  // all reads first: the compiler cannot tell them from the writes below
  float4 o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = *float_at(x, lane, k);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float4 f = make_float4(by_row, by_row, by_row, by_row);
    if (TALL) f = reinterpret_cast<const float4*>(coef)[k];
    o[k].x = fmaf(f.x, o[k].x, acc_scale * __uint_as_float(v[4 * k]));
    o[k].y = fmaf(f.y, o[k].y, acc_scale * __uint_as_float(v[4 * k + 1]));
    o[k].z = fmaf(f.z, o[k].z, acc_scale * __uint_as_float(v[4 * k + 2]));
    o[k].w = fmaf(f.w, o[k].w, acc_scale * __uint_as_float(v[4 * k + 3]));
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) *float_at(x, lane, k) = o[k];
  if (!LAST) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 p = o[2 * k], q = o[2 * k + 1];
      const float y[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
      *half_at(h, lane, k) = float_to_half8(y);
    }
  }
}

// The caller's output of one chunk from the fp32 X' in the slot: 8 lanes a
// row, 4 columns a lane.
__device__ __forceinline__ void ns_put_out(const NsArgs& a, int b, uint8_t* slot, int row,
                                           int col) {
  const int lane = threadIdx.x & 31;
  const int c = col + (lane & 7) * 4;
  const bool whole = (a.cols & 3) == 0;
  if (c >= a.cols) return;
  const long long at0 =
      (static_cast<long long>(b) * a.rows + row + (lane >> 3)) * a.cols + c;
  const long long step = 4ll * a.cols;
  auto value = [&](int q) {
    const int rr = q * 4 + (lane >> 3);
    return *float_at(slot, rr, lane & 7);
  };
  const int rows = min(8, (a.rows - row - (lane >> 3) + 3) / 4);  // of this lane
  if (a.out_mode == kNsOutWeightF32) {
    float* w = reinterpret_cast<float*>(a.out) + at0;
    if (whole) {
#pragma unroll
      for (int q0 = 0; q0 < 8; q0 += 4) {
        float4 o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q0 + q < rows) o[q] = *reinterpret_cast<const float4*>(w + (q0 + q) * step);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q0 + q < rows) {
            const float4 x = value(q0 + q);
            *reinterpret_cast<float4*>(w + (q0 + q) * step) = make_float4(
                fmaf(a.keep, o[q].x, -a.move * x.x), fmaf(a.keep, o[q].y, -a.move * x.y),
                fmaf(a.keep, o[q].z, -a.move * x.z), fmaf(a.keep, o[q].w, -a.move * x.w));
          }
        }
      }
    } else {
      for (int q = 0; q < rows; ++q) {
        const float4 x4 = value(q);
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < a.cols) w[q * step + i] = fmaf(a.keep, w[q * step + i], -a.move * x[i]);
      }
    }
    return;
  }
  __nv_bfloat16* w = reinterpret_cast<__nv_bfloat16*>(a.out) + at0;
  const bool weight = a.out_mode == kNsOutWeightBf16;
  if (whole) {
#pragma unroll
    for (int q0 = 0; q0 < 8; q0 += 4) {
      uint2 o[4];
      if (weight) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q0 + q < rows) o[q] = *reinterpret_cast<const uint2*>(w + (q0 + q) * step);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q0 + q < rows) {
          float4 x = value(q0 + q);
          if (weight) {
            x.x = fmaf(a.keep, __uint_as_float(o[q].x << 16), -a.move * x.x);
            x.y = fmaf(a.keep, __uint_as_float(o[q].x & 0xffff0000u), -a.move * x.y);
            x.z = fmaf(a.keep, __uint_as_float(o[q].y << 16), -a.move * x.z);
            x.w = fmaf(a.keep, __uint_as_float(o[q].y & 0xffff0000u), -a.move * x.w);
          }
          *reinterpret_cast<uint2*>(w + (q0 + q) * step) =
              make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        }
      }
    }
  } else {
    for (int q = 0; q < rows; ++q) {
      const float4 x4 = value(q);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c + i < a.cols) {
          __nv_bfloat16* p = w + q * step + i;
          *p = __float2bfloat16_rn(
              weight ? fmaf(a.keep, __bfloat162float(*p), -a.move * x[i]) : x[i]);
        }
      }
    }
  }
}

// TMA store of a 32 x 32 chunk from shared memory (this thread's bulk group).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0,
                                             int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The sources of all but the N newest groups have been read.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Every group's writes have been made.
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int SHAPE, bool SPLIT>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_iterate_kernel(const __grid_constant__ NsMaps tm, const __grid_constant__ NsArgs a) {
  constexpr bool PAIR = SHAPE == kNsPair;
  constexpr int kNsStages = ns_stages(SHAPE);
  constexpr int kNsStageBytes = ns_stage_bytes(SHAPE);
  constexpr int kSlots = ns_slots(SHAPE);
  constexpr int kWarpBytes = kSlots * (kNsX + kNsH);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* tiles = smem;
  uint8_t* slots = smem + kNsStages * kNsStageBytes;
  float* coefs = reinterpret_cast<float*>(slots + kNsEpiWarps * kWarpBytes);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(coefs + kNsEpiWarps * 32);
  uint64_t* empty_bar = full_bar + kNsStages;
  uint64_t* tfull_bar = empty_bar + kNsStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* done_bar = tempty_bar + 2;
  uint64_t* tr_full = done_bar + 1;         // [kNsRing]
  uint64_t* tr_empty = tr_full + kNsRing;   // [kNsRing], pair: the leader's is used
  uint64_t* slot_bar = tr_empty + kNsRing;  // [kNsEpiWarps][kSlots]
  int* tile_ring = reinterpret_cast<int*>(slot_bar + kSlots * kNsEpiWarps);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tile_ring + kNsRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  constexpr int kBM = ns_bm(SHAPE), kBN = ns_bn(SHAPE);  // tile
  constexpr int kBRows = PAIR ? 128 : kBN;               // of B in this CTA
  constexpr int kTmem = 2 * kBN;                         // two accumulators
  // readers of a published tile: the MMA issuer, the epilogue warps and, in a
  // pair, the other CTA's producer and epilogue warps
  constexpr int kReaders = PAIR ? 2 + 2 * kNsEpiWarps : 1 + kNsEpiWarps;
  constexpr int kStores = (PAIR ? 2 : 1) * kNsEpiWarps;  // arrivals a tile at `done`
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const uint32_t peer_abort =
      PAIR ? mapa_shared(smem_addr(const_cast<int*>(abort_flag)), static_cast<uint32_t>(rank) ^ 1u)
           : 0u;

  // Waits of one thread and of a whole warp. They look a few times without
  // suspending the thread before they fall back to the bounded waits: the phases
  // of a small matrix are a chain of such waits.
  auto look = [&](uint64_t* bar, uint32_t parity) {
    if constexpr (PAIR) return mbar_test_wait_cluster(bar, parity);
    else return mbar_test_wait(bar, parity);
  };
  auto wait1 = [&](uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < kNsLooks; ++i)
      if (look(bar, parity)) return true;
    if constexpr (PAIR) return wait_bounded_pair(bar, parity, abort_flag, peer_abort, a.status);
    else return wait_bounded(bar, parity, abort_flag, a.status);
  };
  auto wait32 = [&](uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < kNsLooks; ++i)
      if (__all_sync(0xffffffffu, look(bar, parity))) return true;
    if constexpr (PAIR) return warp_wait_bounded_pair(bar, parity, abort_flag, peer_abort, a.status);
    else return warp_wait_bounded(bar, parity, abort_flag, a.status);
  };
  auto commit = [&](uint64_t* bar) {
    if constexpr (PAIR) tc_commit_pair(bar, 0x3);
    else tc_commit(bar);
  };
  // One thread: until `want` warps have arrived at a count (acquire; bounded).
  auto wait_count = [&](const int* p, int want) {
    if (ld_acquire_gpu(p) >= want) return true;
    const uint64_t t0 = global_timer_ns();
    uint32_t n = 0;
    while (true) {
      __nanosleep(20);
      if (ld_acquire_gpu(p) >= want) return true;
      if ((++n & 31u) == 0) {
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          if constexpr (PAIR)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_abort), "r"(1u) : "memory");
          atomicOr(a.status, kStatusTimeout);
          return false;
        }
      }
    }
  };
  // One thread: until every tile of the phase before this one of the same
  // matrix that this one reads has been stored.
  auto wait_phase = [&](const NsTile& c) {
    const int* p = a.done + static_cast<long long>(c.b) * a.done_ld + 4 * c.step + c.phase - 1;
    if (c.phase != kNsGram) return wait_count(p, kStores * a.sym_tiles);
    if (c.step == 0) return true;
    if (!wait_count(p - 1, kStores * a.lower)) return false;
    return c.row0 < a.cut || wait_count(p, kStores * (a.apply_tiles - a.lower));
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNsStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], kStores);
    }
    mbar_init(done_bar, 1);
    for (int i = 0; i < kNsRing; ++i) {
      mbar_init(&tr_full[i], 1);
      mbar_init(&tr_empty[i], kReaders);
    }
    for (int i = 0; i < kSlots * kNsEpiWarps; ++i) mbar_init(&slot_bar[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == 2 && lane < sizeof(NsMaps) / sizeof(CUtensorMap))
    tma_prefetch_desc(reinterpret_cast<const CUtensorMap*>(&tm) + lane);
  __syncwarp();
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmem);
      tmem_relinquish();
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after_sync();

  const uint32_t tmem_base = *tmem_slot;
  const int total =
      a.batch * a.steps * (((SPLIT ? a.split : 1) + 1) * a.sym_tiles + a.apply_tiles);
  const uint32_t tr_empty_leader = PAIR ? mapa_shared(smem_addr(&tr_empty[0]), 0) : 0u;

  auto read_tile = [&](int& slot, uint32_t& ph) -> int {
    if (!wait1(&tr_full[slot], ph)) return -2;
    const int t = *reinterpret_cast<volatile int*>(&tile_ring[slot]);
    if constexpr (PAIR)
      mbar_arrive_cluster(tr_empty_leader + 8u * static_cast<uint32_t>(slot));
    else
      mbar_arrive(&tr_empty[slot]);
    if (++slot == kNsRing) {
      slot = 0;
      ph ^= 1u;
    }
    return t;
  };

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      int slot = 0;
      uint32_t slot_ph = 0;
      bool ok = true;
      int t_next = leader ? atomicAdd(a.counter, 1) : 0;
      const uint32_t ring_peer = PAIR ? mapa_shared(smem_addr(&tile_ring[0]), 1) : 0u;
      const uint32_t full_peer = PAIR ? mapa_shared(smem_addr(&tr_full[0]), 1) : 0u;
      while (ok) {
        int t;
        if (leader) {
          t = t_next < total ? t_next : -1;
          if (!wait1(&tr_empty[slot], slot_ph ^ 1u)) break;
          tile_ring[slot] = t;
          if constexpr (PAIR) st_cluster_s32(ring_peer + 4u * static_cast<uint32_t>(slot), t);
          mbar_arrive(&tr_full[slot]);
          if constexpr (PAIR) mbar_arrive_cluster(full_peer + 8u * static_cast<uint32_t>(slot));
          if (++slot == kNsRing) {
            slot = 0;
            slot_ph ^= 1u;
          }
        } else {
          t = read_tile(slot, slot_ph);
        }
        if (t < 0) break;
        const NsTile c = ns_decode<SHAPE, SPLIT>(t, a);
        const CUtensorMap* mx = &tm.x[c.step & 1];
        const CUtensorMap* ma = c.phase == kNsPoly ? &tm.gram : mx;
        const CUtensorMap* mb = ma;
        bool amn = false, bmn = false;
        if (c.phase == kNsGram) {
          amn = bmn = a.tall != 0;
        } else if (c.phase == kNsApply) {
          bmn = a.tall == 0;
          if (a.tall) mb = &tm.poly;
          else ma = &tm.poly;
        }
        const int arow = c.row0 + rank * 128;
        const int brow = c.col0 + rank * 128;
        const int kbs = c.kbs;
        const int ahead = kbs > kNsStages ? kbs - kNsStages : 0;
        if (!wait_phase(c)) break;
        fence_proxy_async_global();
        for (int kb = 0; kb < kbs; ++kb) {
          // the next tile, late: one taken early would wait here behind this one
          // while other CTAs run dry
          if (leader && kb == ahead) t_next = atomicAdd(a.counter, 1);
          if (!wait1(&empty_bar[stage], phase ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* sa = tiles + stage * kNsStageBytes;
          const uint32_t fb = PAIR ? mapa_shared(smem_addr(&full_bar[stage]), 0) : 0u;
          if (leader)
            mbar_arrive_expect_tx(&full_bar[stage], (PAIR ? 2u : 1u) * kNsStageBytes);
          ns_load<PAIR, 128>(ma, amn, &full_bar[stage], fb, sa, arow, (c.kb0 + kb) * kNsBK, c.b,
                             pol);
          ns_load<PAIR, kBRows>(mb, bmn, &full_bar[stage], fb, sa + kNsTileBytes, brow,
                                (c.kb0 + kb) * kNsBK, c.b, pol);
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // drain the copies still in flight (pair: the leader's barriers count both CTAs' bytes)
      if (leader)
        for (int s = 0; s < kNsStages; ++s)
          if (issued_mask & (1u << s)) wait_drain(&full_bar[s], (issued_parity >> s) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      int slot = 0;
      uint32_t slot_ph = 0;
      bool ok = true;
      while (ok) {
        const int t = read_tile(slot, slot_ph);
        if (t < 0) break;
        const NsTile c = ns_decode<SHAPE, SPLIT>(t, a);
        const bool amn = c.phase == kNsGram && a.tall != 0;
        const bool bmn = c.phase == kNsGram ? amn : c.phase == kNsApply && a.tall == 0;
        const uint32_t idesc = instr_desc_f16(kBM, kBN, amn, bmn);
        // 16 elements of K: 32 bytes along a K-major row, 16 rows of 128 bytes otherwise
        const uint64_t step_a = amn ? 128ull : 2ull;
        const uint64_t step_b = bmn ? 128ull : 2ull;
        const int kbs = c.kbs;
        if (!wait1(&tempty_bar[acc], acc_phase ^ 1u)) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = 0; kb < kbs; ++kb) {
          if (!wait1(&full_bar[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint8_t* sa = tiles + stage * kNsStageBytes;
          const uint8_t* sb = sa + kNsTileBytes;
          const uint64_t da = amn ? smem_desc_sw128_mn(sa) : smem_desc_sw128(sa);
          const uint64_t db = bmn ? smem_desc_sw128_mn(sb) : smem_desc_sw128(sb);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t accum = (kb | k) != 0 ? 1u : 0u;
            if constexpr (PAIR)
              tc_mma_pair(d_tmem, da + step_a * k, db + step_b * k, idesc, accum);
            else
              tc_mma(d_tmem, da + step_a * k, db + step_b * k, idesc, accum);
          }
          commit(&empty_bar[stage]);
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit(&tfull_bar[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      commit(done_bar);
      wait_drain(done_bar, 0);
    }
  } else {
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    uint8_t* my_slots = slots + (warp - 2) * kWarpBytes;
    float* coef = coefs + (warp - 2) * 32;
    uint64_t* my_bars = slot_bar + kSlots * (warp - 2);
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_addr(&tempty_bar[0]), 0) : 0u;
    const uint64_t pol = policy_evict_normal();
    int acc = 0;
    uint32_t acc_phase = 0;
    int slot = 0;
    uint32_t slot_ph = 0;
    uint32_t bar_ph = 0;   // bit s: parity of slot s's next load
    uint32_t in_flight = 0;  // lane 0: slots with a load that nobody has waited for
    while (true) {
      int t = 0;
      if (lane == 0) t = read_tile(slot, slot_ph);
      t = __shfl_sync(0xffffffffu, t, 0);
      if (t < 0) break;
      const NsTile c = ns_decode<SHAPE, SPLIT>(t, a);
      const NsStep& f = a.step[c.step];
      const bool sym = c.phase != kNsApply;
      const bool poly = c.phase == kNsPoly;
      const bool last = !sym && c.step + 1 == a.steps;
      const int M = sym ? a.side : a.rows, N = sym ? a.side : a.cols;
      const int row = c.row0 + rank * 128 + quarter * 32;
      const int col0 = c.col0 + half * 32;
      // this warp's chunks: columns col0, col0 + 64, ...
      int chunks = 0;
      if (row < M && col0 < N) chunks = min(kBN / 64, (N - col0 + 63) / 64);
      // lane 0: bring chunk i into slot i % kSlots
      auto load_chunk = [&](int i) {
        uint64_t* bar = &my_bars[i % kSlots];
        mbar_arrive_expect_tx(bar, poly ? kNsH : kNsX);
        tma_load_3d(poly ? &tm.chunk_gram : &tm.chunk_x, bar,
                    my_slots + (i % kSlots) * kNsX, col0 + 64 * i, row, c.b, pol);
        in_flight |= 1u << (i % kSlots);
      };
      // the old values and the diagonals are read while the MMAs run (the slots
      // are free: the last tile's stores have been waited for). by_row: d of the
      // thread's row (poly) or the factor of X in it (apply, wide); by_col: the
      // same by column, to be handed round through `coef`.
      float by_row = 0.0f, by_col = 0.0f;
      const float* diag = (poly ? a.diag_a : a.diag_p) + c.b * a.ld_a;
      const bool cols_differ = poly || (!sym && a.tall);
      auto load_col = [&](int i) {
        const int j = col0 + 64 * i + lane;
        if (cols_differ && i < chunks && j < N) by_col = __ldcg(diag + j);
      };
      if (c.phase != kNsGram && chunks > 0) {
        int ok = 1;
        if (lane == 0) {
          ok = wait_phase(c) ? 1 : 0;
          if (ok) {
            fence_proxy_async_global();
            load_chunk(0);
            if (kSlots > 1 && chunks > 1) load_chunk(1);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        // lane 0 has acquired the count for the warp: a shuffle orders no memory
        __syncwarp();
        if (row + lane < M && (poly || !a.tall)) by_row = __ldcg(diag + row + lane);
        if (!sym) by_row = fmaf(f.d_x, by_row, f.a_x);
        load_col(0);
      }
      if (!wait32(&tfull_bar[acc], acc_phase)) break;
      tc_fence_after_sync();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc * kBN + half * 32);
      bool ok = true;
      // a part of gram's k-blocks: every chunk's sums to memory (turn 0); the warp
      // that comes last for its rows adds the parts and goes on with them (turn 1)
      const bool joined = SPLIT && c.phase == kNsGram;
      bool mine = true;  // this warp's results are the tile's
      float4* parts = nullptr;
      if constexpr (SPLIT) {
        if (joined)
          parts = reinterpret_cast<float4*>(a.parts) +
                  (static_cast<long long>(c.b * a.sym_tiles + c.tile) * a.split) *
                      (kBM * kBN / 4) +
                  (warp - 2) * (kBN / 64) * 256 + lane;
      }
      for (int turn = joined ? 0 : 1; turn < 2 && mine && ok; ++turn) {
        if (joined && turn == 1) {
          // in the order of the parts, so the sum does not depend on who adds it
          int last_in = 0;
          __syncwarp();
          if (lane == 0) {
            __threadfence();
            const int n = atomicAdd(a.done + static_cast<long long>(c.b) * a.done_ld + 4 * a.steps +
                                        c.tile * kNsEpiWarps + (warp - 2),
                                    1);
            __threadfence();
            last_in = (n + 1) % a.split == 0 ? 1 : 0;
          }
          mine = __shfl_sync(0xffffffffu, last_in, 0) != 0;
          if (!mine) break;
          __syncwarp();  // the other lanes' reads come after lane 0's fence
        }
        for (int i = 0; i < chunks; ++i) {
          const int col = col0 + 64 * i;
          const int sl = i % kSlots;
          uint8_t* sx = my_slots + sl * kNsX;
          uint8_t* sh = my_slots + kSlots * kNsX + sl * kNsH;
          uint32_t v[32];
          if (joined && turn == 1) {
            float sum[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) sum[k] = 0.0f;
            // two parts at a time on their way
            for (int p = 0; p < a.split; p += 2) {
              float4 w[2][8];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float4* from =
                    parts + static_cast<long long>(p + h) * (kBM * kBN / 4) + i * 256;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  w[h][k] = p + h < a.split ? __ldcg(from + 32 * k)
                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  sum[4 * k] += w[h][k].x;
                  sum[4 * k + 1] += w[h][k].y;
                  sum[4 * k + 2] += w[h][k].z;
                  sum[4 * k + 3] += w[h][k].w;
                }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(sum[k]);
          } else {
            tmem_ld_32cols(tbase + static_cast<uint32_t>(64 * i), v);
          }
          if (cols_differ) {
            coef[lane] = poly ? f.poly_c * by_col : fmaf(f.d_x, by_col, f.a_x);
            load_col(i + 1);
          }
          if (lane == 0) {
            if (c.phase == kNsGram) {
              bulk_wait_read<1>();  // the chunk before last has left this slot
            } else if (i > 0 && i + 1 < chunks) {
              // the last chunk has left its slot: bring in the next one
              if (!last) bulk_wait_read<0>();
              load_chunk(i + 1);
            }
          }
          if (c.phase != kNsGram) {
            if (!wait32(&my_bars[sl], (bar_ph >> sl) & 1u)) {
              ok = false;
              break;
            }
            bar_ph ^= 1u << sl;
            if (lane == 0) in_flight &= ~(1u << sl);
          }
          __syncwarp();
          tmem_ld_wait();
          if (i + 1 == chunks && !(joined && turn == 1)) {
            // the accumulators are free
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR)
                mbar_arrive_relaxed_cluster(tempty0 + 8u * static_cast<uint32_t>(acc));
              else mbar_arrive(&tempty_bar[acc]);
            }
          }
          if (joined && turn == 0) {
            float4* to = parts + static_cast<long long>(c.part) * (kBM * kBN / 4) + i * 256;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              to[32 * k] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                       __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
            continue;
          }
          if (sym) {
            ns_sym_chunk(a, f, c, sx, coef, v, row, col, by_row);
          } else if (last) {
            if (a.tall) ns_apply_chunk<true, true>(f.apply_acc, by_row, coef, sx, sh, v);
            else ns_apply_chunk<false, true>(f.apply_acc, by_row, coef, sx, sh, v);
            __syncwarp();
            ns_put_out(a, c.b, sx, row, col);
            // the slot's next contents come by TMA
            fence_async_smem();
            __syncwarp();
            continue;
          } else {
            if (a.tall) ns_apply_chunk<true, false>(f.apply_acc, by_row, coef, sx, sh, v);
            else ns_apply_chunk<false, false>(f.apply_acc, by_row, coef, sx, sh, v);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (sym) {
              const CUtensorMap* to = poly ? &tm.chunk_poly : &tm.chunk_gram;
              tma_store_3d(to, sx, col, row, c.b);
              if (c.mirror) tma_store_3d(to, sx + kNsH, row, col, c.b);
            } else {
              tma_store_3d(&tm.chunk_x, sx, col, row, c.b);
              tma_store_3d(&tm.chunk_h[(c.step + 1) & 1], sh, col, row, c.b);
            }
            bulk_commit();
          }
        }
      }
      if (!ok) break;
      if (chunks == 0) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_relaxed_cluster(tempty0 + 8u * static_cast<uint32_t>(acc));
          else mbar_arrive(&tempty_bar[acc]);
        }
      }
      if (!last && mine) {
        // this warp's part is in memory: count it for the next phase's tiles
        __syncwarp();
        if (lane == 0) {
          bulk_wait_all();
          __threadfence();
          atomicAdd(a.done + static_cast<long long>(c.b) * a.done_ld + 4 * c.step + c.phase +
                        (c.upper ? 1 : 0),
                    1);
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) {
      // after a wait that gave up: what is still in flight
      for (int s = 0; s < kSlots; ++s)
        if (in_flight & (1u << s)) wait_drain(&my_bars[s], (bar_ph >> s) & 1u);
      bulk_wait_all();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, kTmem);
    else tmem_dealloc(tmem_base, kTmem);
  }
}

}  // namespace lmoe

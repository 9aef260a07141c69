// Matrix products of the Newton-Schulz iteration X <- a X + (b A + c A^2) X,
// A = X X^T (X wide) or X <- a X + X (b A + c A^2), A = X^T X (X tall), on
// tcgen05 tensor cores. Three products a step, one kernel:
//
//   gram  A = X X^T or X^T X      symmetric: tiles on and below the diagonal,
//   poly  P = b A + c A A         the tiles below stored a second time, mirrored
//   apply X' = a X + P X or a X + X P
//
// Operands are fp16 with a power-of-two scale per matrix kind and step (the
// host derives it from a bound on X's spectral norm, so no entry overflows and
// entries 2^-28 below the largest possible one are still normal numbers),
// accumulators fp32. fp16 and not bf16: 11 bits against 8 at the same MMA
// rate; on gradient-like matrices the result is off by 1.2e-3 to 1.7e-3 of its
// norm, against about 1e-2 with bf16. X itself lives in fp32 beside its fp16
// operand copy and a X is taken from it: the small singular directions, which
// the iteration amplifies up to a^steps = 485 times, pass through the a X term
// alone, and with X held only in fp16 the rounding of the large directions
// drowns them (matrices of low rank plus noise: 2e-2; with the fp32 X 3e-4).
//
// X keeps the caller's orientation. Where the contracted index is X's row
// index, X is read as an MN-major operand (TMA boxes of 64 contiguous columns x
// 64 rows, the transpose bits of the instruction descriptor), so nothing is
// ever transposed in memory:
//   wide: gram K-major x K-major, apply: P K-major, X MN-major
//   tall: gram MN-major x MN-major, apply: X K-major, P K-major (symmetric)
// Sizes that no tile divides need no padding: TMA fills what lies outside a
// matrix with zeros (the batch is the maps' third dimension, so a box never
// reaches into the next matrix) and the epilogue stores what lies inside.
//
// Tiles: PAIR = true: 256 x 256 on two SMs (cta_group::2, each CTA holds 128
// rows of A and 128 of B); PAIR = false: 128 x 128 on one SM, for products
// with few tiles. Either way a CTA takes in 16 KB + 16 KB a k-block.
//
//   warp 0      TMA producer (one lane)
//   warp 1      TMEM allocator, MMA issuer (one lane; pair: the leader's)
//   warps 2..9  epilogue (TMEM lane quarter warp % 4, alternate 32-column chunks)
#pragma once

#include <cuda_fp16.h>

#include "ptx_pair.cuh"

namespace lmoe {

enum NsEpi : int { kNsGram = 0, kNsPoly = 1, kNsApply = 2 };
enum NsOut : int { kNsOutNext = 0, kNsOutBf16 = 1, kNsOutWeightBf16 = 2, kNsOutWeightF32 = 3 };

constexpr int kNsBK = 64;
constexpr int kNsStages = 5;
constexpr int kNsTileBytes = 128 * kNsBK * 2;      // 16 KB: 128 rows of one operand
constexpr int kNsStageBytes = 2 * kNsTileBytes;
constexpr int kNsEpiWarps = 8;
constexpr int kNsThreads = 64 + 32 * kNsEpiWarps;
// epilogue staging: a 32 x 32 fp32 chunk per warp, 33 floats a row, so that
// row-wise and column-wise accesses are both free of bank conflicts
constexpr int kNsPitch = 33;
constexpr int kNsStageWarpBytes = 32 * kNsPitch * 4;
constexpr int kNsBarrierBytes = 8 * (2 * kNsStages + 2 + 2 + 1);
constexpr int kNsSmemBytes =
    1024 + kNsStages * kNsStageBytes + kNsEpiWarps * kNsStageWarpBytes + kNsBarrierBytes + 16;
static_assert(kNsSmemBytes <= 232448, "Newton-Schulz GEMM shared memory");

struct NsArgs {
  int batch;
  int M, N;       // result size
  int k_blocks;   // ceil(K / 64)
  int m_tiles, n_tiles;  // of a result (symmetric: n_tiles unused)
  int tiles;      // tiles of one result
  float alpha;    // factor of the accumulator
  float beta;     // kNsPoly: factor of the old A; kNsApply: a
  float scale;    // kNsApply: 2^s of the next fp16 copy
  __half* out16;          // kNsGram, kNsPoly: result; kNsApply: next fp16 copy (kNsOutNext)
  const __half* old16;    // kNsPoly: A
  float* x32;             // kNsApply: X in fp32, updated in place
  long long ld;           // row stride of out16 / old16 / x32, elements
  long long bstride;      // matrix stride of the same
  int out_mode;           // kNsApply
  void* out;              // kNsApply, last step: [batch, M, N] contiguous
  float keep, move;       // weights: W <- keep W - move X
  unsigned* status;
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

struct NsTile {
  int b;           // matrix
  int row0, col0;  // of the result
  bool mirror;     // symmetric result, tile below the diagonal
};

template <int BT, bool SYM>
__device__ __forceinline__ NsTile ns_decode(int t, const NsArgs& a) {
  NsTile c;
  c.b = t / a.tiles;
  const int local = t - c.b * a.tiles;
  int i, j;
  if (SYM) {
    // row i of the lower triangle starts at i (i + 1) / 2
    i = static_cast<int>((sqrtf(8.0f * static_cast<float>(local) + 1.0f) - 1.0f) * 0.5f);
    while (i > 0 && i * (i + 1) / 2 > local) --i;
    while ((i + 1) * (i + 2) / 2 <= local) ++i;
    j = local - i * (i + 1) / 2;
  } else {
    i = local % a.m_tiles;
    j = local / a.m_tiles;
  }
  c.row0 = i * BT;
  c.col0 = j * BT;
  c.mirror = SYM && i != j;
  return c;
}

// One operand's 128 x 64 tile: rows / columns mn0.. of matrix b, k-block kb.
template <bool MN, bool PAIR>
__device__ __forceinline__ void ns_load(const CUtensorMap* map, uint64_t* bar, uint32_t bar_cluster,
                                        uint8_t* dst, int mn0, int k0, int b, uint64_t pol) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c0 = MN ? mn0 + 64 * h : k0;
    const int c1 = MN ? k0 : mn0 + 64 * h;
    uint8_t* d = dst + h * (kNsTileBytes / 2);
    if constexpr (PAIR)
      tma_load_3d_pair(map, bar_cluster, d, c0, c1, b, pol);
    else
      tma_load_3d(map, bar, d, c0, c1, b, pol);
  }
}

// Epilogue of one 32 x 32 chunk: the warp's accumulators (thread = row) go
// through the staging so that global accesses run along the rows of the
// result (and along its columns for the mirrored copy).
template <int EPI>
__device__ __forceinline__ void ns_store_chunk(const NsArgs& a, const uint32_t (&v)[32], float* st,
                                               int b, int row, int col, bool mirror) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 32; ++j) st[lane * kNsPitch + j] = a.alpha * __uint_as_float(v[j]);
  __syncwarp();
  const int piece = (lane & 7) * 4;
  const long long mbase = static_cast<long long>(b) * a.bstride;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int rr = q * 4 + (lane >> 3);
    const int r = row + rr;
    const int c = col + piece;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = st[rr * kNsPitch + piece + i];
    if (r < a.M && c < a.N) {
      const long long at = mbase + static_cast<long long>(r) * a.ld + c;
      // ld is a multiple of 8 and c of 4: whole 4-element accesses stay inside
      // the padded row
      if constexpr (EPI == kNsPoly) {
        const uint2 o = *reinterpret_cast<const uint2*>(a.old16 + at);
        const float2 o01 = __half22float2(*reinterpret_cast<const __half2*>(&o.x));
        const float2 o23 = __half22float2(*reinterpret_cast<const __half2*>(&o.y));
        x[0] = fmaf(a.beta, o01.x, x[0]);
        x[1] = fmaf(a.beta, o01.y, x[1]);
        x[2] = fmaf(a.beta, o23.x, x[2]);
        x[3] = fmaf(a.beta, o23.y, x[3]);
        // the mirrored copy takes the finished values
        if (mirror) {
#pragma unroll
          for (int i = 0; i < 4; ++i) st[rr * kNsPitch + piece + i] = x[i];
        }
      }
      if constexpr (EPI == kNsApply) {
        const float4 o = *reinterpret_cast<const float4*>(a.x32 + at);
        x[0] = fmaf(a.beta, o.x, x[0]);
        x[1] = fmaf(a.beta, o.y, x[1]);
        x[2] = fmaf(a.beta, o.z, x[2]);
        x[3] = fmaf(a.beta, o.w, x[3]);
        if (a.out_mode == kNsOutNext) {
          *reinterpret_cast<float4*>(a.x32 + at) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
          const long long to = (static_cast<long long>(b) * a.M + r) * a.N + c;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (c + i >= a.N) break;
            if (a.out_mode == kNsOutBf16) {
              reinterpret_cast<__nv_bfloat16*>(a.out)[to + i] = __float2bfloat16_rn(x[i]);
            } else if (a.out_mode == kNsOutWeightBf16) {
              __nv_bfloat16* w = reinterpret_cast<__nv_bfloat16*>(a.out) + to + i;
              *w = __float2bfloat16_rn(fmaf(a.keep, __bfloat162float(*w), -a.move * x[i]));
            } else {
              float* w = reinterpret_cast<float*>(a.out) + to + i;
              *w = fmaf(a.keep, *w, -a.move * x[i]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= a.scale;
      }
      if (EPI != kNsApply || a.out_mode == kNsOutNext) {
        __half2 h01 = __floats2half2_rn(x[0], x[1]), h23 = __floats2half2_rn(x[2], x[3]);
        uint2 w;
        w.x = *reinterpret_cast<uint32_t*>(&h01);
        w.y = *reinterpret_cast<uint32_t*>(&h23);
        *reinterpret_cast<uint2*>(a.out16 + at) = w;
      }
    }
  }
  if (EPI != kNsApply && mirror) {
    __syncwarp();
    // row col + cc of the mirrored copy: column cc of the chunk
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int cc = q * 4 + (lane >> 3);
      const int r = col + cc;   // < row0: always inside
      const int c = row + piece;
      if (c < a.M) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = st[(piece + i) * kNsPitch + cc];
        __half2 h01 = __floats2half2_rn(x[0], x[1]), h23 = __floats2half2_rn(x[2], x[3]);
        uint2 w;
        w.x = *reinterpret_cast<uint32_t*>(&h01);
        w.y = *reinterpret_cast<uint32_t*>(&h23);
        *reinterpret_cast<uint2*>(a.out16 + mbase + static_cast<long long>(r) * a.ld + c) = w;
      }
    }
  }
  __syncwarp();
}

template <bool PAIR, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const NsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* tiles = smem;
  uint8_t* stage_smem = smem + kNsStages * kNsStageBytes;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(stage_smem + kNsEpiWarps * kNsStageWarpBytes);
  uint64_t* empty_bar = full_bar + kNsStages;
  uint64_t* tfull_bar = empty_bar + kNsStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* done_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  constexpr bool kSym = EPI != kNsApply;
  constexpr int kBT = PAIR ? 256 : 128;       // tile rows and columns
  constexpr int kTmem = 2 * kBT;              // two accumulators of kBT columns
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int units = PAIR ? gridDim.x >> 1 : gridDim.x;
  const uint32_t peer_abort =
      PAIR ? mapa_shared(smem_addr(const_cast<int*>(abort_flag)), static_cast<uint32_t>(rank) ^ 1u)
           : 0u;

  // wait of one thread / one warp on a barrier of this CTA
  auto wait1 = [&](uint64_t* bar, uint32_t parity) {
    if constexpr (PAIR) return wait_bounded_pair(bar, parity, abort_flag, peer_abort, a.status);
    else return wait_bounded(bar, parity, abort_flag, a.status);
  };
  auto wait32 = [&](uint64_t* bar, uint32_t parity) {
    if constexpr (PAIR) return warp_wait_bounded_pair(bar, parity, abort_flag, peer_abort, a.status);
    else return warp_wait_bounded(bar, parity, abort_flag, a.status);
  };
  auto commit = [&](uint64_t* bar) {
    if constexpr (PAIR) tc_commit_pair(bar, 0x3);
    else tc_commit(bar);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNsStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], (PAIR ? 2 : 1) * kNsEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_async_smem();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
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
  const int total = a.tiles * a.batch;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const NsTile c = ns_decode<kBT, kSym>(t, a);
        const int arow = c.row0 + rank * 128;
        const int brow = c.col0 + rank * 128;
        for (int kb = 0; kb < a.k_blocks; ++kb) {
          if (!wait1(&empty_bar[stage], phase ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* sa = tiles + stage * kNsStageBytes;
          uint8_t* sb = sa + kNsTileBytes;
          const uint32_t fb = PAIR ? mapa_shared(smem_addr(&full_bar[stage]), 0) : 0u;
          if (leader)
            mbar_arrive_expect_tx(&full_bar[stage], (PAIR ? 2u : 1u) * kNsStageBytes);
          ns_load<AMN, PAIR>(&tmA, &full_bar[stage], fb, sa, arow, kb * kNsBK, c.b, pol);
          ns_load<BMN, PAIR>(&tmB, &full_bar[stage], fb, sb, brow, kb * kNsBK, c.b, pol);
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
      constexpr uint32_t idesc = instr_desc_f16(kBT, kBT, AMN, BMN);
      // 16 elements of K: 32 bytes along a K-major row, 16 rows of 128 bytes otherwise
      constexpr uint64_t kStepA = AMN ? 128ull : 2ull;
      constexpr uint64_t kStepB = BMN ? 128ull : 2ull;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        if (!wait1(&tempty_bar[acc], acc_phase ^ 1u)) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kBT);
        for (int kb = 0; kb < a.k_blocks; ++kb) {
          if (!wait1(&full_bar[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint8_t* sa = tiles + stage * kNsStageBytes;
          const uint64_t da = AMN ? smem_desc_sw128_mn(sa) : smem_desc_sw128(sa);
          const uint64_t db =
              BMN ? smem_desc_sw128_mn(sa + kNsTileBytes) : smem_desc_sw128(sa + kNsTileBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t accum = (kb | k) != 0 ? 1u : 0u;
            if constexpr (PAIR)
              tc_mma_pair(d_tmem, da + kStepA * k, db + kStepB * k, idesc, accum);
            else
              tc_mma(d_tmem, da + kStepA * k, db + kStepB * k, idesc, accum);
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
    float* st = reinterpret_cast<float*>(stage_smem + (warp - 2) * kNsStageWarpBytes);
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_addr(&tempty_bar[0]), 0) : 0u;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = unit; t < total; t += units) {
      const NsTile c = ns_decode<kBT, kSym>(t, a);
      if (!wait32(&tfull_bar[acc], acc_phase)) break;
      tc_fence_after_sync();
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kBT);
      const int row = c.row0 + rank * 128 + quarter * 32;
      if (row < a.M) {
        for (int ch = half; ch < kBT / 32; ch += 2) {
          const int col = c.col0 + ch * 32;
          if (col >= a.N) break;
          uint32_t v[32];
          tmem_ld_32cols(tbase + static_cast<uint32_t>(ch * 32), v);
          tmem_ld_wait();
          ns_store_chunk<EPI>(a, v, st, c.b, row, col, c.mirror);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(tempty0 + 8u * static_cast<uint32_t>(acc));
        else
          mbar_arrive(&tempty_bar[acc]);
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
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

// The gated block's products for few tokens (one to kFewMost): all of the weights
// have to come in for a few rows of x, so DRAM bounds them, and the work is laid out
// for that alone.
//
// D^T = W x^T: 128 rows of weights are the MMA's M (gate+up: 64 gate rows and the up
// rows of the same features; in the gradient, columns of the weights, an MN-major
// operand), the tokens its N, so no lane of the tensor core waits
// for tokens that are not there. The k-blocks of all tiles form one sequence that is
// cut into equal parts, one a CTA, wherever the cuts fall: every SM reads the same
// number of weights (a tile a CTA would leave 8704 rows / 128 = 68 tiles on 152 SMs).
// A CTA's sums of a tile go to memory in fp32; whoever comes last for a tile adds the
// parts in the order of the CTAs, so results do not depend on who that is, and
// finishes it: activation and product, or the rounding to bf16.
//
// The second product's CTAs bring in their first weights where the first product's
// have left an SM (programmatic dependent launch), and wait for the whole of it only
// before they read h.
//
// What bounds it: DRAM, and for small weights the two launches' ends (last loads, parts
// to memory, last arrival, sums: about 5 us each, more with more tokens). 8704 x 10240, one
// token 88 us (6.1 TB/s, 0.90 of the copy rate), 27 tokens 95, 64 tokens 107, 128 tokens 128;
// 2048 x 2048, one token 14. Taking the tile from a unit's number by division in the
// producing thread cost 11 us of 105, a ring of 6 stages in place of 11 another 4.
//
//   warp 0      TMA producer (one lane)
//   warp 1      TMEM allocator, MMA issuer (one lane)
//   warps 2..5  epilogue (TMEM lane quarter warp % 4)
#pragma once

#include "ffn_gemm.cuh"

namespace lmoe {

constexpr int kFewThreads = 64 + 128;
constexpr int kFewWBytes = 128 * kFfnBK * 2;
__host__ __device__ constexpr int few_stages(int nt) {
  return nt == 16 ? 11 : nt == 32 ? 10 : nt == 64 ? 8 : 6;
}
__host__ __device__ constexpr int few_stage_bytes(int nt) { return kFewWBytes + nt * kFfnBK * 2; }
__host__ __device__ constexpr int few_smem_bytes(int nt) {
  return 1024 + few_stages(nt) * few_stage_bytes(nt) + 8 * (2 * few_stages(nt) + 2 + 2 + 1) + 32;
}
static_assert(few_smem_bytes(16) <= 232448 && few_smem_bytes(32) <= 232448 &&
                  few_smem_bytes(64) <= 232448 && few_smem_bytes(128) <= 232448,
              "shared memory of the kernel for few tokens");

// First unit (k-block of the sequence) of CTA c of n.
__device__ __forceinline__ long long few_first(long long units, int c, int n) {
  return units * c / n;
}
// The CTA that has unit u: the largest c with units * c / n <= u, that is with
// units * c < (u + 1) * n.
__device__ __forceinline__ int few_owner(long long units, long long u, int n) {
  return static_cast<int>(((u + 1) * n - 1) / units);
}

// Barrier of the 128 epilogue threads that says whether every one of them brought true.
__device__ __forceinline__ bool few_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

// The sums of a tile's rows r[0], r[1], ... for tokens n, n + step, ...: kFewBatch
// tokens of two parts at a time on their way.
constexpr int kFewBatch = 8;
template <int ROWS>
__device__ __forceinline__ void few_sum(const float* parts, long long part, int c0, int c1,
                                        int tokens, int n, int step, const int (&r)[ROWS],
                                        float (&s)[ROWS][kFewBatch]) {
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int j = 0; j < kFewBatch; ++j) s[i][j] = 0.0f;
  for (int c = c0; c <= c1; c += 2) {
    float v[2][ROWS][kFewBatch];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // of the CTA that begins the tile its last part, of the others their first
      const float* from = parts + (2ll * (c + h) + (c + h > c0 ? 0 : 1)) * part;
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < kFewBatch; ++j)
          v[h][i][j] = c + h <= c1 && n + j * step < tokens
                           ? __ldcg(from + (n + j * step) * 128 + r[i])
                           : 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < kFewBatch; ++j) s[i][j] += v[h][i][j];
  }
}

template <int EPI, int NT, bool MN>
__global__ void __launch_bounds__(kFewThreads, 1) ffn_few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kStages = few_stages(NT);
  constexpr int kStage = few_stage_bytes(NT);
  constexpr int kTmem = 2 * NT;  // two accumulators; at least 32 columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* tfull_bar = empty_bar + kStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* done_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* last_in = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(a.tiles) * a.k_blocks;
  const int ctas = static_cast<int>(gridDim.x);
  const long long u0 = few_first(units, blockIdx.x, ctas);
  const long long u1 = few_first(units, blockIdx.x + 1, ctas);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  const int n_units = static_cast<int>(u1 - u0);
  // brings weights of a tile's k-block into a stage
  auto load_w = [&](int tile, int kb, int stage, uint64_t pol) {
    const int k0 = kb * kFfnBK;
    uint8_t* dst = ring + stage * kStage;
    if (EPI == kFfnGateUp) {
      tma_load_2d(&a.w[0], &full_bar[stage], dst, k0, tile * 64, pol);
      tma_load_2d(&a.w[1], &full_bar[stage], dst + kFewWBytes / 2, k0, tile * 64, pol);
    } else if (MN) {
      const bool second = kb >= a.cut;
      const CUtensorMap* map = second ? &a.w[1] : &a.w[0];
      const int row = second ? k0 - a.cut * kFfnBK : k0;
      tma_load_2d(map, &full_bar[stage], dst, tile * 128, row, pol);
      tma_load_2d(map, &full_bar[stage], dst + kFewWBytes / 2, tile * 128 + 64, row, pol);
    } else {
      tma_load_2d(&a.w[0], &full_bar[stage], dst, k0, tile * 128, pol);
      tma_load_2d(&a.w[0], &full_bar[stage], dst + kFewWBytes / 2, k0, tile * 128 + 64, pol);
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ TMA producer
      tma_prefetch_desc(&a.w[0]);
      if (EPI == kFfnGateUp) tma_prefetch_desc(&a.w[1]);
      tma_prefetch_desc(&a.x[0]);
      const uint64_t pol = policy_evict_first(), pol_x = policy_evict_last();
      // the units in turn: a division for each would take as long as its copies
      int tile = static_cast<int>(u0 / a.k_blocks);
      int kb = static_cast<int>(u0 - static_cast<long long>(tile) * a.k_blocks);
      int x_kb = kb;
      const int early = a.early ? (n_units < kStages ? n_units : kStages) : 0;
      auto next_w = [&](int stage) {
        mbar_arrive_expect_tx(&full_bar[stage], kStage);
        load_w(tile, kb, stage, pol);
        if (++kb == a.k_blocks) {
          kb = 0;
          ++tile;
        }
      };
      for (int i = 0; i < early; ++i) next_w(i);
      pdl_wait();
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      for (int i = 0; i < n_units; ++i) {
        if (i >= early) {
          if (!wait_bounded(&empty_bar[stage], phase ^ 1u, abort_flag, a.status)) break;
          next_w(stage);
        }
        const bool second = MN && x_kb >= a.cut;
        tma_load_2d(second ? &a.x[1] : &a.x[0], &full_bar[stage],
                    ring + stage * kStage + kFewWBytes, (second ? x_kb - a.cut : x_kb) * kFfnBK, 0,
                    pol_x);
        if (++x_kb == a.k_blocks) x_kb = 0;
        issued_mask |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      for (int s = 0; s < kStages; ++s)
        if (issued_mask & (1u << s)) wait_drain(&full_bar[s], (issued_parity >> s) & 1u);
    }
  } else if (warp == 1) {
    pdl_wait();
    if (lane == 0) {
      // ------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = instr_desc_bf16(128, NT) | (MN ? 1u << 15 : 0u);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (long long u = u0; u < u1 && ok;) {
        const long long tile = u / a.k_blocks;
        long long end = (tile + 1) * a.k_blocks;
        if (end > u1) end = u1;
        if (!wait_bounded(&tempty_bar[acc], acc_phase ^ 1u, abort_flag, a.status)) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * NT);
        uint32_t accum = 0;
        for (; u < end; ++u) {
          if (!wait_bounded(&full_bar[stage], phase, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t dw =
              MN ? ffn_desc_mn(ring + stage * kStage) : smem_desc_sw128(ring + stage * kStage);
          const uint64_t dx = smem_desc_sw128(ring + stage * kStage + kFewWBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            tc_mma(d_tmem, dw + (MN ? 128ull : 2ull) * k, dx + 2ull * k, idesc, accum);
            accum = 1u;
          }
          tc_commit(&empty_bar[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&tfull_bar[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      tc_commit(done_bar);
      wait_drain(done_bar, 0);
    }
  } else {
    // ------------------------------------------------ epilogue
    pdl_wait();
    // the next kernel may begin: what is ahead of this one has finished
    pdl_launch_dependents();
    const int quarter = warp & 3;
    const int i = quarter * 32 + lane;  // row of the tile
    const int e = threadIdx.x - 64;     // 0..127
    int acc = 0;
    uint32_t acc_phase = 0;
    float* mine = a.parts + static_cast<long long>(blockIdx.x) * 2 * NT * 128;
    for (long long u = u0; u < u1;) {
      const int tile = static_cast<int>(u / a.k_blocks);
      const long long first = static_cast<long long>(tile) * a.k_blocks;
      const long long end = first + a.k_blocks;
      if (!few_all(warp_wait_bounded(&tfull_bar[acc], acc_phase, abort_flag, a.status))) break;
      tc_fence_after_sync();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc * NT);
      // a part that begins inside a tile is this CTA's first, one that ends inside
      // it its last: two places for the two
      float* part = mine + (u > first ? 0 : NT * 128);
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        uint32_t v[16];
        tmem_ld_16cols(tbase + static_cast<uint32_t>(c), v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < a.tokens) part[(c + j) * 128 + i] = __uint_as_float(v[j]);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[acc]);
      const int c0 = few_owner(units, first, ctas), c1 = few_owner(units, end - 1, ctas);
      __threadfence();
      named_barrier(1, 128);
      if (e == 0) {
        const int n = c1 > c0 ? atomicAdd(&a.arrived[tile], 1) : 0;
        *last_in = n == c1 - c0;
        if (c1 > c0 && n == c1 - c0) a.arrived[tile] = 0;
        __threadfence();
      }
      named_barrier(1, 128);
      if (*last_in) {
        if (EPI == kFfnGateUp) {
          const int r = e & 63, f = tile * 64 + r;
          if (f < a.rows) {
            for (int n = e >> 6; n < a.tokens; n += 2 * kFewBatch) {
              const int both[2] = {r, 64 + r};
              float s[2][kFewBatch];
              few_sum(a.parts, NT * 128, c0, c1, a.tokens, n, 2, both, s);
#pragma unroll
              for (int j = 0; j < kFewBatch; ++j) {
                const long long t = n + 2 * j;
                if (t >= a.tokens) break;
                a.out[t * a.ld + f] = __float2bfloat16_rn(s[0][j] * ffn_sigmoid(s[0][j]) * s[1][j]);
                if (a.gate != nullptr) {
                  a.gate[t * a.rows + f] = __float2bfloat16_rn(s[0][j]);
                  a.up[t * a.rows + f] = __float2bfloat16_rn(s[1][j]);
                }
              }
            }
          }
        } else {
          const int f = tile * 128 + e;
          if (f < a.rows) {
            for (int n = 0; n < a.tokens; n += kFewBatch) {
              const int one[1] = {e};
              float s[1][kFewBatch];
              few_sum(a.parts, NT * 128, c0, c1, a.tokens, n, 1, one, s);
#pragma unroll
              for (int j = 0; j < kFewBatch; ++j) {
                const long long t = n + j;
                if (t >= a.tokens) break;
                if (EPI == kFfnDGate) {
                  const float g = __bfloat162float(a.gate[t * a.rows + f]);
                  const float u = __bfloat162float(a.up[t * a.rows + f]);
                  const float sig = ffn_sigmoid(g), act = g * sig;
                  a.out[t * a.ld + f] =
                      __float2bfloat16_rn(s[0][j] * u * fmaf(act, 1.0f - sig, sig));
                  a.du[t * a.ld + f] = __float2bfloat16_rn(s[0][j] * act);
                  a.h[t * a.ld + f] = __float2bfloat16_rn(act * u);
                } else {
                  a.out[t * a.ld + f] = __float2bfloat16_rn(s[0][j]);
                }
              }
            }
          }
        }
      }
      named_barrier(1, 128);  // last_in is free
      u = end < u1 ? end : u1;
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmem);
  }
}

}  // namespace lmoe

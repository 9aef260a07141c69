// Matrix products of the gated feed-forward block and its gradient on tcgen05
// tensor cores: h = SiLU(x Wg^T) * (x Wu^T), y = h Wd^T, and
//
//   dh = dy Wd;  dg = dh up SiLU'(gate),  du = dh SiLU(gate),  h once more
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h
//
// with SiLU'(g) = s + g s (1 - s), s = 1 / (1 + e^-g). Every product is D = A B^T
// of operands read where the caller (or the launch before) left them: where the
// contracted index is a matrix's row index, the operand is MN-major (TMA boxes of
// 64 contiguous columns x 64 rows, the transpose bits of the instruction
// descriptor), so nothing is transposed in memory and the weights need no second
// layout:
//   gate+up  x K-major, Wg and Wu K-major       dgate  dy K-major, Wd MN-major
//   down     h K-major, Wd K-major              dx     dg, du K-major, Wg, Wu MN-major
//   dW       both operands MN-major (K = tokens)
// Two launches forward, two backward. The gradient's second launch holds all four
// products, dx as one of two K segments: their tiles form one sequence, so the
// GPU runs out of tiles once and not four times.
//
// Numbers. Operands are bf16, accumulators fp32; the activation and its derivative
// are taken in fp32 from the accumulators (forward) or from the gate and up that
// the forward left in bf16 (backward). h, dg and du are rounded to bf16 once, as
// operands of the next product: 2^-9 of an entry in the mean, as much as the
// rounding of a bf16 result; keeping them wider would double those products.
//
// Order. Tiles of one product are alike and go to the units in turn. Those of the
// gradient's last launch differ in length (dx: 2 F / 64 k-blocks, dW: tokens / 64), so
// running units take them from a counter, the longest first (each unit's first tile is its
// own), towards the end of the one before. us, in turn / from the counter: 777 x 1336 x 2040
// 66 / 51, 300 x 4096 x 4096 105 / 78, 200 x 8704 x 10240 311 / 251, 512 x 2048 x 2048 51 / 40.
//
// What bounds it. An SM takes in 64 bytes a clock: 512 clocks for a k-block's 32 KB, as
// many as the MMAs of a pair's k-block take (a single tile's take half of them). The
// producing threads need most of that time too, so each operand has a thread, and nothing
// else is done in their loops (one thread for both: 2 % slower; taking the tiles in its loop:
// 14 %; 16 KB boxes chosen at run time: 10 %). Large products run at the clock that the power
// cap leaves: 8192 x 8704 x 10240 forward 2.8 ms, 1.58 PFLOP/s; 4096 x 2048 x 2048 at the full
// clock 76 us, 1.36 PFLOP/s, with 3.4 and 1.7 rounds of tiles.
//
// Sizes that no tile divides: TMA fills what lies outside an operand with zeros
// and stores only what lies inside a result; boxes that begin past a result's end
// are not stored at all.
//
//   warp 0      TMA producer of A (one lane)
//   warp 1      TMEM allocator, MMA issuer (one lane; pair: the leader's)
//   warp 11     TMA producer of B (one lane)
//   warps 2..9  epilogue (TMEM lane quarter warp % 4, alternate 32-column chunks):
//               a 32 x 32 chunk goes through the warp's slots in shared memory and
//               leaves (dgate: gate and up also arrive) by TMA
//   warp 10     takes the tiles from the counter and publishes them (one lane)
// Tiles: 256 x 256 on SM pairs (cta_group::2), 128 x 128 on one SM; two
// accumulators in TMEM, one filled while the other is drained.
#pragma once

#include "ffn.h"
#include "ptx_pair.cuh"

namespace lmoe {

constexpr int kFfnTileBytes = 128 * kFfnBK * 2;  // 128 rows of one operand
constexpr int kFfnStageBytes = 2 * kFfnTileBytes;
constexpr int kFfnEpiWarps = 8;
constexpr int kFfnThreads = 128 + 32 * kFfnEpiWarps;
constexpr int kFfnChunk = 32 * 64;  // 32 x 32 bf16, 64-byte swizzle; fp32: two, 128-byte swizzle
constexpr int kFfnSlots = 2;
constexpr int kFfnRing = 2;  // published tiles
__host__ __device__ constexpr int ffn_stages(int epi) { return epi == kFfnPlain ? 5 : 4; }
__host__ __device__ constexpr int ffn_slot_bytes(int epi) {
  return epi == kFfnPlain ? 2 * kFfnChunk : 3 * kFfnChunk;
}
// Shared memory: ring, slots (the ring and every slot's parts begin on 1024-byte
// boundaries: 2 KB chunks, whose swizzle patterns repeat every 512 or 1024), barriers.
__host__ __device__ constexpr int ffn_smem_bytes(int epi) {
  return 1024 + ffn_stages(epi) * kFfnStageBytes + kFfnEpiWarps * kFfnSlots * ffn_slot_bytes(epi) +
         8 * (2 * ffn_stages(epi) + 2 + 2 + 1 + kFfnEpiWarps * kFfnSlots + 2 * kFfnRing + 1) +
         4 * kFfnRing + 16;
}
static_assert(ffn_smem_bytes(kFfnGateUp) <= 232448 && ffn_smem_bytes(kFfnPlain) <= 232448,
              "gated block shared memory");

// Shared-memory descriptor of an MN-major bf16 tile, 128-byte swizzle: boxes of
// 64 contiguous MN elements (128 bytes) x 64 k rows, 8 KB a box. Leading offset:
// from one 64-element column of the tile to the next (a box); stride offset: from
// 8 k rows to the next 8 (1024 bytes).
__device__ __forceinline__ uint64_t ffn_desc_mn(const void* tile) {
  const uint64_t addr = smem_addr(tile);
  return ((addr & 0x3FFFFull) >> 4) | (512ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// Arrive on a barrier of this or the peer CTA without ordering this thread's
// memory accesses: what the arrival announces, TMEM reads, is complete and
// ordered by the tcgen05 fence before it.
__device__ __forceinline__ void ffn_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0,
                                             int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_addr(src)), "r"(c0), "r"(c1)
      : "memory");
}
// The same as an addition to what is there (fp32).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int c0,
                                           int c1) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_addr(src)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void ffn_bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void ffn_bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ffn_bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

struct FfnTile {
  int p;           // product
  int row0, col0;  // of the result (gate+up: output features)
};

template <int EPI, int SHAPE>
__device__ __forceinline__ FfnTile ffn_decode(int t, const FfnArgs& a) {
  FfnTile c;
  c.p = 0;
  if (EPI == kFfnPlain) {
#pragma unroll
    for (int i = 1; i < kFfnProducts; ++i)
      if (i < a.products && t >= a.p[i].first) c.p = i;
  }
  const FfnProduct& p = a.p[c.p];
  // bands of m-tiles, n slower: CTAs that run at the same time share rows of A and of B
  const int local = t - p.first;
  const int per = a.band * p.n_tiles;
  const int b = local / per;
  const int gm = min(a.band, p.m_tiles - b * a.band);
  const int in = local - b * per;
  const int n = in / gm;
  c.row0 = (b * a.band + in - n * gm) * ffn_bm(SHAPE);
  c.col0 = n * (EPI == kFfnGateUp ? ffn_bn(SHAPE) / 2 : ffn_bn(SHAPE));
  return c;
}

// One operand box of 64 x 64 at column c0 and row c1 of the matrix.
template <bool PAIR>
__device__ __forceinline__ void ffn_load(const CUtensorMap* map, uint64_t* bar,
                                         uint32_t bar_cluster, uint8_t* dst, int c0, int c1,
                                         uint64_t pol) {
  if constexpr (PAIR) tma_load_2d_pair(map, bar_cluster, dst, c0, c1, pol);
  else tma_load_2d(map, bar, dst, c0, c1, pol);
}

// 16-byte piece k of a slot's row: 8 bf16 (64-byte rows) or 4 floats (128-byte rows).
__device__ __forceinline__ uint4* ffn_half_at(uint8_t* part, int row, int k) {
  return reinterpret_cast<uint4*>(part + row * 64 + ((k ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ float4* ffn_float_at(uint8_t* part, int row, int k) {
  return reinterpret_cast<float4*>(part + row * 128 + ((k ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint4 ffn_pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void ffn_unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// 1 / (1 + e^-g), within a few units of 2^-22 of itself for every g whose sigmoid
// is a normal number (the hardware's exp2 and reciprocal).
__device__ __forceinline__ float ffn_sigmoid(float g) {
  return __fdividef(1.0f, 1.0f + __expf(-g));
}

template <int EPI, int SHAPE>
__global__ void __launch_bounds__(kFfnThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnArgs a) {
  constexpr bool PAIR = SHAPE == kFfnPair;
  constexpr int kStages = ffn_stages(EPI);
  constexpr int kSlotBytes = ffn_slot_bytes(EPI);
  constexpr int kBN = ffn_bn(SHAPE);
  // tiles from the counter; of one product they are all alike
  const bool take = EPI == kFfnPlain && a.products > 1;
  // readers of a published tile: producers, the MMA issuer, epilogue warps
  constexpr int kReaders = PAIR ? 5 + 2 * kFfnEpiWarps : 3 + kFfnEpiWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* tiles = smem;
  uint8_t* slots = smem + kStages * kFfnStageBytes;
  uint64_t* full_bar =
      reinterpret_cast<uint64_t*>(slots + kFfnEpiWarps * kFfnSlots * kSlotBytes);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* tfull_bar = empty_bar + kStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* done_bar = tempty_bar + 2;
  uint64_t* slot_bar = done_bar + 1;  // [kFfnEpiWarps][kFfnSlots]
  uint64_t* tr_full = slot_bar + kFfnEpiWarps * kFfnSlots;  // [kFfnRing]
  uint64_t* tr_empty = tr_full + kFfnRing;                  // [kFfnRing], pair: the leader's is used
  uint64_t* want_bar = tr_empty + kFfnRing;  // the producer nears its tile's end
  int* tile_ring = reinterpret_cast<int*>(want_bar + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tile_ring + kFfnRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int units = PAIR ? gridDim.x >> 1 : gridDim.x;
  const uint32_t peer_abort =
      PAIR ? mapa_shared(smem_addr(const_cast<int*>(abort_flag)), static_cast<uint32_t>(rank) ^ 1u)
           : 0u;
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
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], (PAIR ? 2 : 1) * kFfnEpiWarps);
    }
    mbar_init(done_bar, 1);
    for (int i = 0; i < kFfnEpiWarps * kFfnSlots; ++i) mbar_init(&slot_bar[i], 1);
    for (int i = 0; i < kFfnRing; ++i) {
      mbar_init(&tr_full[i], 1);
      mbar_init(&tr_empty[i], kReaders);
    }
    mbar_init(want_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == 2 && lane < a.products) {
    tma_prefetch_desc(&a.p[lane].a[0]);
    tma_prefetch_desc(&a.p[lane].b[0]);
    tma_prefetch_desc(&a.p[lane].out[0]);
  }
  __syncwarp();
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * kBN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * kBN);
      tmem_relinquish();
    }
  }
  // nothing above reads global memory: the set-up overlaps the previous kernel
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t tr_empty_leader =
      PAIR ? mapa_shared(smem_addr(&tr_empty[0]), 0) : smem_addr(&tr_empty[0]);

  // The tile after t, for one thread; -1: no more. The arrival needs no release: it
  // announces a read, made by the time its value is compared.
  int ring_slot = 0;
  uint32_t ring_ph = 0;
  auto next_tile = [&](int t) -> int {
    if (!take) return t + units < a.tiles ? t + units : -1;
    if (!wait1(&tr_full[ring_slot], ring_ph)) return -1;
    t = *reinterpret_cast<volatile int*>(&tile_ring[ring_slot]);
    if (t >= -1) ffn_arrive_relaxed(tr_empty_leader + 8u * static_cast<uint32_t>(ring_slot));
    if (++ring_slot == kFfnRing) {
      ring_slot = 0;
      ring_ph ^= 1u;
    }
    return t;
  };

  if (warp == 0 || warp == kFfnEpiWarps + 3) {
    if (lane == 0) {
      // ------------------------------------------------ TMA producers: A and B
      const bool of_b = warp != 0;
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int t = unit; ok && t >= 0; t = ok ? next_tile(t) : -1) {
        const FfnTile c = ffn_decode<EPI, SHAPE>(t, a);
        const FfnProduct& p = a.p[c.p];
        const bool mn = (of_b ? p.b_mn : p.a_mn) != 0;
        // first row or column of the tile's two boxes. gate+up: pair, the gate rows in CTA 0
        // and the up rows in CTA 1; single, 64 gate rows, then the up rows of the same features
        const bool both = EPI == kFfnGateUp && of_b;
        const int row = !of_b ? c.row0 + rank * 128 : both ? c.col0 : c.col0 + rank * 128;
        const int step = both && !PAIR ? 0 : 64;
        const int k_blocks = p.k_blocks;
        for (int g = 0; g < p.segments && ok; ++g) {
          const CUtensorMap* m0 = both ? &p.b[PAIR ? rank : 0] : of_b ? &p.b[g] : &p.a[g];
          const CUtensorMap* m1 = both && !PAIR ? &p.b[1] : m0;
          // coordinates of the boxes, and what a k-block adds to them
          int x = mn ? row : 0, y = mn ? 0 : row;
          const int dx = mn ? step : 0, dy = mn ? 0 : step;
          const int kx = mn ? 0 : kFfnBK, ky = mn ? kFfnBK : 0;
          // the next tile is wanted two rings before this one's end: taken earlier, it
          // would wait here behind this one while other units run dry. Two ranges, so that
          // the loop itself has nothing to ask.
          const bool last = g + 1 == p.segments;
          const int cut = !last ? k_blocks : k_blocks > 2 * kStages ? k_blocks - 2 * kStages : 0;
          for (int kb = 0, end = cut;; ++kb) {
            if (kb == end) {
              if (take && leader && !of_b && last && end == cut) mbar_arrive(want_bar);
              if (end == k_blocks) break;
              end = k_blocks;
            }
            if (!wait1(&empty_bar[stage], phase ^ 1u)) {
              ok = false;
              break;
            }
            uint8_t* to = tiles + stage * kFfnStageBytes + (of_b ? kFfnTileBytes : 0);
            uint64_t* bar = &full_bar[stage];
            const uint32_t fb = PAIR ? mapa_shared(smem_addr(bar), 0) : 0u;
            // one arrival a phase, for the bytes of both operands (and CTAs): the others'
            // copies may complete before it
            if (leader && !of_b) mbar_arrive_expect_tx(bar, (PAIR ? 2u : 1u) * kFfnStageBytes);
            ffn_load<PAIR>(m0, bar, fb, to, x, y, pol);
            ffn_load<PAIR>(m1, bar, fb, to + kFfnTileBytes / 2, x + dx, y + dy, pol);
            x += kx;
            y += ky;
            issued_mask |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      // drain the copies still in flight (pair: the leader's barriers count both CTAs' bytes)
      if (leader)
        for (int s = 0; s < kStages; ++s)
          if (issued_mask & (1u << s)) wait_drain(&full_bar[s], (issued_parity >> s) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------ MMA issuer
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int t = unit; ok && t >= 0; t = ok ? next_tile(t) : -1) {
        const FfnTile c = ffn_decode<EPI, SHAPE>(t, a);
        const FfnProduct& p = a.p[c.p];
        const bool amn = p.a_mn != 0, bmn = p.b_mn != 0;
        const uint32_t idesc = instr_desc_bf16(ffn_bm(SHAPE), kBN) | (amn ? 1u << 15 : 0u) |
                               (bmn ? 1u << 16 : 0u);
        // 16 elements of K: 32 bytes along a K-major row, 16 rows of 128 bytes otherwise
        const uint64_t step_a = amn ? 128ull : 2ull;
        const uint64_t step_b = bmn ? 128ull : 2ull;
        const int kbs = p.k_blocks * p.segments;
        if (!wait1(&tempty_bar[acc], acc_phase ^ 1u)) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = 0; kb < kbs; ++kb) {
          if (!wait1(&full_bar[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint8_t* sa = tiles + stage * kFfnStageBytes;
          const uint8_t* sb = sa + kFfnTileBytes;
          const uint64_t da = amn ? ffn_desc_mn(sa) : smem_desc_sw128(sa);
          const uint64_t db = bmn ? ffn_desc_mn(sb) : smem_desc_sw128(sb);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t accum = (kb | k) != 0 ? 1u : 0u;
            if constexpr (PAIR)
              tc_mma_pair(d_tmem, da + step_a * k, db + step_b * k, idesc, accum);
            else
              tc_mma(d_tmem, da + step_a * k, db + step_b * k, idesc, accum);
          }
          commit(&empty_bar[stage]);
          if (++stage == kStages) {
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
  } else if (warp == 2 + kFfnEpiWarps) {
    if (take && lane == 0 && leader) {
      // ------------------------------------------------ tiles
      const uint32_t ring_peer = PAIR ? mapa_shared(smem_addr(&tile_ring[0]), 1) : 0u;
      const uint32_t full_peer = PAIR ? mapa_shared(smem_addr(&tr_full[0]), 1) : 0u;
      int n = 0;
      uint32_t want_ph = 0;
      while (n >= 0) {
        if (!wait1(want_bar, want_ph)) break;
        want_ph ^= 1u;
        if (!wait1(&tr_empty[ring_slot], ring_ph ^ 1u)) break;
        n = units + atomicAdd(a.counter, 1);
        if (n >= a.tiles) n = -1;
        tile_ring[ring_slot] = n;
        if constexpr (PAIR) st_cluster_s32(ring_peer + 4u * static_cast<uint32_t>(ring_slot), n);
        mbar_arrive(&tr_full[ring_slot]);
        if constexpr (PAIR) mbar_arrive_cluster(full_peer + 8u * static_cast<uint32_t>(ring_slot));
        if (++ring_slot == kFfnRing) {
          ring_slot = 0;
          ring_ph ^= 1u;
        }
      }
      if (atomicAdd(a.counter + 1, 1) == units - 1) {
        // every unit has taken its last tile: ready for the next launch
        a.counter[0] = 0;
        a.counter[1] = 0;
      }
    }
  } else {
    // ------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    uint8_t* my_slots = slots + (warp - 2) * kFfnSlots * kSlotBytes;
    uint64_t* my_bars = slot_bar + kFfnSlots * (warp - 2);
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_addr(&tempty_bar[0]), 0) : 0u;
    const uint64_t pol = policy_evict_first();
    constexpr int kCols = EPI == kFfnGateUp ? kBN / 2 : kBN;  // of the result, a tile
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t bar_ph = 0;     // bit s: parity of slot s's next load
    uint32_t in_flight = 0;  // lane 0: slots with a load that nobody has waited for
    int turn = 0;            // slot of the next chunk
    auto next_of_warp = [&](int t) {
      if (!take) return next_tile(t);
      if (lane == 0) t = next_tile(t);
      return __shfl_sync(0xffffffffu, t, 0);
    };
    for (int t = unit; t >= 0; t = next_of_warp(t)) {
      const FfnTile c = ffn_decode<EPI, SHAPE>(t, a);
      const FfnProduct& p = a.p[c.p];
      const int row = c.row0 + rank * 128 + quarter * 32;
      const int col0 = c.col0 + half * 32;
      int chunks = 0;  // this warp's: columns col0, col0 + 64, ...
      if (row < p.M && col0 < p.N) chunks = min(kCols / 64, (p.N - col0 + 63) / 64);
      // dgate, lane 0: bring gate and up of chunk i into slot s
      auto load_chunk = [&](int i, int s) {
        mbar_arrive_expect_tx(&my_bars[s], 2 * kFfnChunk);
        tma_load_2d(&a.gate, &my_bars[s], my_slots + s * kSlotBytes, col0 + 64 * i, row, pol);
        tma_load_2d(&a.up, &my_bars[s], my_slots + s * kSlotBytes + kFfnChunk, col0 + 64 * i, row,
                    pol);
        in_flight |= 1u << s;
      };
      if (EPI == kFfnDGate && lane == 0 && chunks > 0) {
        // read while the MMAs run; the last tile's chunks have left their slots
        ffn_bulk_wait_read<0>();
        load_chunk(0, turn);
        if (chunks > 1) load_chunk(1, turn ^ 1);
      }
      if (!wait32(&tfull_bar[acc], acc_phase)) break;
      tc_fence_after_sync();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(acc * kBN + half * 32);
      bool ok = true;
      for (int i = 0; i < chunks; ++i) {
        const int col = col0 + 64 * i;
        uint8_t* slot = my_slots + turn * kSlotBytes;
        uint32_t v[32], w[32];
        tmem_ld_32cols(tbase + static_cast<uint32_t>(64 * i), v);
        if (EPI == kFfnGateUp) tmem_ld_32cols(tbase + static_cast<uint32_t>(kBN / 2 + 64 * i), w);
        if (lane == 0) {
          if (EPI != kFfnDGate) {
            ffn_bulk_wait_read<kFfnSlots - 1>();  // the chunk before last has left this slot
          } else if (i > 0 && i + 1 < chunks) {
            ffn_bulk_wait_read<0>();  // the last chunk has left its slot: bring in the next one
            load_chunk(i + 1, turn ^ 1);
          }
        }
        if (EPI == kFfnDGate) {
          if (!wait32(&my_bars[turn], (bar_ph >> turn) & 1u)) {
            ok = false;
            break;
          }
          bar_ph ^= 1u << turn;
          if (lane == 0) in_flight &= ~(1u << turn);
        }
        __syncwarp();
        tmem_ld_wait();
        if (i + 1 == chunks) {
          // the accumulators are free
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) ffn_arrive_relaxed(tempty0 + 8u * static_cast<uint32_t>(acc));
            else mbar_arrive(&tempty_bar[acc]);
          }
        }
        if constexpr (EPI == kFfnPlain) {
          if (p.out_mode == kFfnBf16) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *ffn_half_at(slot, lane, k) = ffn_pack8(reinterpret_cast<const float*>(v) + 8 * k);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *ffn_float_at(slot, lane, k) =
                  make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                              __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
          }
        } else if constexpr (EPI == kFfnGateUp) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* g = reinterpret_cast<const float*>(v) + 8 * k;
            const float* u = reinterpret_cast<const float*>(w) + 8 * k;
            if (p.save) {
              *ffn_half_at(slot + kFfnChunk, lane, k) = ffn_pack8(g);
              *ffn_half_at(slot + 2 * kFfnChunk, lane, k) = ffn_pack8(u);
            }
            float h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = g[j] * ffn_sigmoid(g[j]) * u[j];
            *ffn_half_at(slot, lane, k) = ffn_pack8(h);
          }
        } else {
          uint4 gs[4], us[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            gs[k] = *ffn_half_at(slot, lane, k);
            us[k] = *ffn_half_at(slot + kFfnChunk, lane, k);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float g[8], u[8], h[8];
            ffn_unpack8(gs[k], g);
            ffn_unpack8(us[k], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float dh = __uint_as_float(v[8 * k + j]);
              const float s = ffn_sigmoid(g[j]);
              const float act = g[j] * s;
              h[j] = act * u[j];
              g[j] = dh * u[j] * fmaf(act, 1.0f - s, s);
              u[j] = dh * act;
            }
            *ffn_half_at(slot, lane, k) = ffn_pack8(g);
            *ffn_half_at(slot + kFfnChunk, lane, k) = ffn_pack8(u);
            *ffn_half_at(slot + 2 * kFfnChunk, lane, k) = ffn_pack8(h);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (EPI == kFfnPlain && p.out_mode == kFfnF32Add)
            tma_add_2d(&p.out[0], slot, col, row);
          else
            tma_store_2d(&p.out[0], slot, col, row);
          if (EPI == kFfnDGate || (EPI == kFfnGateUp && p.save)) {
            tma_store_2d(&p.out[1], slot + kFfnChunk, col, row);
            tma_store_2d(&p.out[2], slot + 2 * kFfnChunk, col, row);
          }
          ffn_bulk_commit();
        }
        turn ^= 1;
      }
      if (!ok) break;
      if (chunks == 0) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) ffn_arrive_relaxed(tempty0 + 8u * static_cast<uint32_t>(acc));
          else mbar_arrive(&tempty_bar[acc]);
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) {
      // after a wait that gave up: what is still in flight
      for (int s = 0; s < kFfnSlots; ++s)
        if (in_flight & (1u << s)) wait_drain(&my_bars[s], (bar_ph >> s) & 1u);
      ffn_bulk_wait_all();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  // every MMA of the pair has completed (the leader waited on its last commit)
  // and both epilogues are done with TMEM
  if constexpr (PAIR) cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 2 * kBN);
    else tmem_dealloc(tmem_base, 2 * kBN);
  }
}

}  // namespace lmoe

// The Newton-Schulz iteration for matrices with a short side of at most 128,
// whole, in one launch: a cluster of CTAs holds the matrix on chip from the
// gradient to the result.
//
// The matrix is taken as X [m, n], m the short side (a tall one is transposed on
// the way in and out). CTA r of the cluster keeps columns [r W, (r + 1) W) of X:
// in fp32 in tensor memory (128 lanes x W columns) and in fp16 in shared memory,
// where the same bytes serve as K-major operand of the gram product and as
// MN-major operand of the apply product. A step:
//   gram   partial A = X_r X_r^T (M = N = 128, K = W), to shared memory in fp32;
//          each CTA adds its share of the rows over the cluster (in a fixed order)
//          through distributed shared memory and hands the fp16 A' and the fp32
//          diagonal d to all CTAs
//   poly   P = b A + c A A, by every CTA for itself (K = m)
//   apply  X_r <- a X_r + P X_r (N = W, K = m)
// with the number formats, scales and factors of ns_iterate.cuh. The norm and
// the momentum update are the head of the same launch, the weight update its
// tail. What bounds it is latency: five steps of three short products each with
// its hand-over, 2.5 us a step for one CTA, 5 to 9 us with the exchange of partial
// grams over a cluster; as tiles of the general kernel the same phases take 20 us a
// step, because each goes through global memory. Measured: 64 x 2048 28 us (general
// kernel 83), 128 x 128 22, 128 x 256 28, 128 x 4096 52, 64 matrices of 128 x 256
// 29, 64 of 128 x 512 54, 16 of 100 x 500 42 us. Rows that are no whole vectors go through shared
// memory (read as they lie, 100 x 500 took 54 us).
//
// Every thread runs through every barrier whatever happened: a wait that gave up
// sets the status and the kernel goes on (with wrong numbers), so that no CTA of
// the cluster waits for one that left.
#pragma once

#include "ns.h"

namespace lmoe {

constexpr int kSmallX = 128 * kSmallW * 2;   // 64 KB: tiles of 128 rows x 64 columns
constexpr int kSmallA = 128 * 128 * 2;       // 32 KB: A', and P
constexpr int kSmallPart = 128 * 128 * 4;    // 64 KB: partial gram
constexpr int kSmallBytes = 1024 + kSmallX + 2 * kSmallA + kSmallPart + 128 * 4 * 2 +
                            kSmallCluster * 8 + 8 * 8 + 64;
static_assert(kSmallBytes <= 232448, "Newton-Schulz small kernel shared memory");

__device__ __forceinline__ void tmem_st_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u2(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y)
               : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// MN-major tile whose 64-element columns are 128 k rows (16 KB) apart.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn16(const void* tile) {
  const uint64_t addr = smem_addr(tile);
  return ((addr & 0x3FFFFull) >> 4) | (1024ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// Byte offset of the 16-byte piece that holds columns 8 k8 .. of a row, in tiles
// of 128 rows x 64 columns of fp16 with the 128-byte swizzle.
__device__ __forceinline__ int op_at(int row, int k8) {
  return (k8 >> 3) * 16384 + row * 128 + (((k8 & 7) ^ (row & 7)) << 4);
}

// A warp's 32 x 32 chunk X[i0 .., j0 ..] of a [m, n] matrix that is stored as it is
// (wide) or transposed (tall), thread = row; zeros outside. Whole vectors where
// rows start on them; transposed, the lanes of a column are neighbours in memory;
// else row by row through `turn` (32 x 33 floats of this warp).
template <class T>
__device__ __forceinline__ void small_load(const T* p, const NsSmallArgs& a, int i0, int j0,
                                           float* turn, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const int i = i0 + lane;
  if (a.tall) {
    const T* at = p + static_cast<long long>(j0) * a.cols + i;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      v[k] = i < a.m && j0 + k < a.n ? static_cast<float>(at[static_cast<long long>(k) * a.cols])
                                     : 0.0f;
  } else if ((a.cols & 7) == 0 && j0 + 32 <= a.n) {
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = 0.0f;
    if (i >= a.m) return;
    const T* row = p + static_cast<long long>(i) * a.cols + j0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 f = reinterpret_cast<const float4*>(row)[q];
        v[4 * q] = f.x;
        v[4 * q + 1] = f.y;
        v[4 * q + 2] = f.z;
        v[4 * q + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = reinterpret_cast<const uint4*>(row)[q];
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          v[8 * q + 2 * h] = __uint_as_float(x[h] << 16);
          v[8 * q + 2 * h + 1] = __uint_as_float(x[h] & 0xffff0000u);
        }
      }
    }
  } else {
    const T* at = p + static_cast<long long>(i0) * a.cols + j0 + lane;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      v[k] = i0 + k < a.m && j0 + lane < a.n
                 ? static_cast<float>(at[static_cast<long long>(k) * a.cols])
                 : 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) turn[k * 33 + lane] = v[k];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = turn[lane * 33 + k];
    __syncwarp();
  }
}

// The same places written: T = float or bf16.
template <class T>
__device__ __forceinline__ void small_store(T* p, const NsSmallArgs& a, int i0, int j0, float* turn,
                                            const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const int i = i0 + lane;
  auto put = [](T* to, float x) {
    if constexpr (sizeof(T) == 4) *to = x;
    else *to = __float2bfloat16_rn(x);
  };
  if (a.tall) {
    T* at = p + static_cast<long long>(j0) * a.cols + i;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (i < a.m && j0 + k < a.n) put(at + static_cast<long long>(k) * a.cols, v[k]);
  } else if ((a.cols & 7) == 0 && j0 + 32 <= a.n) {
    if (i >= a.m) return;
    T* row = p + static_cast<long long>(i) * a.cols + j0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        reinterpret_cast<float4*>(row)[q] =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        reinterpret_cast<uint4*>(row)[q] =
            make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                       pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                       pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k) turn[lane * 33 + k] = v[k];
    __syncwarp();
    T* at = p + static_cast<long long>(i0) * a.cols + j0 + lane;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (i0 + k < a.m && j0 + lane < a.n)
        put(at + static_cast<long long>(k) * a.cols, turn[k * 33 + lane]);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kSmallThreads, 1)
    ns_small_kernel(const __grid_constant__ NsSmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xop = smem;
  uint8_t* aop = xop + kSmallX;
  uint8_t* pop = aop + kSmallA;
  uint8_t* part = pop + kSmallA;
  float* diag = reinterpret_cast<float*>(part + kSmallPart);  // d of A, then of P
  float* diag_p = diag + 128;
  float* norms = diag_p + 128;                                // [2][kSmallCluster]
  float* warp_sum = norms + 2 * kSmallCluster;                // [2][8]
  uint64_t* bar = reinterpret_cast<uint64_t*>(warp_sum + 16);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = warp >> 2;
  const int rank = static_cast<int>(cluster_ctarank());
  const int b = blockIdx.x / a.ctas;
  const int row = quarter * 32 + lane;
  const int col0 = rank * a.width;  // of X
  const int chunks = a.width / 32;
  const int mk = (a.m + 15) & ~15;  // rows (and k) that hold something
  float* turn = reinterpret_cast<float*>(part) + warp * (32 * 33);  // while part is idle

  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  // rows and columns of A' past m stay zero
  for (int i = threadIdx.x; i < kSmallA / 16; i += kSmallThreads)
    reinterpret_cast<uint4*>(aop)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 128) diag[threadIdx.x] = diag_p[threadIdx.x] = 0.0f;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t t_acc = tmem + lanes;         // columns [0, 256): accumulators
  const uint32_t t_x = tmem + lanes + 256u;    // columns [256, 512): X in fp32
  uint32_t phase = 0;
  // after the MMAs that thread 0 has issued
  auto wait_mma = [&]() {
    bool ok = false;
    for (int i = 0; i < kNsLooks && !ok; ++i) ok = mbar_test_wait(bar, phase);
    if (!ok) wait_bounded(bar, phase, abort_flag, a.status);
    phase ^= 1u;
    __syncwarp();
    tc_fence_after_sync();
  };
  // this CTA's shared-memory writes before its next MMAs
  auto to_mma = [&]() {
    fence_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  };

  // ---- the update U, its norm
  const long long base = static_cast<long long>(b) * a.rows * a.cols;
  NsSquares sq;
  for (int ch = half; ch < chunks; ch += 2) {
    const int j0 = col0 + ch * 32;
    float v[32];
    if (a.g_f32) small_load(static_cast<const float*>(a.g) + base, a, quarter * 32, j0, turn, v);
    else small_load(static_cast<const __nv_bfloat16*>(a.g) + base, a, quarter * 32, j0, turn, v);
    if (a.momentum != nullptr) {
      float mo[32];
      small_load(a.momentum + base, a, quarter * 32, j0, turn, mo);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        mo[k] = __fadd_rn(__fmul_rn(a.mu, mo[k]), v[k]);
        v[k] = a.nesterov ? __fadd_rn(v[k], __fmul_rn(a.mu, mo[k])) : mo[k];
      }
      small_store(a.momentum + base, a, quarter * 32, j0, turn, mo);
    }
    uint32_t r[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      sq.sum = fmaf(v[k], v[k], sq.sum);
      r[k] = __float_as_uint(v[k]);
    }
    tmem_st_32cols(t_x + static_cast<uint32_t>(32 * ch), r);
  }
  tmem_st_wait();
  const bool apart = a.eps < kNsPlainEps;
  if (apart) {  // the squares again, from tensor memory
    sq.sum = 0.0f;
    for (int ch = half; ch < chunks; ch += 2) {
      uint32_t r[32];
      float v[32];
      tmem_ld_32cols(t_x + static_cast<uint32_t>(32 * ch), r);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
      sq.add(v, true);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq.tiny += __shfl_xor_sync(0xffffffffu, sq.tiny, o);
    if (lane == 0) warp_sum[8 + warp] = sq.tiny;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq.sum += __shfl_xor_sync(0xffffffffu, sq.sum, o);
  if (lane == 0) warp_sum[warp] = sq.sum;
  __syncthreads();
  // every CTA of the cluster has started: its shared memory may be written
  cluster_sync();
  if (threadIdx.x < a.ctas) {
    float t = 0.0f;
    for (int w = 0; w < 8; ++w) t += warp_sum[w];
    st_cluster_f32(mapa_shared(smem_addr(&norms[rank]), threadIdx.x), t);
    if (apart) {
      t = 0.0f;
      for (int w = 8; w < 16; ++w) t += warp_sum[w];
      st_cluster_f32(mapa_shared(smem_addr(&norms[kSmallCluster + rank]), threadIdx.x), t);
    }
  }
  __syncwarp();
  cluster_sync();
  NsSquares all;
  for (int r = 0; r < a.ctas; ++r) all.sum += norms[r];
  if (apart)
    for (int r = 0; r < a.ctas; ++r) all.tiny += norms[kSmallCluster + r];
  const float inv = 1.0f / (all.norm() + a.eps);
  for (int ch = half; ch < chunks; ch += 2) {
    uint32_t r[32];
    tmem_ld_32cols(t_x + static_cast<uint32_t>(32 * ch), r);
    tmem_ld_wait();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __uint_as_float(r[8 * q + i]) * inv * a.scale0;
        r[8 * q + i] = __float_as_uint(x[i]);
      }
      *reinterpret_cast<uint4*>(xop + op_at(row, 4 * ch + q)) = float_to_half8(x);
    }
    tmem_st_32cols(t_x + static_cast<uint32_t>(32 * ch), r);
  }
  tmem_st_wait();

  for (int s = 0; s < a.steps; ++s) {
    const NsStep& f = a.step[s];
    const bool last = s + 1 == a.steps;
    // ---- gram
    to_mma();
    if (threadIdx.x == 0) {
      constexpr uint32_t idesc = instr_desc_f16(128, 128, false, false);
      for (int t = 0; t < a.width / 64; ++t) {
        const uint64_t d = smem_desc_sw128(xop + t * 16384);
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_mma(tmem, d + 2ull * k, d + 2ull * k, idesc, (t | k) != 0);
      }
      tc_commit(bar);
    }
    wait_mma();
    if (a.ctas == 1) {
      // the accumulators are the whole A
      if (quarter * 32 < mk) {
        for (int ch = half; ch * 32 < mk; ch += 2) {
          uint32_t r[32];
          tmem_ld_32cols(t_acc + static_cast<uint32_t>(32 * ch), r);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = f.gram_off * __uint_as_float(r[8 * q + i]);
            *reinterpret_cast<uint4*>(aop + op_at(row, 4 * ch + q)) = float_to_half8(x);
          }
          if (ch == quarter) {
            float acc = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) acc = lane == j ? __uint_as_float(r[j]) : acc;
            diag[row] = f.gram_diag * acc;
            *reinterpret_cast<__half*>(aop + op_at(row, row >> 3) + (row & 7) * 2) =
                __float2half_rn(0.0f);
          }
        }
      }
    } else {
      if (quarter * 32 < mk) {
        for (int ch = half; ch * 32 < mk; ch += 2) {
          uint32_t r[32];
          tmem_ld_32cols(t_acc + static_cast<uint32_t>(32 * ch), r);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(part + row * 512 + (((8 * ch + q) ^ (row & 7)) << 4)) =
                make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
        }
      }
      tc_fence_before_sync();
      cluster_sync();
      {
        // rows rank, rank + ctas, ... of the sum, 4 columns a thread
        const int per_row = mk / 4;
        const int items = ((mk - rank + a.ctas - 1) / a.ctas) * per_row;
        const uint32_t part0 = smem_addr(part);
        for (int it = threadIdx.x; it < items; it += kSmallThreads) {
          const int r = rank + (it / per_row) * a.ctas;
          const int q = it % per_row;
          const uint32_t at = part0 + static_cast<uint32_t>(r * 512 + ((q ^ (r & 7)) << 4));
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int p0 = 0; p0 < a.ctas; p0 += 8) {
            float4 w[8];
            // in turn from this CTA on, so that not all ask the same one at a time
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              int from = rank + p0 + p;
              if (from >= a.ctas) from -= a.ctas;
              w[p] = p0 + p < a.ctas ? ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(from)))
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              v.x += w[p].x;
              v.y += w[p].y;
              v.z += w[p].z;
              v.w += w[p].w;
            }
          }
          float x[4] = {v.x, v.y, v.z, v.w};
          float d = 0.0f;
          const bool has_d = r >= 4 * q && r < 4 * q + 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (4 * q + i == r) d = x[i] * f.gram_diag;
            x[i] = 4 * q + i == r ? 0.0f : x[i] * f.gram_off;
          }
          const __half2 h01 = __floats2half2_rn(x[0], x[1]), h23 = __floats2half2_rn(x[2], x[3]);
          const uint2 h = make_uint2(*reinterpret_cast<const uint32_t*>(&h01),
                                     *reinterpret_cast<const uint32_t*>(&h23));
          const uint32_t to = smem_addr(aop) + static_cast<uint32_t>(op_at(r, q >> 1) + (q & 1) * 8);
          const uint32_t dto = smem_addr(&diag[r]);
          for (int p = 0; p < a.ctas; ++p) {
            int dst = rank + p;
            if (dst >= a.ctas) dst -= a.ctas;
            st_cluster_u2(mapa_shared(to, static_cast<uint32_t>(dst)), h);
            if (has_d) st_cluster_f32(mapa_shared(dto, static_cast<uint32_t>(dst)), d);
          }
        }
      }
      // other CTAs' shared memory is written: ordered before their MMAs by this
      // fence, the cluster barrier and their own fence
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      cluster_sync();
    }
    // ---- poly
    to_mma();
    if (threadIdx.x == 0) {
      constexpr uint32_t idesc = instr_desc_f16(128, 128, false, false);
      for (int k = 0; k < mk / 16; ++k) {
        const uint64_t d = smem_desc_sw128(aop + (k >> 2) * 16384) + 2ull * (k & 3);
        tc_mma(tmem, d, d, idesc, k != 0);
      }
      tc_commit(bar);
    }
    wait_mma();
    if (quarter * 32 < mk) {
      const float di = diag[row];
      const float f_row = fmaf(f.poly_c, di, f.poly_b);
      for (int ch = half; ch * 32 < mk; ch += 2) {
        uint32_t r[32];
        tmem_ld_32cols(t_acc + static_cast<uint32_t>(32 * ch), r);
        uint4 before[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          before[q] = *reinterpret_cast<const uint4*>(aop + op_at(row, 4 * ch + q));
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float old[8], x[8];
          half8_to_float(before[q], old);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float dj = diag[32 * ch + 8 * q + i];
            x[i] = fmaf(old[i], fmaf(f.poly_c, dj, f_row),
                        f.poly_acc * __uint_as_float(r[8 * q + i]));
          }
          *reinterpret_cast<uint4*>(pop + op_at(row, 4 * ch + q)) = float_to_half8(x);
        }
        if (32 * ch == quarter * 32) {
          float acc = 0.0f;
#pragma unroll
          for (int j = 0; j < 32; ++j) acc = lane == j ? __uint_as_float(r[j]) : acc;
          float d = fmaf(f.diag_acc, acc, di * fmaf(f.c, di, f.b));
          __half h = __float2half_rn(0.0f);
          if (s < kNsEarly) {
            h = __float2half_rn(d * f.s_p);
            d -= __half2float(h) / f.s_p;  // what the rounding left
          }
          *reinterpret_cast<__half*>(pop + op_at(row, row >> 3) + (row & 7) * 2) = h;
          diag_p[row] = d;
        }
      }
    }
    // ---- apply
    to_mma();
    if (threadIdx.x == 0) {
      const uint32_t idesc = instr_desc_f16(128, a.width, false, true);
      for (int k = 0; k < mk / 16; ++k) {
        const uint64_t dp = smem_desc_sw128(pop + (k >> 2) * 16384) + 2ull * (k & 3);
        const uint64_t dx = smem_desc_sw128_mn16(xop) + 128ull * k;
        tc_mma(tmem, dp, dx, idesc, k != 0);
      }
      tc_commit(bar);
    }
    wait_mma();
    if (quarter * 32 < mk) {
      const float by_row = fmaf(f.d_x, diag_p[row], f.a_x);
      for (int ch = half; ch < chunks; ch += 2) {
        uint32_t r[32], o[32];
        tmem_ld_32cols(t_acc + static_cast<uint32_t>(32 * ch), r);
        tmem_ld_32cols(t_x + static_cast<uint32_t>(32 * ch), o);
        tmem_ld_wait();
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          x[j] = fmaf(by_row, __uint_as_float(o[j]), f.apply_acc * __uint_as_float(r[j]));
        if (!last) {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(x[j]);
          tmem_st_32cols(t_x + static_cast<uint32_t>(32 * ch), o);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float y[8] = {x[8 * q],     x[8 * q + 1], x[8 * q + 2], x[8 * q + 3],
                                x[8 * q + 4], x[8 * q + 5], x[8 * q + 6], x[8 * q + 7]};
            *reinterpret_cast<uint4*>(xop + op_at(row, 4 * ch + q)) = float_to_half8(y);
          }
        } else {
          const int j0 = col0 + 32 * ch;
          if (a.out_mode == kNsOutBf16) {
            small_store(static_cast<__nv_bfloat16*>(a.out) + base, a, quarter * 32, j0, turn, x);
          } else if (a.out_mode == kNsOutWeightBf16) {
            __nv_bfloat16* w = static_cast<__nv_bfloat16*>(a.out) + base;
            float old[32];
            small_load(w, a, quarter * 32, j0, turn, old);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = fmaf(a.keep, old[j], -a.move * x[j]);
            small_store(w, a, quarter * 32, j0, turn, x);
          } else {
            float* w = static_cast<float*>(a.out) + base;
            float old[32];
            small_load(w, a, quarter * 32, j0, turn, old);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = fmaf(a.keep, old[j], -a.move * x[j]);
            small_store(w, a, quarter * 32, j0, turn, x);
          }
        }
      }
      tmem_st_wait();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  // no CTA leaves while another may still read its shared memory
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace lmoe

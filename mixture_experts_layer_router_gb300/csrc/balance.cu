// The router's balance loss with per-expert counts, and its backward pass
// together with that of the gates.
//
// "The Training and RL Infrastructure Behind MAI-Thinking-1", section
// "Sharding and parallelism": a global-batch load-balancing loss; "Frontier
// Pre-training at Microsoft AI", section "Reducing per-expert overhead".
// Neither gives a formula; this is the usual product of load and mean
// probability, per sequence s of L tokens of which N_s count:
//   balance_s = E / (k N_s^2) sum_e counts[s,e] sum_t p[t,e]
//   z_s       = 1 / N_s sum_t lse_t^2,   lse_t = log sum_e exp(logit[t,e])
//   loss      = mean_s (balance_coef balance_s + z_coef z_s)
// The counts are integers, so only p and lse carry gradients:
//   d logit[t,e] = p_e (w_e - sum_f w_f p_f + q lse)   tokens that count
//                + the gates' part (see router_backward_kernel)
//   w_e = balance_coef E / (S k N_s^2) counts[s,e],  q = 2 z_coef / (S N_s)
//
// Both passes read the logits once (a row lives in the registers of the lanes
// that share it: softmax, sums and outputs need no second read) and are bound
// by memory traffic for large batches, by launch latency for small ones.
// Rows: LANES lanes of a warp hold one row, NV float4 a lane (E <= LANES NV 4),
// so a warp works on 32 / LANES rows at a time, U of those in flight.
// All sums over tokens are fp32 in a fixed order: lanes, warps, CTAs, groups
// of CTAs (integers may be added in any order).
//
// Measured (device time, inputs in turn: the last two larger than L2 together):
//                          loss                 backward with the gates' part
//   128 x 16, top-2        3.8 us
//   4096 x 64, top-4       8.5 us               3.4 us
//   16384 x 512, top-8    14.2 us (2.4 TB/s)   14.6 us (4.7 TB/s)
//   16 x 4096 x 256       20.7 us (3.3 TB/s)   25.9 us (5.3 TB/s, copy: 6.7)
// The loss: launch and one warp's chain, then two levels of sums over the CTAs (4
// us in all) and 16 warps an SM that issue about 0.6 instructions a cycle and
// scheduler; 24 or 32 warps leave too few registers for the rows in flight (slower).
// The backward: DRAM traffic, and the issue slots at 58 %.
#include <math.h>

#include "balance.h"
#include "kernels.h"
#include "ptx.cuh"

namespace lmoe {

namespace {

constexpr int kBalThreads = 512;  // E <= 512: a thread an expert in the tail
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalGroup = 16;  // CTAs whose partial sums one CTA adds
constexpr int kBackThreads = 128;

// How a row of E logits lies in a warp's registers.
template <int LANES_, int NV_, bool VEC_>
struct Row {
  static constexpr int LANES = LANES_;
  static constexpr int NV = NV_;
  static constexpr bool VEC = VEC_;
  static constexpr int N = 4 * NV;              // elements a lane
  static constexpr int ROWS = 32 / LANES;       // rows of a warp at once
  static constexpr int U = NV >= 3 ? 1 : 4 / NV;  // of those in flight
  static constexpr int BATCH = ROWS * U;
  static constexpr int WIDTH = LANES * N;       // columns covered, >= E
  static constexpr int J = (16 + LANES - 1) / LANES;  // choices a lane (loss; k <= 16)
  // column of element i of lane q
  __device__ static __forceinline__ int col(int q, int i) {
    return VEC ? 4 * (q + LANES * (i >> 2)) + (i & 3) : q + LANES * i;
  }
  __device__ static __forceinline__ void load(const float* row, int q, int E, float (&x)[N]) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = 4 * (q + LANES * v);
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (c < E) f = *reinterpret_cast<const float4*>(row + c);  // E % 4 == 0
        x[4 * v] = f.x;
        x[4 * v + 1] = f.y;
        x[4 * v + 2] = f.z;
        x[4 * v + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = q + LANES * i;
        x[i] = c < E ? row[c] : -INFINITY;
      }
    }
  }
};

struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// V values (1, 2 or 4) reduced over the LANES lanes of a row at once; every lane
// gets all results. Halves (quarters) of the lanes first take over one value
// each, so V = 4 takes 2 + 1 + (log2 LANES - 2) + 4 shuffles instead of 4 log2
// LANES. A fixed order.
template <int LANES, int V, class Op>
__device__ __forceinline__ void reduce_row(float (&v)[V], Op op) {
  static_assert(V == 1 || V == 2 || V == 4, "values");
  static_assert(LANES >= V, "lanes");
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  if constexpr (V == 1) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(kAll, v[0], o));
  } else if constexpr (V == 2) {
    const bool up = (lane & (LANES / 2)) != 0;
    float w = op(up ? v[1] : v[0], __shfl_xor_sync(kAll, up ? v[0] : v[1], LANES / 2));
#pragma unroll
    for (int o = LANES / 4; o > 0; o >>= 1) w = op(w, __shfl_xor_sync(kAll, w, o));
    v[0] = __shfl_sync(kAll, w, 0, LANES);
    v[1] = __shfl_sync(kAll, w, LANES / 2, LANES);
  } else {
    const bool up = (lane & (LANES / 2)) != 0;
    const float a = op(up ? v[2] : v[0], __shfl_xor_sync(kAll, up ? v[0] : v[2], LANES / 2));
    const float b = op(up ? v[3] : v[1], __shfl_xor_sync(kAll, up ? v[1] : v[3], LANES / 2));
    const bool up2 = (lane & (LANES / 4)) != 0;
    float w = op(up2 ? b : a, __shfl_xor_sync(kAll, up2 ? a : b, LANES / 4));
#pragma unroll
    for (int o = LANES / 8; o > 0; o >>= 1) w = op(w, __shfl_xor_sync(kAll, w, o));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(kAll, w, i * (LANES / 4), LANES);
  }
}

// Exponentials as powers of two: exp(x - max) = 2^(c (x - max)), c = log2 e. The
// difference comes first: as one fused multiply-add, 2^(c x - fl(c max)), the rounding
// of c max would stay in the exponent, harmless for ordinary logits (it is common to
// the row) but beyond fp32 from |max| of about 1e9 on, where masks of -1e10 or -1e30
// are. The special functions are the hardware's (2 ulp): errors of p stay below 5e-6
// for x within 32 of max, those of lse below 1e-6 + 2^-24 |max|.
constexpr float kLog2E = 1.44269504f;
constexpr float kLn2 = 0.693147181f;
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_of(float m, float x) { return pow2((x - m) * kLog2E); }
__device__ __forceinline__ float recip(float x) { return __fdividef(1.0f, x); }

// The maxima of a batch's rows (0 for a row of -inf alone).
template <class R>
struct Tops {
  float max[R::U];
  __device__ __forceinline__ explicit Tops(const float (&x)[R::U][R::N]) {
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      float m = x[u][0];
#pragma unroll
      for (int i = 1; i < R::N; ++i) m = fmaxf(m, x[u][i]);
      max[u] = m;
    }
    reduce_row<R::LANES>(max, Max());
#pragma unroll
    for (int u = 0; u < R::U; ++u)
      if (max[u] == -INFINITY) max[u] = 0.0f;
  }
  // x <- exp(x - max); the lane's part of the sum. A row of -inf alone sums to 0,
  // a NaN makes its row's sum NaN.
  __device__ __forceinline__ float exp_row(int u, float (&x)[R::N]) const {
    float s = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < R::N; ++i) x[i] = exp_of(max[u], x[i]);
#pragma unroll
    for (int i = 0; i < R::N; i += 2) {
      s += x[i];
      s2 += x[i + 1];
    }
    return s + s2;
  }
  // log sum exp of a row from its sum (about 1 or more)
  __device__ __forceinline__ float lse(int u, float sum) const {
    return fmaf(__log2f(sum), kLn2, max[u]);
  }
};

// Fixed-order sum over the block; every thread gets it. `buf`: kBalWarps floats.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  float t = lane < kBalWarps ? buf[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// True in every thread of the CTA that arrives last of `n` at *ticket; the
// others' global writes before their arrival are visible to it. The last one
// leaves the ticket at zero. One thread's release and acquire stand for the CTA:
// the barriers around it carry the other threads' writes and reads.
__device__ __forceinline__ bool arrive_last(unsigned* ticket, unsigned n, int* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(old)
                 : "l"(ticket)
                 : "memory");
    *flag = old == n - 1;
    if (old == n - 1) *ticket = 0;
  }
  __syncthreads();
  return *flag != 0;
}

// Without its coefficient z is no part of the loss: the square of an lse beyond 1.8e19
// is infinite, and 0 times that no number.
__device__ __forceinline__ void store_loss(float* loss, float balance, float z, float bc,
                                           float zc) {
  loss[0] = zc != 0.0f ? bc * balance + zc * z : bc * balance;
  loss[1] = balance;
  loss[2] = z;
}

}  // namespace

// What the loss reads for one batch of rows.
template <class R>
struct LossRows {
  float x[R::U][R::N];
  int id[R::U][R::J];
  bool in[R::U];
  int valid[R::U];  // compared when it is used: a comparison here would wait for the load
  __device__ __forceinline__ void load(const BalanceArgs& a, long long t0, int base, int r1, int q,
                                       int sub) {
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      const int r = base + u * R::ROWS + sub;
      const long long t = t0 + r;
      in[u] = r < r1;
      // a row past the part is read as the batch's first row (in range) and dropped
      R::load(a.logits + (in[u] ? t : t0 + base) * a.ld, q, a.E, x[u]);
#pragma unroll
      for (int j = 0; j < R::J; ++j) {
        const int c = q + R::LANES * j;
        id[u][j] = in[u] && c < a.k ? a.idx[t * a.k + c] : -1;
      }
      valid[u] = in[u] && a.valid != nullptr ? a.valid[t] : 1;
    }
  }
};

// Unit u: part u % parts of sequence u / parts. With one part a sequence the
// CTA has the sequence's sums itself; otherwise the last CTA of each group of
// kBalGroup parts adds the group's, and the last group of the sequence adds
// the groups'. The last sequence adds the sequences' losses.
template <class R>
__global__ void __launch_bounds__(kBalThreads, 1)
    balance_loss_kernel(const BalanceArgs a, const BalanceScratch w, int parts, int part_rows) {
  extern __shared__ float red[];  // [kBalWarps][E] column sums
  __shared__ int hist[512];
  __shared__ float warp_z[kBalWarps];
  __shared__ int warp_n[kBalWarps];
  __shared__ float buf[kBalWarps];
  __shared__ int flag;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % R::LANES, sub = lane / R::LANES;
  const int E = a.E, k = a.k;
  const int units = a.seqs * parts;
  // the loss from the sequences', by the CTA that arrives last of n
  auto last_sequence = [&](unsigned n) {
    if (!arrive_last(w.ticket + 2 * w.units, n, &flag)) return;
    float bs = 0.0f, zs = 0.0f;
    for (int i = threadIdx.x; i < a.seqs; i += kBalThreads) {
      bs += __ldcg(w.seq + 2ll * i);
      zs += __ldcg(w.seq + 2ll * i + 1);
    }
    bs = block_sum(bs, buf) / static_cast<float>(a.seqs);
    zs = block_sum(zs, buf) / static_cast<float>(a.seqs);
    if (threadIdx.x == 0) store_loss(a.loss, bs, zs, a.balance_coef, a.z_coef);
  };
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int s = unit / parts, part = unit - s * parts;
    for (int e = threadIdx.x; e < E; e += kBalThreads) hist[e] = 0;
    __syncthreads();
    const int r0 = part * part_rows;
    const int r1 = min(a.seq_len, r0 + part_rows);
    const long long t0 = static_cast<long long>(s) * a.seq_len;
    float acc[R::N];
#pragma unroll
    for (int i = 0; i < R::N; ++i) acc[i] = 0.0f;
    float zsum = 0.0f;
    int ntok = 0;
    bool bad = false;
    constexpr int kStride = kBalWarps * R::BATCH;
    int base = r0 + warp * R::BATCH;
    auto add = [&](LossRows<R>& cur) {
      const Tops<R> tops(cur.x);
      float sums[R::U];
#pragma unroll
      for (int u = 0; u < R::U; ++u) sums[u] = tops.exp_row(u, cur.x[u]);
      reduce_row<R::LANES>(sums, Add());
#pragma unroll
      for (int u = 0; u < R::U; ++u) {
        const float sum = sums[u];
        const bool ok = cur.in[u] && cur.valid[u] != 0 && !(sum == 0.0f);
        const float inv = recip(sum);
        if (ok) {
#pragma unroll
          for (int i = 0; i < R::N; ++i) acc[i] = fmaf(cur.x[u][i], inv, acc[i]);
          if (q == 0) {
            const float lse = tops.lse(u, sum);
            zsum = fmaf(lse, lse, zsum);
            ntok += 1;
          }
#pragma unroll
          for (int j = 0; j < R::J; ++j) {
            if (q + R::LANES * j < k) {
              const int id = cur.id[u][j];
              if (static_cast<unsigned>(id) < static_cast<unsigned>(E))
                atomicAdd(&hist[id], 1);
              else
                bad = true;
            }
          }
        }
      }
    };
    // two sets of registers in turn: the next batch's rows are on their way
    // while this one's are summed
    if (base < r1) {
      LossRows<R> even, odd;
      even.load(a, t0, base, r1, q, sub);
      while (true) {
        base += kStride;
        if (base < r1) odd.load(a, t0, base, r1, q, sub);
        add(even);
        if (base >= r1) break;
        base += kStride;
        if (base < r1) even.load(a, t0, base, r1, q, sub);
        add(odd);
        if (base >= r1) break;
      }
    }
    if (bad) atomicOr(a.status, kStatusBadExpert);
    // lanes of other rows, then warps
#pragma unroll
    for (int o = R::LANES; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < R::N; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      zsum += __shfl_xor_sync(0xffffffffu, zsum, o);
      ntok += __shfl_xor_sync(0xffffffffu, ntok, o);
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < R::N; ++i) {
        const int c = R::col(q, i);
        if (c < E) red[warp * E + c] = acc[i];
      }
    }
    if (lane == 0) {
      warp_z[warp] = zsum;
      warp_n[warp] = ntok;
    }
    __syncthreads();
    // thread e owns expert e from here on (E <= kBalThreads)
    const int e = threadIdx.x;
    float prob = 0.0f, z = 0.0f;
    int count = 0, n = 0;
    if (e < E) {
#pragma unroll
      for (int v = 0; v < kBalWarps; ++v) prob += red[v * E + e];
      count = hist[e];
    }
    for (int v = 0; v < kBalWarps; ++v) {
      z += warp_z[v];
      n += warp_n[v];
    }
    bool mine = true;  // this CTA holds the sequence's totals
    if (parts > 1) {
      const int groups = (parts + kBalGroup - 1) / kBalGroup;
      const int g = part / kBalGroup;
      int rows = min(kBalGroup, parts - g * kBalGroup);  // partial sums to add
      int first = s * parts + g * kBalGroup;
      int at = unit;
      unsigned* ticket = w.ticket + s * groups + g;
      // twice at most: the group's parts, then the sequence's groups
      for (int level = 0; level < 2 && mine; ++level) {
        if (rows > 1) {
          if (e < E) {
            w.prob[static_cast<long long>(at) * E + e] = prob;
            w.count[static_cast<long long>(at) * E + e] = count;
          }
          if (e == 0) {
            w.z[at] = z;
            w.tokens[at] = n;
          }
          mine = arrive_last(ticket, static_cast<unsigned>(rows), &flag);
          if (mine) {
            prob = 0.0f;
            count = 0;
            // the loads of a sum in flight at once
            float pv[kBalGroup];
            int cv[kBalGroup];
#pragma unroll
            for (int v = 0; v < kBalGroup; ++v) {
              const long long from = first + v;
              const bool has = v < rows && e < E;
              pv[v] = has ? __ldcg(w.prob + from * E + e) : 0.0f;
              cv[v] = has ? __ldcg(w.count + from * E + e) : 0;
            }
            z = lane < rows ? __ldcg(w.z + first + lane) : 0.0f;
            n = lane < rows ? __ldcg(w.tokens + first + lane) : 0;
#pragma unroll
            for (int v = 0; v < kBalGroup; ++v) {
              prob += pv[v];
              count += cv[v];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              z += __shfl_xor_sync(0xffffffffu, z, o);
              n += __shfl_xor_sync(0xffffffffu, n, o);
            }
          }
        }
        rows = groups;
        first = w.units + s * groups;
        at = first + g;
        ticket = w.ticket + w.units + s;
      }
    }
    if (mine) {
      const float inv = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
      float term = 0.0f;
      if (e < E) {
        a.counts[static_cast<long long>(s) * E + e] = count;
        a.prob_sum[static_cast<long long>(s) * E + e] = prob;
        if (n > 0) term = (static_cast<float>(count) * inv) * (prob * inv);
      }
      const float balance =
          block_sum(term, buf) * (static_cast<float>(E) / static_cast<float>(k));
      const float zmean = n > 0 ? z * inv : 0.0f;
      if (e == 0) {
        a.z_sum[s] = z;
        a.tokens[s] = n;
      }
      if (a.seqs == 1) {
        if (e == 0) store_loss(a.loss, balance, zmean, a.balance_coef, a.z_coef);
      } else {
        if (e == 0) {
          w.seq[2ll * s] = balance;
          w.seq[2ll * s + 1] = zmean;
        }
        if (parts > 1) last_sequence(static_cast<unsigned>(a.seqs));
      }
    }
    __syncthreads();
  }
  // a CTA with whole sequences arrives once for all of its own
  if (parts == 1 && a.seqs > 1) last_sequence(gridDim.x);
}

// Sums of other ranks or micro-batches added: one CTA, a warp per sequence.
__global__ void __launch_bounds__(kBalThreads)
    balance_from_stats_kernel(const int* counts, const float* prob_sum, const float* z_sum,
                              const int* tokens, int seqs, int E, int k, float bc, float zc,
                              float* loss) {
  __shared__ float buf[kBalWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float bs = 0.0f, zs = 0.0f;
  for (int s = warp; s < seqs; s += kBalWarps) {
    const int n = tokens[s];
    if (n <= 0) continue;
    const float inv = 1.0f / static_cast<float>(n);
    for (int e = lane; e < E; e += 32) {
      const long long at = static_cast<long long>(s) * E + e;
      bs = fmaf(static_cast<float>(counts[at]) * inv, prob_sum[at] * inv, bs);
    }
    if (lane == 0) zs = fmaf(z_sum[s], inv, zs);
  }
  bs = block_sum(bs, buf) * (static_cast<float>(E) / static_cast<float>(k)) /
       static_cast<float>(seqs);
  zs = block_sum(zs, buf) / static_cast<float>(seqs);
  if (threadIdx.x == 0) store_loss(loss, bs, zs, bc, zc);
}

// A warp's lanes over the choices of its batch of rows: `span` lanes (the power of
// two from k on) a row, one choice each, so one round covers 32 / span rows. (With
// the choices of a row on the row's own lanes, a round for every row: 16 x 4096 x
// 256 33.8 us instead of 25.4, 4096 x 64 5.0 instead of 3.4. In the loss, which
// does little with a choice, it is the other way round: 23.1 against 21.1 us.)
template <class R>
struct Choices {
  static constexpr int ROUNDS = R::BATCH > 2 ? R::BATCH / 2 : 1;  // k = 16
  int span, rounds, sub, c;
  __device__ __forceinline__ explicit Choices(int k) {
    const int lane = threadIdx.x & 31;
    const int shift = k > 1 ? 32 - __clz(k - 1) : 0;
    span = 1 << shift;
    rounds = ((R::BATCH << shift) + 31) >> 5;
    sub = lane >> shift;
    c = lane & (span - 1);
  }
  __device__ __forceinline__ int row(int round) const { return round * (32 / span) + sub; }
  // whether any of the row's lanes has it
  __device__ __forceinline__ bool any(bool has) const {
    return ((__ballot_sync(0xffffffffu, has) >> (sub * span)) & (0xffffffffu >> (32 - span))) != 0;
  }
  template <class Op>
  __device__ __forceinline__ float reduce(float v, Op op) const {
    for (int o = span >> 1; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
};

// What the backward reads for one batch of rows: the logits and, for the
// gates' part, the lane's choices, their gradients and their logits.
template <class R, bool GATES>
struct BackRows {
  static constexpr int ROUNDS = GATES ? Choices<R>::ROUNDS : 1;
  float x[R::U][R::N];
  int valid[R::U];
  int id[ROUNDS];
  float dg[ROUNDS], xi[ROUNDS];
  __device__ __forceinline__ void load(const RouterBackwardArgs& a, long long t0, int base, int r1,
                                       int q, int sub, const Choices<R>& ch) {
    if constexpr (GATES) {
#pragma unroll
      for (int p = 0; p < ROUNDS; ++p) {
        if (p >= ch.rounds) break;
        const int row = ch.row(p);
        const bool has = row < R::BATCH && base + row < r1 && ch.c < a.k;
        const long long at = (t0 + base + row) * a.k + ch.c;
        id[p] = has ? a.idx[at] : -1;
        dg[p] = has ? a.d_gates[at] : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      const int r = base + u * R::ROWS + sub;
      const bool in = r < r1;
      R::load(a.logits + (t0 + (in ? r : base)) * a.ld, q, a.E, x[u]);
      valid[u] = in && a.valid != nullptr ? a.valid[t0 + r] : 1;
    }
  }
  // after load: the choices' logits (ids outside [0, E): none, and no gradient)
  __device__ __forceinline__ void gather(const RouterBackwardArgs& a, long long t0, int base,
                                         const Choices<R>& ch) {
    if constexpr (GATES) {
#pragma unroll
      for (int p = 0; p < ROUNDS; ++p) {
        if (p >= ch.rounds) break;
        const bool has = static_cast<unsigned>(id[p]) < static_cast<unsigned>(a.E);
        if (!has) {  // its gradient, which may be anything, with it
          id[p] = -1;
          dg[p] = 0.0f;
        }
        xi[p] = has ? a.logits[(t0 + base + ch.row(p)) * a.ld + id[p]] : -INFINITY;
      }
    }
  }
};

// d_logits. The gates' part, with D = sum_j g_j dg_j over the token's choices:
//   g_j = p[idx_j]:            sum_{j: idx_j = e} g_j dg_j  -  p_e D
//   g_j = p[idx_j] / sum_i p[idx_i], i.e. a softmax over the chosen logits
//   alone (evaluated as that: no quotient of underflowed probabilities):
//                              sum_{j: idx_j = e} g_j (dg_j - D)
// A token whose d_gates are all zero has no gates' part, and one that does not count no
// loss's part, whatever its logits hold: by selection, because padding may hold NaN.
// The choices of a batch's rows are spread over the whole warp (see Choices), put
// their terms into the rows' shared copies (zero between batches), and every lane
// of a row picks up its own columns there.
// From three vectors a lane on the gates' form keeps the registers of six CTAs an SM (left
// alone it takes 95 and 121 instead of 80, and 16384 x 511, top-8, 16.9 instead of 15.7 us;
// with fewer vectors such a limit costs up to a tenth).
template <class R, bool GATES>
__global__ void __launch_bounds__(kBackThreads, GATES && R::NV > 2 ? 6 : 0)
    router_backward_kernel(const RouterBackwardArgs a, int parts, int part_rows) {
  extern __shared__ float back_smem[];  // [warps][BATCH][WIDTH], [warps][BATCH][2]
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % R::LANES, sub = lane / R::LANES;
  const int E = a.E, k = a.k;
  float* sparse = back_smem + warp * (R::BATCH * R::WIDTH);
  float2* stat = reinterpret_cast<float2*>(back_smem + (kBackThreads / 32) * R::BATCH * R::WIDTH) +
                 warp * R::BATCH;  // max and 1 / sum of a row, then the sum of its terms
  if (GATES) {
    for (int i = lane; i < R::BATCH * R::WIDTH; i += 32) sparse[i] = 0.0f;
    __syncwarp();
  }
  const Choices<R> ch(k);
  const int s = blockIdx.x / parts, part = blockIdx.x - s * parts;
  const int r0 = part * part_rows;
  const int r1 = min(a.seq_len, r0 + part_rows);
  const long long t0 = static_cast<long long>(s) * a.seq_len;
  // w_e = c counts[s,e]; q lse: zq lse
  const int n = a.tokens[s];
  const float up = (a.d_loss != nullptr ? *a.d_loss : 1.0f) / static_cast<float>(a.seqs);
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  const float wc =
      up * a.balance_coef * (static_cast<float>(E) / static_cast<float>(k)) * inv_n * inv_n;
  const float zq = up * 2.0f * a.z_coef * inv_n;
  float wt[R::N];
#pragma unroll
  for (int i = 0; i < R::N; ++i) {
    const int c = R::col(q, i);
    wt[i] = c < E ? wc * static_cast<float>(a.counts[static_cast<long long>(s) * E + c]) : 0.0f;
  }
  constexpr int kStride = (kBackThreads / 32) * R::BATCH;
  // where there are registers for a second batch its rows are on their way while
  // the first one's are worked on
  constexpr bool kAhead = R::BATCH <= 8;
  BackRows<R, GATES> cur;
  int base = r0 + warp * R::BATCH;
  if (kAhead && base < r1) cur.load(a, t0, base, r1, q, sub, ch);
  for (; base < r1; base += kStride) {
    BackRows<R, GATES> next;
    if constexpr (kAhead) {
      if (base + kStride < r1) next.load(a, t0, base + kStride, r1, q, sub, ch);
    } else {
      cur.load(a, t0, base, r1, q, sub, ch);
    }
    cur.gather(a, t0, base, ch);
    const Tops<R> tops(cur.x);
    // the rows' sums and sums of w e
    float sum[R::U], dot[R::U];
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      sum[u] = tops.exp_row(u, cur.x[u]);
      dot[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < R::N; ++i) dot[u] = fmaf(cur.x[u][i], wt[i], dot[u]);
    }
    if constexpr (R::U == 1) {
      float v[2] = {sum[0], dot[0]};
      reduce_row<R::LANES>(v, Add());
      sum[0] = v[0];
      dot[0] = v[1];
    } else {
#pragma unroll
      for (int u = 0; u < R::U; u += 2) {
        float v[4] = {sum[u], dot[u], sum[u + 1], dot[u + 1]};
        reduce_row<R::LANES>(v, Add());
        sum[u] = v[0];
        dot[u] = v[1];
        sum[u + 1] = v[2];
        dot[u + 1] = v[3];
      }
    }
    float inv[R::U];
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      inv[u] = sum[u] == 0.0f ? 0.0f : recip(sum[u]);
      if (GATES && !a.renorm && q == 0)
        stat[u * R::ROWS + sub] = make_float2(tops.max[u], inv[u]);
    }
    if constexpr (GATES) {
      if (!a.renorm) __syncwarp();
#pragma unroll
      for (int p = 0; p < BackRows<R, GATES>::ROUNDS; ++p) {
        if (p >= ch.rounds) break;
        const int row = ch.row(p);
        const bool live = ch.any(cur.dg[p] != 0.0f);
        const bool has = live && cur.id[p] >= 0;
        float g = 0.0f, term;
        if (a.renorm) {
          float own = ch.reduce(cur.xi[p], Max());
          if (own == -INFINITY) own = 0.0f;
          if (has) g = exp_of(own, cur.xi[p]);
          const float gs = ch.reduce(g, Add());
          const float gd = ch.reduce(g * cur.dg[p], Add());
          const float ginv = gs == 0.0f ? 0.0f : recip(gs);
          term = g * ginv * (cur.dg[p] - gd * ginv);
        } else {
          const float2 st = row < R::BATCH ? stat[row] : make_float2(0.0f, 0.0f);
          if (has) g = exp_of(st.x, cur.xi[p]) * st.y;
          term = g * cur.dg[p];
          const float gd = ch.reduce(term, Add());
          __syncwarp();
          if (ch.c == 0 && row < R::BATCH) stat[row].x = gd;
        }
        // A token's choices differ as a rule, which every lane sees when it finds
        // its own mark; given choices may repeat, and then their terms are added in
        // the order of the choices.
        float* at = sparse + (has ? row * R::WIDTH + cur.id[p] : 0);
        if (has) *at = static_cast<float>(lane);
        __syncwarp();
        const bool own_mark = !has || *at == static_cast<float>(lane);
        if (__all_sync(0xffffffffu, own_mark)) {
          if (has) *at = term;
        } else {
          if (has) *at = 0.0f;
          __syncwarp();
          for (int o = 0; o < ch.span; ++o) {
            if (has && ch.c == o) *at += term;
            __syncwarp();
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      const int r = base + u * R::ROWS + sub;
      const bool in = r < r1;
      // p_e (wt_e + shift)
      const bool on = in && cur.valid[u] != 0 && sum[u] != 0.0f;
      float shift = on ? fmaf(zq, tops.lse(u, sum[u]), -dot[u] * inv[u]) : 0.0f;
      if (GATES && !a.renorm) shift -= stat[u * R::ROWS + sub].x;
      // With e_e = p_e / inv as e_e (wt_e inv + shift inv): two multiply-adds an element,
      // the gates' terms included. A token that does not count gets no loss's part.
      const bool dense = on || shift != 0.0f;
      const float wi = on ? inv[u] : 0.0f, si = shift * inv[u];
      float* mine = sparse + (u * R::ROWS + sub) * R::WIDTH;
      float d[R::N];
#pragma unroll
      for (int v = 0; v < R::NV; ++v) {
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (GATES && R::VEC) {
          float4* at = reinterpret_cast<float4*>(mine + 4 * (q + R::LANES * v));
          const float4 o = *at;
          *at = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          f[0] = o.x;
          f[1] = o.y;
          f[2] = o.z;
          f[3] = o.w;
        } else if constexpr (GATES) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = mine[R::col(q, 4 * v + i)];
            mine[R::col(q, 4 * v + i)] = 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = cur.x[u][4 * v + i];
          d[4 * v + i] = dense ? fmaf(e, fmaf(wt[4 * v + i], wi, si), f[i]) : f[i];
        }
      }
      if (in) {
        float* out = a.d_logits + (t0 + r) * a.ldd;
        if constexpr (R::VEC) {
#pragma unroll
          for (int v = 0; v < R::NV; ++v) {
            const int c = 4 * (q + R::LANES * v);
            if (c < E)
              *reinterpret_cast<float4*>(out + c) =
                  make_float4(d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < R::N; ++i) {
            const int c = q + R::LANES * i;
            if (c < E) out[c] = d[i];
          }
        }
      }
    }
    if constexpr (GATES) __syncwarp();
    if constexpr (kAhead) cur = next;
  }
}

namespace {

int div_up(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

template <class R>
cudaError_t loss_impl(const BalanceArgs& a, const BalanceScratch& w, cudaStream_t s) {
  const int smem = kBalWarps * a.E * 4;
  static bool set[kMaxDevices] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        balance_loss_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBalWarps * 512 * 4);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  // parts of a sequence: as many CTAs as there are for each, no more than give
  // every warp a batch of rows
  int parts = w.units / a.seqs;
  const int most = div_up(a.seq_len, kBalWarps * R::BATCH);
  if (parts > most) parts = most;
  if (parts > kBalGroup * kBalGroup) parts = kBalGroup * kBalGroup;  // two levels of sums
  if (parts < 1) parts = 1;
  const int part_rows = div_up(a.seq_len, parts);
  parts = div_up(a.seq_len, part_rows);
  const long long units = static_cast<long long>(a.seqs) * parts;
  const int grid = static_cast<int>(units < w.units ? units : w.units);
  return launch_kernel(balance_loss_kernel<R>, dim3(grid), dim3(kBalThreads), smem, s, 1, false, a,
                       w, parts, part_rows);
}

template <class R, bool GATES>
cudaError_t backward_impl(const RouterBackwardArgs& a, int sms, cudaStream_t s) {
  constexpr int warps = kBackThreads / 32;
  const int smem = GATES ? warps * R::BATCH * (R::WIDTH + 2) * 4 : 0;
  static int resident_of[kMaxDevices] = {};
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (resident_of[dev] == 0) {
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &n, router_backward_kernel<R, GATES>, kBackThreads, smem);
    if (e != cudaSuccess) return e;
    resident_of[dev] = n > 0 ? n : 1;
  }
  // parts of a sequence: a batch of rows for every warp, but no more CTAs in
  // all than the SMs hold at once
  const int slots = resident_of[dev] * sms;
  int parts = div_up(a.seq_len, warps * R::BATCH);
  if (parts > slots / a.seqs) parts = slots / a.seqs;
  if (parts < 1) parts = 1;
  const int part_rows = div_up(a.seq_len, parts);
  parts = div_up(a.seq_len, part_rows);
  return launch_kernel(router_backward_kernel<R, GATES>,
                       dim3(static_cast<unsigned>(a.seqs) * static_cast<unsigned>(parts)),
                       dim3(kBackThreads), smem, s, 1, false, a, parts, part_rows);
}

// The layout for E experts: the fewest lanes that hold a row in one float4
// each, then more float4 a lane.
template <bool VEC, class F>
cudaError_t with_row(int E, const F& f) {
  if (E <= 16) return f(Row<4, 1, VEC>());
  if (E <= 32) return f(Row<8, 1, VEC>());
  if (E <= 64) return f(Row<16, 1, VEC>());
  if (E <= 128) return f(Row<32, 1, VEC>());
  if (E <= 256) return f(Row<32, 2, VEC>());
  if (E <= 384) return f(Row<32, 3, VEC>());
  return f(Row<32, 4, VEC>());
}

}  // namespace

cudaError_t launch_balance_loss(const BalanceArgs& a, const BalanceScratch& w, cudaStream_t s) {
  const auto go = [&](auto r) { return loss_impl<decltype(r)>(a, w, s); };
  // float4 loads: rows that start on 16 bytes and end on whole vectors
  return a.E % 4 == 0 && a.ld % 4 == 0 ? with_row<true>(a.E, go) : with_row<false>(a.E, go);
}

cudaError_t launch_balance_from_stats(const int* counts, const float* prob_sum, const float* z_sum,
                                      const int* tokens, int seqs, int E, int k,
                                      float balance_coef, float z_coef, float* loss,
                                      cudaStream_t s) {
  return launch_kernel(balance_from_stats_kernel, dim3(1), dim3(kBalThreads), 0, s, 1, false,
                       counts, prob_sum, z_sum, tokens, seqs, E, k, balance_coef, z_coef, loss);
}

cudaError_t launch_router_backward(const RouterBackwardArgs& a, int sms, cudaStream_t s) {
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && a.ldd % 4 == 0;
  if (a.d_gates != nullptr) {
    const auto go = [&](auto r) { return backward_impl<decltype(r), true>(a, sms, s); };
    return vec ? with_row<true>(a.E, go) : with_row<false>(a.E, go);
  }
  const auto go = [&](auto r) { return backward_impl<decltype(r), false>(a, sms, s); };
  return vec ? with_row<true>(a.E, go) : with_row<false>(a.E, go);
}

}  // namespace lmoe

// Launchers of the router's balance loss and backward (internal interface).
#pragma once

#include <cuda_runtime.h>

namespace lmoe {

// Scratch of the balance loss (device memory): partial sums of the CTAs that
// share a sequence, the sequences' loss terms, and arrival counters that are
// zero before the first launch and that every launch leaves at zero.
struct BalanceScratch {
  float* prob;      // [2 * units, E]: CTAs, then groups of CTAs
  int* count;       // [2 * units, E]
  float* z;         // [2 * units]
  int* tokens;      // [2 * units]
  float* seq;       // [2, max_tokens]: balance and z of each sequence
  unsigned* ticket; // [2 * units + 1]
  int units;        // CTAs that may share sequences (one per SM)
};

struct BalanceArgs {
  const float* logits;
  long long ld;
  const int* idx;
  const unsigned char* valid;  // may be null
  int seqs, seq_len, E, k;
  float balance_coef, z_coef;
  int* counts;     // [seqs, E]
  float* prob_sum; // [seqs, E]
  float* z_sum;    // [seqs]
  int* tokens;     // [seqs]
  float* loss;     // [3]
  unsigned* status;
};
cudaError_t launch_balance_loss(const BalanceArgs& a, const BalanceScratch& w, cudaStream_t s);

// loss [3] from counts, prob_sum, z_sum and tokens of `seqs` sequences.
cudaError_t launch_balance_from_stats(const int* counts, const float* prob_sum, const float* z_sum,
                                      const int* tokens, int seqs, int E, int k,
                                      float balance_coef, float z_coef, float* loss,
                                      cudaStream_t s);

struct RouterBackwardArgs {
  const float* logits;
  long long ld;
  const int* idx;              // may be null without d_gates
  const float* d_gates;        // [T, k], may be null
  const unsigned char* valid;  // may be null
  const int* counts;           // [seqs, E]
  const int* tokens;           // [seqs]
  const float* d_loss;         // [1], may be null: 1
  int seqs, seq_len, E, k;
  bool renorm;
  float balance_coef, z_coef;
  float* d_logits;
  long long ldd;
};
cudaError_t launch_router_backward(const RouterBackwardArgs& a, int sms, cudaStream_t s);

}  // namespace lmoe

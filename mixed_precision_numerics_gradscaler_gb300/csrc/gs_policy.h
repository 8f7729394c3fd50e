// gs_policy.h -- arguments and workspace of the policy loss.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gs {

// CTAs that may leave partial sums.
constexpr int kPolicyCtas = 2048;

struct PolicyPart {
  double loss, ratio, kl;
  unsigned long long held;
};
// Counts and arrivals; zero at the start of a call's kernels.
struct PolicyHead {
  unsigned long long tokens, seqs;
  unsigned int arrived[2];
  unsigned int pad[10];
};
static_assert(sizeof(PolicyHead) == 64, "the counts behind it are 8-byte aligned");

// Words of a mask of T tokens, in runs of 256.
inline int64_t policy_mask_words(int64_t T) { return (T + 255) / 256 * 8; }

// A real number as the sum of two fp32 ones.
struct Border {
  float hi, lo;
};

struct PolicyArgs {
  const float *logprob, *old, *ref, *adv;  // ref may be null
  const int64_t *targets, *offsets;        // either may be null
  const float* dloss;
  float *loss, *stats, *grad;              // stats, grad may be null
  int64_t T, S;
  int reduction;
  bool adv_per_seq;
  bool counted;                            // head->tokens holds the tokens that count
  Border high, low, dual;                  // logarithms of the three borders
  float factor_high, factor_low, factor_dual, kl;
  PolicyHead* head;
  unsigned long long* n;                   // tokens that count, by sequence
  unsigned* mask;                          // a bit per token, where there are targets
  PolicyPart* part;
};

cudaError_t launch_policy_loss(PolicyArgs a, cudaStream_t st);

}  // namespace gs

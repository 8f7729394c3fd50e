// policy_loss.cu -- the clipped policy loss with a divergence term over packed
// sequences, and its gradient with respect to the tokens' log probabilities.
//
// For a token with log probability x, x' under the policy that sampled it, x''
// under the reference, advantage A:
//   d = x - x',  rho = e^d,  y = x'' - x,
//   l = -obj + kl (e^y - 1 - y),
//   obj = rho A, but (1 + clip_high) A where A > 0 and d > log(1 + clip_high),
//         (1 - clip_low) A where A < 0 and d < log(1 - clip_low), and
//         dual_clip A where A < 0 and d > log(dual_clip);
//   dl/dx = -(rho A, or 0 where obj is held) - kl (e^y - 1),
// and loss = sum w l with w = 1/N, 1/(S' n_s) or 1 (N tokens that count in all,
// n_s in the token's sequence, S' sequences that have any).
//
// Whether a token is held is a comparison of d, not of the rounded ratio: d is
// formed as an unevaluated sum of two fp32 numbers (the rounding error of a
// difference is itself an fp32 number; O. Moller, "Quasi double-precision in
// floating point addition", 1965) and compared with the logarithm in the same
// form, so that the border lies where the real numbers put it, as 2^-48.
// e^y - 1 - y is summed as a series below 1/2, where the difference would keep
// few digits of a quadratic.
//
// One pass reads 8 to 24 bytes per token and writes 4: HBM is the bound of a
// long batch.  The gradient's weights need the counts first: a pass over the
// targets alone (8 bytes per token) counts them with integer additions, whose
// order changes nothing, and leaves a bit per token for the pass over the rest.
// Sums: eight tokens' terms in fp32, a thread's sums with their rounding errors
// carried along, everything beyond in fp64, joined in a fixed order by the last
// CTA to finish.  A thread that meets a term of 2^100 or more, Inf or NaN takes its
// tokens once more in fp64.  Short batches are done by one CTA,
// which counts and sums in one launch.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gs_internal.h"
#include "gs_policy.h"
#include "gsfp8.h"

namespace gs {

constexpr int kPThreads = 256;
constexpr int kPRun = 8;                     // tokens per thread and step
constexpr int kPTile = kPThreads * kPRun;    // tokens per CTA and step
constexpr int kPSpan = 1024;                 // sequences of a step kept in shared memory

// Tokens that one CTA does alone, and their sequences.  Alone and by many CTAs, in
// two or three launches, on the device: 1024 tokens 7.0 and 14.4 us, 5120 11.1 and
// 14.5 (13.4 and 21.5 by sequences), 4608 in 2048 sequences 15.5 and 30.1.  8192 alone
// take 14.9 where many CTAs take 14.4 (18.5 and 22.6 by sequences), and eight tokens a
// thread spill: 5120 tokens then take 13.7.
constexpr int64_t kPSmallTokens = 5120;
constexpr int64_t kPSmallSeqs = 2048;  // times kPSmallTokens: below 2^24, exact in fp32
constexpr int kPSmallThreads = 1024;

// A sum in fp32 with its rounding errors carried along (the fp64 pipe would
// take as long as everything else here).
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), w = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, w)), __fsub_rn(v, w)));
    hi = s;
  }
  // Takes in the sum of the lane o further on.
  __device__ __forceinline__ void merge(int o) {
    const float h = __shfl_down_sync(0xFFFFFFFFu, hi, o), l = __shfl_down_sync(0xFFFFFFFFu, lo, o);
    add(h);
    lo = __fadd_rn(lo, l);
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

struct Sums {
  double loss, ratio, kl;
  unsigned long long held;
};
// Sums from here on (and Inf and NaN) are a thread's in fp64: fp32 pairs of them could
// leave its range, where the error of an addition would become Inf - Inf.  Below,
// 2^27 of them fit into a pair.
constexpr float kPFar = 0x1p100f;
__device__ __forceinline__ bool is_far(float v) { return !(fabsf(v) < kPFar); }
// Adds N (a power of two) lanes' sums; the result in lane 0.
template <int N>
__device__ __forceinline__ Sums warp_sums(Sums s) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    s.loss += __shfl_down_sync(0xFFFFFFFFu, s.loss, o);
    s.ratio += __shfl_down_sync(0xFFFFFFFFu, s.ratio, o);
    s.kl += __shfl_down_sync(0xFFFFFFFFu, s.kl, o);
    s.held += __shfl_down_sync(0xFFFFFFFFu, s.held, o);
  }
  return s;
}

// The first s in [lo, hi] with end[s] > t (hi where none is), end = offsets + 1.
__device__ __forceinline__ int64_t seq_of(const int64_t* __restrict__ end, int64_t lo, int64_t hi,
                                          int64_t t) {
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (end[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
// The same by a whole warp, 32 probes a round (three rounds for 32768
// sequences, where one lane would wait for fifteen loads in turn).
__device__ __forceinline__ int64_t seq_of_warp(const int64_t* __restrict__ end, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n - 1;
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + step * lane;
    const bool after = at >= hi || end[at] > t;
    const unsigned m = __ballot_sync(0xFFFFFFFFu, after);
    // the first probe after t bounds it above, the one before it below
    const int first = m ? __ffs(m) - 1 : 32;
    const int64_t above = first < 32 ? min(hi, lo + step * first) : hi;
    lo = first > 0 ? min(hi, lo + step * (first - 1) + 1) : lo;
    hi = above;
  }
  return lo;
}

// x - y as d + e exactly (e undefined where d is not finite).
__device__ __forceinline__ void two_diff(float x, float y, float& d, float& e) {
  d = __fsub_rn(x, y);
  const float v = __fsub_rn(d, x);
  e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, v)), __fadd_rn(y, v));
}
__device__ __forceinline__ bool above(float d, float e, const Border& b) {
  return d > b.hi || (d == b.hi && e > b.lo);
}
__device__ __forceinline__ bool below(float d, float e, const Border& b) {
  return d < b.hi || (d == b.hi && e < b.lo);
}

// e^y - 1, and e^y - 1 - y: y^2 (1/2 + y/6 + ... + y^7/9!), cut off at 2e-9 of
// it, for |y| <= 1/2; beyond, e^y - 1 keeps its digits but for two bits.
__device__ __forceinline__ void exp_less(float y, float& em1, float& em1y) {
  float p = 1.0f / 362880.0f;
  p = __fmaf_rn(p, y, 1.0f / 40320.0f);
  p = __fmaf_rn(p, y, 1.0f / 5040.0f);
  p = __fmaf_rn(p, y, 1.0f / 720.0f);
  p = __fmaf_rn(p, y, 1.0f / 120.0f);
  p = __fmaf_rn(p, y, 1.0f / 24.0f);
  p = __fmaf_rn(p, y, 1.0f / 6.0f);
  p = __fmaf_rn(p, y, 0.5f);
  p = __fmul_rn(__fmul_rn(y, y), p);
  const bool near = fabsf(y) <= 0.5f;
  const float far_em1 = __fsub_rn(expf(y), 1.0f);
  em1 = near ? __fadd_rn(y, p) : far_em1;
  em1y = near ? p : __fsub_rn(far_em1, y);
}

struct Token {
  float value, slope, ratio, kl;  // l and dl/dx without the weight
  float rest;                     // EXACT: l is value + rest
  bool held;
};
// EXACT: the objective as a sum of two fp32 numbers, A and A (rho - 1) or the
// parts of a product: advantages that cancel over a batch leave a loss far smaller
// than its terms.
template <bool REF, bool EXACT>
__device__ __forceinline__ Token token(const PolicyArgs& a, float x, float old, float ref, float adv) {
  Token t;
  float d, e;
  two_diff(x, old, d, e);
  float em1 = 0.0f, unused;
  if constexpr (EXACT) {
    exp_less(d, em1, unused);
    t.ratio = fabsf(d) <= 0.5f ? __fadd_rn(1.0f, em1) : expf(d);
    if (fabsf(d) <= 0.5f) em1 = __fmaf_rn(e, t.ratio, em1);  // (e is a number there)
  } else {
    t.ratio = expf(d);
  }
  const bool gains = adv > 0.0f, loses = adv < 0.0f;
  const Border top = gains ? a.high : a.dual;
  const bool over = (gains || loses) && above(d, e, top);
  const bool under = loses && below(d, e, a.low);
  t.held = over || under;
  const float factor = over ? (gains ? a.factor_high : a.factor_dual) : under ? a.factor_low : t.ratio;
  // (a ratio beyond fp32 times 0 is NaN here, and 0 in fp64: see FarToken)
  const float obj = __fmul_rn(factor, adv);
  t.slope = t.held ? 0.0f : -obj;
  t.kl = 0.0f;
  t.value = -obj;
  t.rest = 0.0f;
  if constexpr (EXACT) {
    if (t.held) {
      t.rest = __fmaf_rn(-factor, adv, obj);
    } else if (fabsf(d) <= 0.5f && adv != 0.0f) {
      t.value = -adv;
      t.rest = -__fmul_rn(adv, em1);
    }
  }
  if constexpr (REF) {
    const float y = __fsub_rn(ref, x);
    float em1y;
    exp_less(y, em1y, t.kl);
    // (a divergence without a coefficient is watched alone: it may be infinite)
    if (a.kl != 0.0f) {
      if constexpr (EXACT) t.rest = __fmaf_rn(a.kl, t.kl, t.rest);
      else t.value = __fmaf_rn(a.kl, t.kl, t.value);
      t.slope = __fmaf_rn(-a.kl, em1y, t.slope);
    }
  }
  return t;
}

// The same in fp64, for terms that fp32 has no room for (an exponential beyond its
// range whose mean is inside it, say): what is held, and at which factor, is decided
// as above.
struct FarToken {
  double value, slope, ratio, kl;
};
__device__ __noinline__ FarToken far_token(const PolicyArgs& a, float x, float old, float ref, float adv) {
  FarToken t;
  float d, e;
  two_diff(x, old, d, e);
  const double diff = (double)x - (double)old;
  t.ratio = exp(diff);
  const bool gains = adv > 0.0f, loses = adv < 0.0f;
  const bool over = (gains || loses) && above(d, e, gains ? a.high : a.dual);
  const bool under = loses && below(d, e, a.low);
  const double factor = over ? (gains ? a.factor_high : a.factor_dual) : under ? (double)a.factor_low : t.ratio;
  // (a finite ratio times 0, whatever exp(diff) makes of it)
  const double obj = adv == 0.0f && isfinite(diff) ? 0.0 : factor * (double)adv;
  t.value = -obj;
  t.slope = over || under ? 0.0 : -obj;
  t.kl = 0.0;
  if (a.ref) {
    const double y = (double)ref - (double)x, em1 = expm1(y);
    t.kl = em1 - y;
    if (a.kl != 0.0f) {
      t.value += (double)a.kl * t.kl;
      t.slope -= (double)a.kl * em1;
    }
  }
  return t;
}
// What a thread sums in fp64 after all, because a part of it was far: all of its
// tokens' terms, once more from the start (rare, and nothing of it is held in the
// loops over tokens).  With kFarLoss their gradients are written again too.
enum { kFarLoss = 1, kFarRatio = 2, kFarKl = 4 };
struct Far {
  unsigned which = 0;
  double loss = 0.0, ratio = 0.0, kl = 0.0;
  __device__ __forceinline__ void see(float loss, float ratio, float kl) {
    which |= (is_far(loss) ? kFarLoss : 0u) | (is_far(ratio) ? kFarRatio : 0u) | (is_far(kl) ? kFarKl : 0u);
  }
  // Token t, with the weight in the loss and the gradient's factor.
  __device__ __forceinline__ void add(const PolicyArgs& a, int64_t t, float adv, double w, double up) {
    const FarToken f = far_token(a, a.logprob[t], a.old[t], a.ref ? a.ref[t] : 0.0f, adv);
    if (which & kFarLoss) {
      loss += w * f.value;
      if (a.grad) a.grad[t] = (float)(up * f.slope);
    }
    if (which & kFarRatio) ratio += f.ratio;
    if (which & kFarKl) kl += f.kl;
  }
};

// Adds a block's sums, the threads' as fp32 pairs within a warp (512 threads'
// additions in fp64 would take 2 us), the warps' in fp64; the result in thread 0.
// far: sums of this thread that take the place of its pairs.
template <int NT>
__device__ __forceinline__ Sums block_sums(Pair loss, Pair ratio, Pair kl, unsigned long long held, const Far& far) {
  __shared__ Sums red[NT / 32];
  if (far.which & kFarLoss) loss = Pair{0.0f, 0.0f};
  if (far.which & kFarRatio) ratio = Pair{0.0f, 0.0f};
  if (far.which & kFarKl) kl = Pair{0.0f, 0.0f};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    loss.merge(o);
    ratio.merge(o);
    kl.merge(o);
    held += __shfl_down_sync(0xFFFFFFFFu, held, o);
  }
  Sums own = {loss.value(), ratio.value(), kl.value(), held};
  if (__any_sync(0xFFFFFFFFu, far.which != 0)) {
    const Sums w = warp_sums<32>(Sums{far.loss, far.ratio, far.kl, 0ull});
    own = Sums{own.loss + w.loss, own.ratio + w.ratio, own.kl + w.kl, held};
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = own;
  __syncthreads();
  Sums s = {0.0, 0.0, 0.0, 0ull};
  if (threadIdx.x < 32) {
    if (threadIdx.x < NT / 32) s = red[threadIdx.x];
    s = warp_sums<NT / 32>(s);
  }
  __syncthreads();
  return s;
}

// The loss and the statistics from the sums (one thread).
__device__ __forceinline__ void finish(const PolicyArgs& a, const Sums& s, unsigned long long n) {
  const double each = n ? 1.0 / (double)n : 0.0;
  *a.loss = (float)(a.reduction == GS_LOSS_TOKEN_MEAN ? s.loss * each : s.loss);
  if (a.stats) {
    a.stats[0] = (float)n;
    a.stats[1] = (float)(s.ratio * each);
    a.stats[2] = (float)((double)s.held * each);
    a.stats[3] = (float)(s.kl * each);
  }
}

// First and one past the last token that lies in a sequence.
__device__ __forceinline__ void token_range(const PolicyArgs& a, int64_t& lo, int64_t& hi) {
  lo = 0;
  hi = a.T;
  if (a.offsets) {
    lo = max((int64_t)0, min(a.T, a.offsets[0]));
    hi = max(lo, min(a.T, a.offsets[a.S]));
  }
}

// ---- counts -------------------------------------------------------------------
// Tokens that count: a bit each in mask (those in no sequence do not), their
// number in all (head->tokens) and by sequence (n[s]); the last CTA counts the
// sequences that have any.  head and n are zero at the start.
__global__ void __launch_bounds__(kPThreads) policy_count_kernel(PolicyArgs a) {
  __shared__ unsigned long long red[kPThreads / 32];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t lo, hi;
  token_range(a, lo, hi);
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  unsigned long long total = 0;
  if (a.targets) {
    // a warp takes 256 tokens at a time: eight words of the mask
    constexpr int kTokens = 256;
    const int64_t runs = (a.T + kTokens - 1) / kTokens;
    const int64_t warps = (int64_t)gridDim.x * (kPThreads / 32);
    for (int64_t run = (int64_t)blockIdx.x * (kPThreads / 32) + warp; run < runs; run += warps) {
      const int64_t base = run * kTokens;
      unsigned m[8], mine = 0, some = 0;
      if (base >= lo && base + kTokens <= hi) {
        int64_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __ldcs(a.targets + base + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = v[j] >= 0;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t t = base + 32 * j + lane;
          m[j] = t >= lo && t < hi ? (unsigned)(a.targets[t] >= 0) : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = __ballot_sync(0xFFFFFFFFu, m[j]);
        if (lane == j) mine = m[j];
        some += __popc(m[j]);
      }
      if (lane < 8) a.mask[run * 8 + lane] = mine;
      total += some;
      if (by_seq && some) {
        const int64_t s0 = seq_of_warp(a.offsets + 1, a.S, base);
        const int64_t s1 = seq_of_warp(a.offsets + 1, a.S, min(base + kTokens, a.T) - 1);
        if (s0 == s1) {
          if (lane == 0) atomicAdd(&a.n[s0], (unsigned long long)some);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool in = m[j] >> lane & 1;
            const int64_t s = in ? seq_of(a.offsets + 1, s0, s1, base + 32 * j + lane) : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, s);
            if (in && lane == __ffs(same) - 1) atomicAdd(&a.n[s], (unsigned long long)__popc(same));
          }
        }
      }
    }
  } else if (by_seq) {  // every token counts: lengths
    for (int64_t s = (int64_t)blockIdx.x * kPThreads + threadIdx.x; s < a.S;
         s += (int64_t)gridDim.x * kPThreads) {
      // (no offsets: one sequence, all of it)
      const int64_t b = a.offsets ? max(lo, min(hi, a.offsets[s])) : lo;
      const int64_t e = a.offsets ? max(lo, min(hi, a.offsets[s + 1])) : hi;
      a.n[s] = (unsigned long long)max((int64_t)0, e - b);
    }
  }
  if (a.targets) {
    if (lane == 0) red[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kPThreads / 32; ++i) total += red[i];
      if (total) atomicAdd(&a.head->tokens, total);
    }
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.head->tokens = (unsigned long long)(hi - lo);
  }
  if (!by_seq) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(&a.head->arrived[0], 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  unsigned long long any = 0;
  for (int64_t s = threadIdx.x; s < a.S; s += kPThreads) any += __ldcg(&a.n[s]) != 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) any += __shfl_down_sync(0xFFFFFFFFu, any, o);
  if (lane == 0) red[warp] = any;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kPThreads / 32; ++i) any += red[i];
    a.head->seqs = any;
  }
}

// ---- loss and gradient --------------------------------------------------------
__device__ __forceinline__ void get8(const float* p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// This thread's tokens that count, for sums that are far; w_token: the token mean's
// weight, which the loss gets at the end.
__device__ __noinline__ void far_tokens(const PolicyArgs& a, Far& far, int64_t lo, int64_t hi, bool by_seq, double w_token) {
  const double up = a.dloss ? (double)*a.dloss : 1.0;
  for (int64_t t0 = ((int64_t)blockIdx.x * kPThreads + threadIdx.x) * kPRun; t0 < hi; t0 += (int64_t)gridDim.x * kPTile)
    for (int64_t t = max(t0, lo); t < min(t0 + kPRun, hi); ++t) {
      if (a.targets && a.targets[t] < 0) continue;
      const int64_t s = a.offsets && (by_seq || a.adv_per_seq) ? seq_of(a.offsets + 1, 0, a.S - 1, t) : 0;
      const double w = by_seq ? 1.0 / ((double)a.head->seqs * (double)a.n[s]) : 1.0;
      far.add(a, t, a.adv[a.adv_per_seq ? s : t], w, up * w * w_token);
    }
}

// VEC: 16-byte aligned arrays; REF: a reference policy; FIND: a token's sequence
// is needed, for its advantage or its weight.
template <bool VEC, bool REF, bool FIND>
__global__ void __launch_bounds__(kPThreads, 4) policy_loss_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ int64_t range[2];
  __shared__ bool last;
  __shared__ int64_t ends[kPSpan];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t lo, hi;
  token_range(a, lo, hi);
  const bool by_seq = FIND && a.reduction == GS_LOSS_SEQUENCE_MEAN;
  const bool adv_per_seq = FIND && a.adv_per_seq;
  const unsigned long long n = a.counted ? a.head->tokens : (unsigned long long)(hi - lo);
  const float up = a.dloss ? *a.dloss : 1.0f;
  const float seqs = by_seq ? (float)a.head->seqs : 1.0f;
  // the weight of the token mean is applied to the sum, and to each gradient
  const float w_token = a.reduction == GS_LOSS_TOKEN_MEAN ? (n ? (float)(1.0 / (double)n) : 0.0f) : 1.0f;
  const float up_token = __fmul_rn(up, w_token);
  Pair loss_sum = {0.0f, 0.0f}, ratio_sum = loss_sum, kl_sum = loss_sum;
  Far far;
  unsigned long long held_sum = 0;
  const int64_t tiles = (a.T + kPTile - 1) / kPTile;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t base = tile * kPTile, t0 = base + (int64_t)threadIdx.x * kPRun;
    float x[kPRun], old[kPRun], ref[kPRun], adv[kPRun];
    const bool whole = VEC && t0 + kPRun <= a.T;
    // bit j: token t0 + j lies in a sequence, and counts
    unsigned inside = 0;
    if (base >= lo && base + kPTile <= hi) {
      inside = 0xFFu;
    } else {
#pragma unroll
      for (int j = 0; j < kPRun; ++j) inside |= (unsigned)(t0 + j >= lo && t0 + j < hi) << j;
    }
    unsigned live = inside;
    if (a.targets && t0 < a.T) live &= reinterpret_cast<const uint8_t*>(a.mask)[t0 / kPRun];
    if (whole) {
      get8(a.logprob + t0, x);
      get8(a.old + t0, old);
      if constexpr (REF) get8(a.ref + t0, ref);
      if (!adv_per_seq) get8(a.adv + t0, adv);
    } else {
#pragma unroll
      for (int j = 0; j < kPRun; ++j) {
        const int64_t t = t0 + j;
        const bool there = t < a.T;
        x[j] = there ? a.logprob[t] : 0.0f;
        old[j] = there ? a.old[t] : 0.0f;
        ref[j] = REF && there ? a.ref[t] : 0.0f;
        adv[j] = there && !adv_per_seq ? a.adv[t] : 0.0f;
      }
    }
    float w[FIND ? kPRun : 1];
    if constexpr (FIND) {
#pragma unroll
      for (int j = 0; j < kPRun; ++j) w[j] = 1.0f;
      __syncthreads();
      if (warp < 2) {
        const int64_t s = seq_of_warp(a.offsets + 1, a.S, warp ? min(base + kPTile, a.T) - 1 : base);
        if (lane == 0) range[warp] = s;
      }
      __syncthreads();
      const int64_t first = range[0], span = range[1] - range[0];
      const bool near = span < kPSpan;
      if (span > 0 && near) {
        for (int64_t i = threadIdx.x; i <= span; i += kPThreads) ends[i] = a.offsets[first + i + 1];
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kPRun; ++j) {
        if (!(live >> j & 1)) continue;
        const int64_t s = span <= 0 ? first
                          : near    ? first + seq_of(ends, 0, span, t0 + j)
                                    : seq_of(a.offsets + 1, first, range[1], t0 + j);
        if (adv_per_seq) adv[j] = a.adv[s];
        if (by_seq) w[j] = __fdiv_rn(1.0f, __fmul_rn(seqs, (float)a.n[s]));
      }
    }
    float loss = 0.0f, ratio = 0.0f, kl = 0.0f, grad[kPRun];
    unsigned held = 0;
#pragma unroll
    for (int j = 0; j < kPRun; ++j) {
      const Token tk = token<REF, false>(a, x[j], old[j], ref[j], adv[j]);
      const bool in = live >> j & 1;
      loss = __fadd_rn(loss, in ? (FIND ? __fmul_rn(tk.value, w[j]) : tk.value) : 0.0f);
      ratio = __fadd_rn(ratio, in ? tk.ratio : 0.0f);
      kl = __fadd_rn(kl, in ? tk.kl : 0.0f);
      held += in && tk.held;
      grad[j] = in ? __fmul_rn(FIND ? __fmul_rn(up_token, w[j]) : up_token, tk.slope) : 0.0f;
    }
    held_sum += held;
    far.see(loss, ratio, kl);
    loss_sum.add(loss);
    ratio_sum.add(ratio);
    kl_sum.add(kl);
    if (a.grad) {
      if (whole && inside == 0xFFu) {
        __stcs(reinterpret_cast<float4*>(a.grad + t0), make_float4(grad[0], grad[1], grad[2], grad[3]));
        __stcs(reinterpret_cast<float4*>(a.grad + t0) + 1, make_float4(grad[4], grad[5], grad[6], grad[7]));
      } else {
#pragma unroll
        for (int j = 0; j < kPRun; ++j)
          if (inside >> j & 1) a.grad[t0 + j] = grad[j];
      }
    }
  }
  if (far.which)
    far_tokens(a, far, lo, hi, by_seq, a.reduction == GS_LOSS_TOKEN_MEAN && n ? 1.0 / (double)n : 1.0);
  const Sums s = block_sums<kPThreads>(loss_sum, ratio_sum, kl_sum, held_sum, far);
  if (threadIdx.x == 0) {
    a.part[blockIdx.x] = PolicyPart{s.loss, s.ratio, s.kl, s.held};
    __threadfence();
    last = atomicAdd(&a.head->arrived[1], 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  if (warp > 0) return;
  Sums all = {0.0, 0.0, 0.0, 0ull};
  for (unsigned i = lane; i < gridDim.x; i += 32) {
    const volatile PolicyPart& p = a.part[i];
    all.loss += p.loss;
    all.ratio += p.ratio;
    all.kl += p.kl;
    all.held += p.held;
  }
  all = warp_sums<32>(all);
  if (lane == 0) finish(a, all, n);
}

// The same of a CTA that does everything, with its ends, counts, sequences and tokens.
__device__ __noinline__ void far_small_tokens(const PolicyArgs& a, Far& far, int lo, int hi, const int* ends,
                                              const unsigned* counts, unsigned seqs, unsigned n) {
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  const double up = a.dloss ? (double)*a.dloss : 1.0;
  const double w_token = a.reduction == GS_LOSS_TOKEN_MEAN && n ? 1.0 / (double)n : 1.0;
  for (int t = threadIdx.x; t < hi; t += kPSmallThreads) {
    if (t < lo || (a.targets && a.targets[t] < 0)) continue;
    int s = 0;
    if (by_seq || a.adv_per_seq)
      while (s < (int)a.S - 1 && ends[s] <= t) ++s;
    const double w = by_seq ? 1.0 / ((double)seqs * (double)counts[s]) : 1.0;
    far.add(a, t, a.adv[a.adv_per_seq ? s : t], w, up * w * w_token);
  }
}

// Everything by one CTA: offsets, counts and weights in shared memory, the
// tokens' values loaded once, PER of them a thread.
template <int PER, bool REF>
__global__ void __launch_bounds__(kPSmallThreads) policy_loss_small_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ int ends[kPSmallSeqs];
  __shared__ unsigned counts[kPSmallSeqs];
  __shared__ unsigned totals[2];  // tokens, sequences that have any
  const int tid = threadIdx.x;
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  const bool find = by_seq || a.adv_per_seq;
  const int T = (int)a.T, S = (int)a.S;
  float x[PER], old[PER], ref[PER], adv[PER];
  bool in[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int t = j * kPSmallThreads + tid;
    const bool there = t < T;
    in[j] = there && (!a.targets || a.targets[t] >= 0);
    x[j] = there ? a.logprob[t] : 0.0f;
    old[j] = there ? a.old[t] : 0.0f;
    ref[j] = REF && there ? a.ref[t] : 0.0f;
    adv[j] = there && !a.adv_per_seq ? a.adv[t] : 0.0f;
  }
  const float up = a.dloss ? *a.dloss : 1.0f;
  int64_t lo, hi;
  token_range(a, lo, hi);
  if (find)
    for (int s = tid; s < S; s += kPSmallThreads) {
      // (no two tokens of one sequence are told apart by what lies past T)
      ends[s] = a.offsets ? (int)max((int64_t)0, min(a.T, a.offsets[s + 1])) : T;
      counts[s] = 0;
    }
  if (tid < 2) totals[tid] = 0;
  __syncthreads();
  int seq[PER];
  unsigned mine = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int t = j * kPSmallThreads + tid;
    in[j] = in[j] && t >= lo && t < hi;
    mine += in[j];
    seq[j] = 0;
    if (find) {
      int l = 0, h = S - 1;
      while (l < h) {
        const int mid = (l + h) >> 1;
        if (ends[mid] > t) h = mid;
        else l = mid + 1;
      }
      seq[j] = l;
    }
    if (a.adv_per_seq && in[j]) adv[j] = a.adv[seq[j]];
    if (by_seq) {
      const unsigned same = __match_any_sync(0xFFFFFFFFu, in[j] ? seq[j] : -1);
      if (in[j] && (tid & 31) == __ffs(same) - 1) atomicAdd(&counts[seq[j]], (unsigned)__popc(same));
    }
  }
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  if ((tid & 31) == 0 && mine) atomicAdd(&totals[0], mine);
  __syncthreads();
  if (by_seq) {
    unsigned any = 0;
    for (int s = tid; s < S; s += kPSmallThreads) any += counts[s] != 0;
    any = __reduce_add_sync(0xFFFFFFFFu, any);
    if ((tid & 31) == 0 && any) atomicAdd(&totals[1], any);
    __syncthreads();
  }
  const unsigned n = totals[0];
  // a sequence's weight as the sum of two fp32 numbers, from the rounding error
  // of its quotient (sequences times tokens is below 2^24, so exact)
  const float seqs = (float)totals[1];
  const float w_token = a.reduction == GS_LOSS_TOKEN_MEAN && n ? __fdiv_rn(1.0f, (float)n) : 1.0f;
  Pair loss = {0.0f, 0.0f}, ratio = loss, kl = loss;
  Far far;
  unsigned held = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int t = j * kPSmallThreads + tid;
    float w = 1.0f, w_lo = 0.0f;  // (of the token mean: the sum's, in fp64)
    if (by_seq && in[j]) {
      const float count = __fmul_rn(seqs, (float)counts[seq[j]]);
      w = __fdiv_rn(1.0f, count);
      w_lo = __fmul_rn(__fmaf_rn(-w, count, 1.0f), w);
    }
    const Token tk = token<REF, true>(a, x[j], old[j], ref[j], adv[j]);
    if (in[j]) {
      const float part = __fmul_rn(w, tk.value);
      far.see(__fadd_rn(fabsf(tk.value), fabsf(tk.rest)), tk.ratio, tk.kl);
      loss.add(part);
      loss.lo = __fadd_rn(loss.lo, __fmaf_rn(w, tk.rest, __fmaf_rn(w_lo, tk.value, __fmaf_rn(w, tk.value, -part))));
      ratio.add(tk.ratio);
      kl.add(tk.kl);
      held += tk.held;
    }
    if (a.grad && t >= lo && t < hi)
      a.grad[t] = in[j] ? __fmul_rn(__fmul_rn(up, by_seq ? w : w_token), tk.slope) : 0.0f;
  }
  if (far.which) far_small_tokens(a, far, (int)lo, (int)hi, ends, counts, totals[1], n);
  const Sums s = block_sums<kPSmallThreads>(loss, ratio, kl, held, far);
  if (tid == 0) finish(a, s, n);
}

template <int PER>
static void launch_small(const PolicyArgs& a, cudaStream_t st) {
  if (a.ref) policy_loss_small_kernel<PER, true><<<1, kPSmallThreads, 0, st>>>(a);
  else policy_loss_small_kernel<PER, false><<<1, kPSmallThreads, 0, st>>>(a);
}
template <bool VEC, bool REF>
static void launch_large(const PolicyArgs& a, unsigned grid, bool find, cudaStream_t st) {
  if (find) policy_loss_kernel<VEC, REF, true><<<grid, kPThreads, 0, st>>>(a);
  else policy_loss_kernel<VEC, REF, false><<<grid, kPThreads, 0, st>>>(a);
}

cudaError_t launch_policy_loss(PolicyArgs a, cudaStream_t st) {
  if (a.T <= kPSmallTokens && a.S <= kPSmallSeqs) {
    if (a.T <= kPSmallThreads) launch_small<1>(a, st);
    else launch_small<(int)(kPSmallTokens / kPSmallThreads)>(a, st);
    return cudaGetLastError();
  }
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  a.counted = a.targets != nullptr || by_seq;
  const size_t zero = sizeof(PolicyHead) + (by_seq ? (size_t)a.S * sizeof(*a.n) : 0);
  cudaError_t e = cudaMemsetAsync(a.head, 0, zero, st);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.T + kPTile - 1) / kPTile;
  // one wave: four CTAs per SM (64 us for 8 M tokens; three 67, two 71)
  const int64_t most = std::min<int64_t>(kPolicyCtas, (int64_t)sm_count() * 4);
  if (a.counted) {
    const int64_t work = a.targets ? (a.T + 8 * kPThreads - 1) / (8 * kPThreads) : (a.S + kPThreads - 1) / kPThreads;
    policy_count_kernel<<<(unsigned)std::max<int64_t>(1, std::min<int64_t>(work, (int64_t)sm_count() * 8)), kPThreads, 0, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min(tiles, most));
  bool vec = true;
  for (const void* p : {(const void*)a.logprob, (const void*)a.old, (const void*)a.ref,
                        a.adv_per_seq ? nullptr : (const void*)a.adv, (const void*)a.grad})
    vec = vec && (uintptr_t)p % 16 == 0;
  const bool find = by_seq || a.adv_per_seq;
  if (vec) {
    if (a.ref) launch_large<true, true>(a, grid, find, st);
    else launch_large<true, false>(a, grid, find, st);
  } else {
    if (a.ref) launch_large<false, true>(a, grid, find, st);
    else launch_large<false, false>(a, grid, find, st);
  }
  return cudaGetLastError();
}

}  // namespace gs

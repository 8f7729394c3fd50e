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
// order changes nothing; the targets' second read comes from L2 where they fit
// it.  Sums: four tokens' terms in fp32, everything beyond in fp64, joined in a
// fixed order by the last CTA to finish.  Short batches are done by one CTA,
// which counts and sums in one launch.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gs_internal.h"
#include "gs_policy.h"
#include "gsfp8.h"

namespace gs {

constexpr int kPThreads = 256;
constexpr int kPRun = 4;                     // tokens per thread and step
constexpr int kPTile = kPThreads * kPRun;    // tokens per CTA and step
constexpr int kPSpan = 1024;                 // sequences of a step kept in shared memory

// Tokens that one CTA of 1024 threads does alone (see launch_policy_loss).
constexpr int64_t kPSmallTokens = 8192;
constexpr int64_t kPSmallSeqs = 2048;
constexpr int kPSmallThreads = 1024;

struct Sums {
  double loss, ratio, kl;
  unsigned long long held;
};

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

struct Token {
  float value, slope, ratio, kl;  // l and dl/dx without the weight
  bool held;
};
__device__ __forceinline__ Token token(const PolicyArgs& a, float x, float old, float ref, float adv) {
  Token t;
  float d, e;
  two_diff(x, old, d, e);
  t.ratio = expf(d);
  const bool up = adv > 0.0f && above(d, e, a.high);
  const bool down = adv < 0.0f && below(d, e, a.low);
  const bool far = adv < 0.0f && above(d, e, a.dual);
  t.held = up || down || far;
  const float factor = up ? a.factor_high : down ? a.factor_low : far ? a.factor_dual : t.ratio;
  const float obj = adv == 0.0f ? 0.0f : __fmul_rn(factor, adv);
  t.slope = t.held ? 0.0f : -obj;
  t.kl = 0.0f;
  t.value = -obj;
  if (a.ref) {
    const float y = __fsub_rn(ref, x);
    const float em1 = expm1f(y);
    // y^2 (1/2 + y/6 + ... + y^7/9!): cut off at 2e-9 of it for |y| <= 1/2
    float p = 1.0f / 362880.0f;
    p = __fmaf_rn(p, y, 1.0f / 40320.0f);
    p = __fmaf_rn(p, y, 1.0f / 5040.0f);
    p = __fmaf_rn(p, y, 1.0f / 720.0f);
    p = __fmaf_rn(p, y, 1.0f / 120.0f);
    p = __fmaf_rn(p, y, 1.0f / 24.0f);
    p = __fmaf_rn(p, y, 1.0f / 6.0f);
    p = __fmaf_rn(p, y, 0.5f);
    t.kl = fabsf(y) <= 0.5f ? __fmul_rn(__fmul_rn(y, y), p) : __fsub_rn(em1, y);
    t.value = __fmaf_rn(a.kl, t.kl, t.value);
    t.slope = __fmaf_rn(-a.kl, em1, t.slope);
  }
  return t;
}

// Adds a block's sums; the result in thread 0.
template <int NT>
__device__ __forceinline__ Sums block_sums(Sums s) {
  __shared__ Sums red[NT / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.loss += __shfl_down_sync(0xFFFFFFFFu, s.loss, o);
    s.ratio += __shfl_down_sync(0xFFFFFFFFu, s.ratio, o);
    s.kl += __shfl_down_sync(0xFFFFFFFFu, s.kl, o);
    s.held += __shfl_down_sync(0xFFFFFFFFu, s.held, o);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < NT / 32; ++i) {
      s.loss += red[i].loss;
      s.ratio += red[i].ratio;
      s.kl += red[i].kl;
      s.held += red[i].held;
    }
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
// Tokens that count, in all (head->tokens) and by sequence (n[s]); the last
// CTA counts the sequences that have any.  Both are zero at the start.
__global__ void __launch_bounds__(kPThreads) policy_count_kernel(PolicyArgs a) {
  __shared__ unsigned red[kPThreads / 32];
  __shared__ int64_t range[2];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t lo, hi;
  token_range(a, lo, hi);
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  unsigned long long total = 0;
  if (a.targets) {
    const int64_t tiles = (a.T + kPTile - 1) / kPTile;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int64_t base = tile * kPTile;
      if (by_seq) {
        __syncthreads();
        if (warp < 2) {
          const int64_t s = seq_of_warp(a.offsets + 1, a.S, warp ? min(base + kPTile, a.T) - 1 : base);
          if (lane == 0) range[warp] = s;
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kPRun; ++j) {
        const int64_t t = base + j * kPThreads + threadIdx.x;
        const bool in = t >= lo && t < hi && a.targets[t] >= 0;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, in);
        if (lane == 0) total += __popc(m);
        if (by_seq && m) {
          if (range[0] == range[1]) {
            if (lane == 0) atomicAdd(&a.n[range[0]], (unsigned long long)__popc(m));
          } else {
            const int64_t s = in ? seq_of(a.offsets + 1, range[0], range[1], t) : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, s);
            if (in && lane == __ffs(same) - 1)
              atomicAdd(&a.n[s], (unsigned long long)__popc(same));
          }
        }
      }
    }
  } else if (by_seq) {  // every token counts: lengths
    for (int64_t s = (int64_t)blockIdx.x * kPThreads + threadIdx.x; s < a.S;
         s += (int64_t)gridDim.x * kPThreads) {
      const int64_t b = max(lo, min(hi, a.offsets[s])), e = max(lo, min(hi, a.offsets[s + 1]));
      a.n[s] = (unsigned long long)max((int64_t)0, e - b);
    }
  }
  if (a.targets) {
    if (lane == 0) red[warp] = (unsigned)total;  // below 2^32 tokens per CTA
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long sum = 0;
      for (int i = 0; i < kPThreads / 32; ++i) sum += red[i];
      if (sum) atomicAdd(&a.head->tokens, sum);
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
  unsigned any = 0;
  for (int64_t s = threadIdx.x; s < a.S; s += kPThreads) any += __ldcg(&a.n[s]) != 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) any += __shfl_down_sync(0xFFFFFFFFu, any, o);
  if (lane == 0) red[warp] = any;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long sum = 0;
    for (int i = 0; i < kPThreads / 32; ++i) sum += red[i];
    a.head->seqs = sum;
  }
}

// ---- loss and gradient --------------------------------------------------------
template <bool VEC>
__global__ void __launch_bounds__(kPThreads) policy_loss_kernel(PolicyArgs a) {
  __shared__ int64_t range[2];
  __shared__ bool last;
  __shared__ int64_t ends[kPSpan];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t lo, hi;
  token_range(a, lo, hi);
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  const bool find = by_seq || a.adv_per_seq;
  const unsigned long long n = a.counted ? a.head->tokens : (unsigned long long)(hi - lo);
  const float up = a.dloss ? *a.dloss : 1.0f;
  const double seqs = by_seq ? (double)a.head->seqs : 1.0;
  // the weight of the token mean is applied to the sum, and to each gradient
  const float w_token = a.reduction == GS_LOSS_TOKEN_MEAN ? (n ? (float)(1.0 / (double)n) : 0.0f) : 1.0f;
  Sums sums = {0.0, 0.0, 0.0, 0ull};
  const int64_t tiles = (a.T + kPTile - 1) / kPTile;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t base = tile * kPTile, t0 = base + (int64_t)threadIdx.x * kPRun;
    float x[kPRun], old[kPRun], ref[kPRun], adv[kPRun];
    bool live[kPRun], inside[kPRun];
    const bool whole = VEC && t0 + kPRun <= a.T;
    if (whole) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(a.logprob + t0));
      const float4 o = __ldcs(reinterpret_cast<const float4*>(a.old + t0));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      old[0] = o.x, old[1] = o.y, old[2] = o.z, old[3] = o.w;
      if (a.ref) {
        const float4 r = __ldcs(reinterpret_cast<const float4*>(a.ref + t0));
        ref[0] = r.x, ref[1] = r.y, ref[2] = r.z, ref[3] = r.w;
      }
      if (!a.adv_per_seq) {
        const float4 v2 = __ldcs(reinterpret_cast<const float4*>(a.adv + t0));
        adv[0] = v2.x, adv[1] = v2.y, adv[2] = v2.z, adv[3] = v2.w;
      }
      if (a.targets) {
        const longlong2 p = __ldcs(reinterpret_cast<const longlong2*>(a.targets + t0));
        const longlong2 q = __ldcs(reinterpret_cast<const longlong2*>(a.targets + t0 + 2));
        live[0] = p.x >= 0, live[1] = p.y >= 0, live[2] = q.x >= 0, live[3] = q.y >= 0;
      }
    }
#pragma unroll
    for (int j = 0; j < kPRun; ++j) {
      const int64_t t = t0 + j;
      inside[j] = t >= lo && t < hi;
      if (!whole) {
        const bool there = t < a.T;
        x[j] = there ? a.logprob[t] : 0.0f;
        old[j] = there ? a.old[t] : 0.0f;
        ref[j] = there && a.ref ? a.ref[t] : 0.0f;
        adv[j] = there && !a.adv_per_seq ? a.adv[t] : 0.0f;
        live[j] = there && (!a.targets || a.targets[t] >= 0);
      } else {
        if (!a.ref) ref[j] = 0.0f;
        if (!a.targets) live[j] = true;
      }
      live[j] = live[j] && inside[j];
    }
    float w[kPRun];
#pragma unroll
    for (int j = 0; j < kPRun; ++j) w[j] = w_token;
    if (find) {
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
        if (!live[j]) continue;
        const int64_t s = span <= 0 ? first
                          : near    ? first + seq_of(ends, 0, span, t0 + j)
                                    : seq_of(a.offsets + 1, first, range[1], t0 + j);
        if (a.adv_per_seq) adv[j] = a.adv[s];
        if (by_seq) w[j] = (float)(1.0 / (seqs * (double)a.n[s]));
      }
    }
    float loss = 0.0f, ratio = 0.0f, kl = 0.0f, grad[kPRun];
#pragma unroll
    for (int j = 0; j < kPRun; ++j) {
      grad[j] = 0.0f;
      if (!live[j]) continue;
      const Token tk = token(a, x[j], old[j], ref[j], adv[j]);
      loss = __fadd_rn(loss, by_seq ? __fmul_rn(tk.value, w[j]) : tk.value);
      ratio = __fadd_rn(ratio, tk.ratio);
      kl = __fadd_rn(kl, tk.kl);
      sums.held += tk.held;
      grad[j] = __fmul_rn(__fmul_rn(up, w[j]), tk.slope);
    }
    sums.loss += (double)loss;
    sums.ratio += (double)ratio;
    sums.kl += (double)kl;
    if (a.grad) {
      bool all = whole;
#pragma unroll
      for (int j = 0; j < kPRun; ++j) all = all && inside[j];
      if (all) {
        __stcs(reinterpret_cast<float4*>(a.grad + t0), make_float4(grad[0], grad[1], grad[2], grad[3]));
      } else {
#pragma unroll
        for (int j = 0; j < kPRun; ++j)
          if (inside[j]) a.grad[t0 + j] = grad[j];
      }
    }
  }
  const Sums s = block_sums<kPThreads>(sums);
  if (threadIdx.x == 0) {
    a.part[blockIdx.x] = PolicyPart{s.loss, s.ratio, s.kl, s.held};
    __threadfence();
    last = atomicAdd(&a.head->arrived[1], 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  Sums all = {0.0, 0.0, 0.0, 0ull};
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kPThreads) {
    const volatile PolicyPart& p = a.part[i];
    all.loss += p.loss;
    all.ratio += p.ratio;
    all.kl += p.kl;
    all.held += p.held;
  }
  all = block_sums<kPThreads>(all);
  if (threadIdx.x == 0) finish(a, all, n);
}

// Everything by one CTA: counts in shared memory, then loss and gradient.
__global__ void __launch_bounds__(kPSmallThreads) policy_loss_small_kernel(PolicyArgs a) {
  __shared__ unsigned counts[kPSmallSeqs];
  __shared__ unsigned totals[2];  // tokens, sequences that have any
  const int tid = threadIdx.x;
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  const bool find = by_seq || a.adv_per_seq;
  int64_t lo, hi;
  token_range(a, lo, hi);
  if (by_seq)
    for (int64_t s = tid; s < a.S; s += kPSmallThreads) counts[s] = 0;
  if (tid < 2) totals[tid] = 0;
  __syncthreads();
  constexpr int kMost = (int)(kPSmallTokens / kPSmallThreads);
  int seq[kMost];
  float x[kMost], old[kMost], ref[kMost], adv[kMost];
  unsigned live = 0;
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    const int64_t t = (int64_t)j * kPSmallThreads + tid;
    const bool in = t >= lo && t < hi && (!a.targets || a.targets[t] >= 0);
    x[j] = in ? a.logprob[t] : 0.0f;
    old[j] = in ? a.old[t] : 0.0f;
    ref[j] = in && a.ref ? a.ref[t] : 0.0f;
    adv[j] = in && !a.adv_per_seq ? a.adv[t] : 0.0f;
    seq[j] = in && find ? (int)seq_of(a.offsets + 1, 0, a.S - 1, t) : 0;
    if (in && a.adv_per_seq) adv[j] = a.adv[seq[j]];
    if (in) live |= 1u << j;
    if (by_seq) {
      const unsigned same = __match_any_sync(0xFFFFFFFFu, in ? seq[j] : -1);
      if (in && (tid & 31) == __ffs(same) - 1) atomicAdd(&counts[seq[j]], (unsigned)__popc(same));
    }
  }
  const unsigned mine = __reduce_add_sync(0xFFFFFFFFu, (unsigned)__popc(live));
  if ((tid & 31) == 0 && mine) atomicAdd(&totals[0], mine);
  __syncthreads();
  if (by_seq) {
    unsigned any = 0;
    for (int64_t s = tid; s < a.S; s += kPSmallThreads) any += counts[s] != 0;
    any = __reduce_add_sync(0xFFFFFFFFu, any);
    if ((tid & 31) == 0 && any) atomicAdd(&totals[1], any);
    __syncthreads();
  }
  const unsigned n = totals[0];
  const float up = a.dloss ? *a.dloss : 1.0f;
  const float w_token = a.reduction == GS_LOSS_TOKEN_MEAN ? (n ? (float)(1.0 / (double)n) : 0.0f) : 1.0f;
  Sums sums = {0.0, 0.0, 0.0, 0ull};
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    const int64_t t = (int64_t)j * kPSmallThreads + tid;
    float grad = 0.0f;
    if (live >> j & 1) {
      const float w = by_seq ? (float)(1.0 / ((double)totals[1] * (double)counts[seq[j]])) : w_token;
      const Token tk = token(a, x[j], old[j], ref[j], adv[j]);
      sums.loss += (double)(by_seq ? __fmul_rn(tk.value, w) : tk.value);
      sums.ratio += (double)tk.ratio;
      sums.kl += (double)tk.kl;
      sums.held += tk.held;
      grad = __fmul_rn(__fmul_rn(up, w), tk.slope);
    }
    if (a.grad && t >= lo && t < hi) a.grad[t] = grad;
  }
  const Sums s = block_sums<kPSmallThreads>(sums);
  if (tid == 0) finish(a, s, n);
}

cudaError_t launch_policy_loss(PolicyArgs a, cudaStream_t st) {
  if (a.T <= kPSmallTokens && a.S <= kPSmallSeqs) {
    policy_loss_small_kernel<<<1, kPSmallThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const bool by_seq = a.reduction == GS_LOSS_SEQUENCE_MEAN;
  a.counted = a.targets != nullptr || by_seq;
  const size_t zero = sizeof(PolicyHead) + (by_seq ? (size_t)a.S * sizeof(*a.n) : 0);
  cudaError_t e = cudaMemsetAsync(a.head, 0, zero, st);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.T + kPTile - 1) / kPTile;
  const int64_t most = std::min<int64_t>(kPolicyCtas, (int64_t)sm_count() * 8);
  if (a.counted) {
    const int64_t work = a.targets ? tiles : (a.S + kPThreads - 1) / kPThreads;
    policy_count_kernel<<<(unsigned)std::max<int64_t>(1, std::min(work, most)), kPThreads, 0, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min(tiles, most));
  bool vec = true;
  for (const void* p : {(const void*)a.logprob, (const void*)a.old, (const void*)a.ref,
                        a.adv_per_seq ? nullptr : (const void*)a.adv, (const void*)a.targets,
                        (const void*)a.grad})
    vec = vec && (uintptr_t)p % 16 == 0;
  if (vec) policy_loss_kernel<true><<<grid, kPThreads, 0, st>>>(a);
  else policy_loss_kernel<false><<<grid, kPThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gs

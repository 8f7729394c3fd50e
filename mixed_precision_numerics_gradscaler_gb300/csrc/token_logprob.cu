// token_logprob.cu -- log probabilities of given tokens, entropy and the
// largest alternatives of each row of logits, and their gradient under the
// loss scale ("Loss scaling, FP8, and the failure that never crashes",
// section "Loss scaling, derived from the chain rule you already have": the
// scaled loss's gradient is where S enters the backward pass).
//
//   lse = m + log s,  m = max x,  s = sum e^(x - m)
//   entropy = log s - t / s,  t = sum e^(x - m) (x - m)
//   dlogits = S (dlogprob (1[target] - p) - dentropy p (x - lse + entropy))
//
// Forward: one pass over the logits.  Every thread keeps the running maximum
// m of what it has read and s, t relative to it, in powers of two
// (e^d = 2^(d log2 e), one ex2 instruction); pairs join by rescaling to the
// larger maximum.  A row is one CTA's, or a cluster's where there are few
// rows: its CTAs take one part each and the first joins them through
// distributed shared memory.
//
// The alternatives come out of the same pass.  A thread's maximum is the
// largest of the elements it read, so the k-th largest of any 32 of the
// threads' maxima is a lower bound of the k-th largest logit (k elements reach
// it), and only the elements of threads whose maximum reaches it can be among
// the first k: with each warp's largest maxima as the 32, about k threads (a
// few in a hundred).  Each thread keeps the block (four vectors) in which its
// maximum first occurred in shared memory, and the maximum of its other
// blocks: the elements of a chosen thread are at hand, and only where its
// other blocks reach the bound too is everything it read loaded again.  What
// reaches the bound, little more than k elements, is sorted by one warp.
// (Loading the chosen threads' elements again, a microsecond or two under
// load at the end of every row, cost 4096 x 128256 bf16 with 8 alternatives
// 204 us, all of them, and 212 us, the one block; collecting candidates while
// the row is read, against a bound formed on the way, 282 us; from the kept
// blocks 195 us.)
//
// HBM-bound where rows are long and many: 4096 x 128256 bf16 takes 158 us
// (6.7 TB/s), 178 us with 8 alternatives, whose choice at a row's end only other
// CTAs' loads can cover; with short rows, or few of them, the joins decide.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gs_elem.cuh"
#include "gs_internal.h"
#include "gs_quant.cuh"

namespace gs {

constexpr int kLossCluster = 8;  // most CTAs of a row
constexpr int kCandidates = 256; // alternatives' candidates kept for sorting
constexpr int kLossVecs = 4;     // 16-byte vectors of a thread's block

// Beyond this |lse| its rounding to fp32 (2^-24 |lse|, the relative error it
// brings to every p) is no longer small beside the rest, and the gradient
// forms the row's sum anew: every run's CTA for itself (32 reads of a row of
// 128256 16-bit logits, out of L2: 8192 such rows 5370 us, 593 without), in place
// one CTA for the row (1095 us).
constexpr float kLseExact = 256.0f;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A logit and its index as one number whose unsigned order is the order of
// the alternatives: larger logits first (NaN above all, -0 equal to +0), and
// the lower index first among equals.  Key 0 stands for no element.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_pair(float x, uint32_t i) {
  return ((uint64_t)order_key(x) << 32) | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k ^ 0x80000000u) : ~k);
}

// ---- running softmax statistics -------------------------------------------
// m: the maximum (NaN left out); s: sum 2^d, t: sum 2^d d with
// d = (x - m) log2 e.  A NaN or +Inf logit makes s NaN.
struct Stats {
  float m, s, t;
};

// Brings (s, t) from maximum m to the larger M.  m = -Inf (nothing yet,
// s = 0) must not turn into 0 * Inf: the shift is kept finite.
__device__ __forceinline__ void rescale(float m, float M, float& s, float& t) {
  const float D = fmaxf((m - M) * kLog2e, -1e30f);
  const float f = ex2(D);
  t = __fmaf_rn(D, s, t) * f;
  s *= f;
}
__device__ __forceinline__ Stats join(Stats a, Stats b) {
  const float M = fmaxf(a.m, b.m);
  if (M > -CUDART_INF_F) {  // else both are empty (or NaN: s tells)
    rescale(a.m, M, a.s, a.t);
    rescale(b.m, M, b.s, b.t);
  }
  return Stats{M, a.s + b.s, a.t + b.t};
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int N>
__device__ __forceinline__ float max_of(const float* x) {
  float m = x[0];
  if constexpr (N % 2 == 0) m = fmaxf(m, x[1]);
#pragma unroll
  for (int i = N % 2 ? 1 : 2; i < N; i += 2) m = max3(m, x[i], x[i + 1]);
  return m;
}

// 16 bytes of logits as fp32.
template <int DT>
constexpr int kVec = DT == GS_F32 ? 4 : 8;
template <int DT>
__device__ __forceinline__ void unpack16(const uint4& v, float* x) {
  if constexpr (DT == GS_F32) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  } else {
    using Tag = std::conditional_t<DT == GS_BF16, BF16Tag, F16Tag>;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = lo16<Tag>(w[i]);
      x[2 * i + 1] = hi16<Tag>(w[i]);
    }
  }
}


// N logits with maximum lm (N even).  d is kept above -1024, where 2^d is 0
// all the same, so that a masked logit adds 0 and not 0 * Inf to t.
template <int N>
__device__ __forceinline__ void take(Stats& a, const float* x, float lm) {
  if (lm > a.m) {
    rescale(a.m, lm, a.s, a.t);
    a.m = lm;
  }
  const float mm = a.m == -CUDART_INF_F ? 0.0f : a.m;
  const uint64_t nm = pk_f32x2(-mm, -mm), l2e = pk_f32x2(kLog2e, kLog2e);
  uint64_t s2 = pk_f32x2(a.s, 0.0f), t2 = pk_f32x2(a.t, 0.0f);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float d0, d1;
    upk_f32x2(mul_f32x2(add_f32x2(pk_f32x2(x[i], x[i + 1]), nm), l2e), d0, d1);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d0) : "f"(-1024.0f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d1) : "f"(-1024.0f));
    const uint64_t e = pk_f32x2(ex2(d0), ex2(d1));
    s2 = add_f32x2(s2, e);
    t2 = fma_f32x2(e, pk_f32x2(d0, d1), t2);
  }
  float lo, hi;
  upk_f32x2(s2, lo, hi);
  a.s = lo + hi;
  upk_f32x2(t2, lo, hi);
  a.t = lo + hi;
}

// A run of a row: `head` elements up to the first 16-byte boundary, nv
// 16-byte vectors, then `tail` elements (head, tail < kVec).
template <int DT>
struct Run {
  const char* p;  // first element
  int head, tail;
  int nv;
  static constexpr int kSize = sizeof(typename Elem<DT>::type);
  __device__ __forceinline__ Run(const void* base, int64_t n) : p(static_cast<const char*>(base)) {
    const int64_t h = (int64_t)((16u - ((uint32_t)(uintptr_t)p & 15u)) & 15u) / kSize;
    head = (int)(h < n ? h : n);
    nv = (int)((n - head) / kVec<DT>);
    tail = (int)(n - head - (int64_t)nv * kVec<DT>);
  }
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(p + head * kSize);
  }
  // Index of the odd element that thread i holds (the heads, then the
  // tails), or -1.
  __device__ __forceinline__ int64_t odd(int i) const {
    if (i < head) return i;
    return i < head + tail ? (int64_t)nv * kVec<DT> + i : -1;
  }
};

// ---- sorted lists across a warp -------------------------------------------
// Lane i holds the i-th largest of up to 32 values.

// Sorts 32 lanes' values, largest in lane 0 (bitonic).
template <typename T>
__device__ __forceinline__ T sort_desc(T v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const T o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
      const bool up = ((lane & k) == 0) == ((lane & j) == 0);  // this lane keeps the larger
      v = up ? (v > o ? v : o) : (v < o ? v : o);
    }
  return v;
}
// The 32 largest of two sorted lists, sorted: the lane-wise maximum of one and
// the other reversed holds them as a bitonic sequence.
template <typename T>
__device__ __forceinline__ T merge_desc(T a, T b, int lane) {
  const T r = __shfl_sync(0xFFFFFFFFu, b, 31 - lane);
  T v = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const T o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
    v = (lane & j) == 0 ? (v > o ? v : o) : (v < o ? v : o);
  }
  return v;
}
// A warp's k best pairs so far; a pair below `bound` is none of the row's k
// best.
struct Best {
  unsigned long long v, bound;
  int k;
  __device__ __forceinline__ void offer(unsigned long long q, bool have, int lane) {
    unsigned mask = __ballot_sync(0xFFFFFFFFu, have && q >= bound);
    while (mask) {
      const unsigned long long c = __shfl_sync(0xFFFFFFFFu, q, __ffs(mask) - 1);
      mask &= mask - 1;
      if (c < bound) continue;
      const int at = __popc(__ballot_sync(0xFFFFFFFFu, v > c));
      const unsigned long long up = __shfl_up_sync(0xFFFFFFFFu, v, 1);
      v = lane < at ? v : lane == at ? c : up;
      const unsigned long long last = __shfl_sync(0xFFFFFFFFu, v, k - 1);
      if (last > bound) bound = last;
    }
  }
};

// ---- forward ---------------------------------------------------------------

struct LogprobArgs {
  const void* logits;
  int64_t ld, R, V, part;  // part: columns of each CTA of a row, a multiple of 8
  const int64_t* targets;
  float* logprob;
  float* lse;
  float* entropy;
  int top_k;
  int32_t* top_ids;
  float* top_logprob;
};

__device__ __forceinline__ float remote_f32(const void* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)));
  return v;
}
__device__ __forceinline__ unsigned long long remote_u64(const void* p, uint32_t rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)));
  return v;
}

// The k-th largest of 32 of the CTA's keys, each warp's largest ones: a lower
// bound of the CTA's k-th largest.  `buf` holds 32 values that no thread still
// reads; every thread returns the same.
template <int NT, typename T>
__device__ __forceinline__ T bound_of(T key, int k, T* buf, int warp, int lane) {
  constexpr int kWarps = NT / 32, kEach = 32 / kWarps;
  T v = key;
  if constexpr (sizeof(T) == 4 && kEach <= 4) {  // a few rounds beat a sort
    T mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const T top = __reduce_max_sync(0xFFFFFFFFu, v);
      if (lane == i) mine = top;
      if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, v == top)) - 1) v = 0;
    }
    v = mine;
  } else {
    v = sort_desc(v, lane);
  }
  if constexpr (kWarps > 1) {
    if (lane < kEach) buf[warp * kEach + lane] = v;
    __syncthreads();
    v = sort_desc(buf[lane], lane);
  }
  return __shfl_sync(0xFFFFFFFFu, v, k - 1);
}

// Where a thread's maximum lies: its value, the block in which it first
// occurred, and the maximum of the other blocks.
struct Peak {
  float m, other;
  int64_t block;
  // True when the block's maximum lm is the largest so far (or the first).
  __device__ __forceinline__ bool see(float lm, int64_t blk) {
    if (lm > m || blk == 0) {
      other = m;
      m = lm;
      block = blk;
      return true;
    }
    other = fmaxf(other, lm);
    return false;
  }
};

// The candidates for the alternatives.
struct Candidates {
  unsigned long long* pair;
  int* n;
  // Those of a vector's elements (column i0 and on) whose pair reaches `bound`;
  // low: the logit of the bound's key (an element below it does not reach it;
  // NaN is not below).
  template <int DT>
  __device__ __forceinline__ void offer(const uint4& w, uint32_t i0, unsigned long long bound,
                                        float low) const {
    float x[kVec<DT>];
    unpack16<DT>(w, x);
#pragma unroll
    for (int j = 0; j < kVec<DT>; ++j)
      if (!(x[j] < low)) offer1(order_pair(x[j], i0 + j), bound);
  }
  __device__ __forceinline__ void offer1(unsigned long long q, unsigned long long bound) const {
    if (q < bound) return;
    const int at = atomicAdd(n, 1);
    if (at < kCandidates) pair[at] = q;
  }
};

// A vector whose logits are all -Inf.
template <int DT>
__device__ __forceinline__ uint4 masked16() {
  const uint32_t w = DT == GS_F32 ? 0xFF800000u : DT == GS_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  return make_uint4(w, w, w, w);
}

// The 32 largest of the warps' sorted lists, sorted, in warp 0.  `buf` holds
// NT values; its reads before and after are the caller's to separate by
// barriers.
template <int NT>
__device__ __forceinline__ unsigned long long join_warps(unsigned long long v,
                                                         unsigned long long* buf, int warp,
                                                         int lane) {
#pragma unroll
  for (int half = NT / 64; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) buf[warp * 32 + lane] = v;
    __syncthreads();
    if (warp < half) v = merge_desc(v, buf[(warp + half) * 32 + lane], lane);
  }
  return v;
}

// The CTA's top_k pairs in order in warp 0 (other warps' result is unused).
// `nan`: this thread read a NaN or +Inf; kept: the threads' peak blocks.
template <int DT, int NT>
__device__ __forceinline__ unsigned long long alternatives(const Run<DT>& run, const char* row,
                                                           int64_t c0, const Peak& peak, bool nan,
                                                           int top_k, const uint4* kept,
                                                           unsigned long long* cand,
                                                           unsigned long long* shared_bound,
                                                           int* n_cand) {
  constexpr int N = kVec<DT>, kWarps = NT / 32, U = kLossVecs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint4* p = run.vec();
  const uint32_t first_col = (uint32_t)(c0 + run.head);
  const int64_t odd = run.odd(tid);
  uint32_t key = tid < run.nv || odd >= 0 ? order_key(peak.m) : 0;
  uint32_t other = order_key(peak.other);
  if (nan) {  // the keys from the elements: NaN is above all others
    for (int64_t i = tid; i < run.nv; i += NT) {
      float x[N];
      unpack16<DT>(ld_stream(p + i), x);
#pragma unroll
      for (int j = 0; j < N; ++j) key = max(key, order_key(x[j]));
    }
    if (odd >= 0) key = max(key, order_key(load1<DT>(row, odd)));
    other = key;  // look at every block
  }
  if (tid == 0) *n_cand = 0;
  unsigned long long bound =
      (unsigned long long)bound_of<NT>(key, top_k, reinterpret_cast<uint32_t*>(cand), warp, lane)
      << 32;
  bool mine = key != 0 && key >= (uint32_t)(bound >> 32);
  // (the barrier also ends the reads of `cand`)
  if (__syncthreads_count(mine) > 4 * top_k + 32) {
    // Many equal maxima (a masked part, a row of few values): order them by
    // where each first occurs, which leaves about k threads.
    unsigned long long first = 0;
    if (mine) {
      for (int64_t i = tid + (nan ? 0 : peak.block * U * NT); i < run.nv && first == 0; i += NT) {
        float x[N];
        unpack16<DT>(ld_stream(p + i), x);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (first == 0 && order_key(x[j]) == key)
            first = order_pair(x[j], first_col + (uint32_t)(i * N + j));
      }
      if (odd >= 0) {
        const unsigned long long q = order_pair(load1<DT>(row, odd), (uint32_t)(c0 + odd));
        if (q > first) first = q;
      }
    }
    // (The exact k-th: in rows in order the first ones are one warp's.)
    const unsigned long long best_first = join_warps<NT>(sort_desc(first, lane), cand, warp, lane);
    if (warp == 0 && lane == top_k - 1) *shared_bound = best_first;
    __syncthreads();
    bound = *shared_bound;
    mine = first != 0 && first >= bound;
  }
  const Candidates list{cand, n_cand};
  // Whether another of this thread's blocks may hold one: its maximum is above
  // the bound's logit, or equal to it and the next block (equal ones come after
  // the first) begins before the bound's column.
  const uint32_t bound_key = (uint32_t)(bound >> 32), bound_col = 0xFFFFFFFFu - (uint32_t)bound;
  const uint32_t next_col = first_col + (uint32_t)((peak.block + 1) * U * NT + tid) * N;
  const bool all = mine && (nan || other > bound_key || (other == bound_key && next_col <= bound_col));
  const float low = key_value(bound_key);
  if (mine && !all) {  // the block of the maximum
    const int v = tid + peak.block * U * NT;
#pragma unroll 1
    for (int u = 0; u < U; ++u)
      if (v + u * NT < run.nv)
        list.offer<DT>(kept[u * NT + tid], first_col + (uint32_t)((v + u * NT) * N), bound, low);
  }
  // all blocks of a thread, by its whole warp
  const unsigned whole = __ballot_sync(0xFFFFFFFFu, all);
  for (unsigned m = whole; m; m &= m - 1) {
    const int o = warp * 32 + __ffs(m) - 1;
    for (int64_t i0 = o + (int64_t)lane * NT; i0 < run.nv; i0 += (int64_t)64 * NT) {
      const int64_t i1 = i0 + (int64_t)32 * NT;
      const uint4 w0 = ld_stream(p + i0);
      const uint4 w1 = i1 < run.nv ? ld_stream(p + i1) : w0;
      list.offer<DT>(w0, first_col + (uint32_t)(i0 * N), bound, low);
      if (i1 < run.nv) list.offer<DT>(w1, first_col + (uint32_t)(i1 * N), bound, low);
    }
  }
  if (mine && odd >= 0) list.offer1(order_pair(load1<DT>(row, odd), (uint32_t)(c0 + odd)), bound);
  const unsigned chosen = __ballot_sync(0xFFFFFFFFu, mine);
  __syncthreads();
  const int n = *n_cand;
  unsigned long long best = 0;
  if (n <= 32) {
    if (warp == 0) best = sort_desc(lane < n ? cand[lane] : 0ull, lane);
    return best;
  }
  if (n <= kCandidates) {  // every warp sorts its share, then pairs of warps join
    const auto sorted = [&](int i) {
      return sort_desc(i + lane < n ? cand[i + lane] : 0ull, lane);
    };
    best = sorted(warp * 32);
    for (int i = (warp + kWarps) * 32; i < n; i += kWarps * 32)
      best = merge_desc(best, sorted(i), lane);
    __syncthreads();  // the reads of `cand` have ended
    return join_warps<NT>(best, cand, warp, lane);
  }
  // A thread held many of the largest: insert them one by one instead.
  __syncthreads();
  Best b{0, bound, top_k};
  for (unsigned m = chosen; m; m &= m - 1) {
    const int o = warp * 32 + __ffs(m) - 1;
    for (int64_t i0 = o; i0 < run.nv; i0 += (int64_t)32 * NT) {
      const int64_t i = i0 + (int64_t)lane * NT;
      const bool have = i < run.nv;
      float x[N];
      unpack16<DT>(have ? ld_stream(p + i) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
      for (int j = 0; j < N; ++j)
        b.offer(order_pair(x[j], first_col + (uint32_t)(i * N + j)), have, lane);
    }
    const int64_t i = run.odd(o);
    if (i >= 0) b.offer(order_pair(load1<DT>(row, i), (uint32_t)(c0 + i)), lane == 0, lane);
  }
  static_assert(kWarps * 32 <= kCandidates, "the warps' lists must fit");
  cand[warp * 32 + lane] = b.v;
  __syncthreads();
  best = b.v;
  if (warp == 0)
    for (int i = 1; i < kWarps; ++i) best = merge_desc(best, cand[i * 32 + lane], lane);
  return best;
}

template <int DT, int NT, int CTAS, bool TOP>
__global__ void __launch_bounds__(NT, CTAS) token_logprob_kernel(const LogprobArgs a) {
  constexpr int kWarps = NT / 32;
  __shared__ Stats part_stats[kWarps];
  __shared__ float row_stats[3];
  __shared__ uint4 kept[TOP ? kLossVecs * NT : 1];
  __shared__ unsigned long long cand[TOP ? kCandidates : 1];
  __shared__ unsigned long long row_list[TOP ? 32 : 1];
  __shared__ int n_cand;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t parts = cluster_size(), rank = cluster_rank();
  constexpr int N = kVec<DT>, U = kLossVecs;

  for (int64_t r = blockIdx.x / parts; r < a.R; r += gridDim.x / parts) {
    const int64_t c0 = a.part * rank < a.V ? a.part * rank : a.V;
    const int64_t n = a.V - c0 < a.part ? a.V - c0 : a.part;
    const char* row = static_cast<const char*>(a.logits) +
                      (r * a.ld + c0) * (int64_t)sizeof(typename Elem<DT>::type);
    const Run<DT> run(row, n);
    Stats st{-CUDART_INF_F, 0.0f, 0.0f};
    Peak peak{-CUDART_INF_F, -CUDART_INF_F, 0};
    const uint4* p = run.vec();
    for (int blk = 0; blk * (U * NT) < run.nv; ++blk) {
      const int v = blk * (U * NT) + tid, next = (blk + 1) * (U * NT);
      // The next block is brought to the L2 cache while this one is worked on
      // (4096 x 128256 bf16 with 8 alternatives: 195 us without, 178 with; 164 and
      // 158 without alternatives; two blocks ahead the same, four 187).
      if (tid == 0 && next < run.nv)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p + next),
                     "r"(min(U * NT, run.nv - next) * 16)
                     : "memory");
      uint4 w[U];
      if (next <= run.nv) {
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = ld_stream(p + v + u * NT);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          w[u] = v + u * NT < run.nv ? ld_stream(p + v + u * NT) : masked16<DT>();
      }
      float bm = -CUDART_INF_F;
#pragma unroll
      for (int h = 0; h < U; h += 2) {
        float x[2 * N];
        unpack16<DT>(w[h], x);
        unpack16<DT>(w[h + 1], x + N);
        const float lm = max_of<2 * N>(x);
        take<2 * N>(st, x, lm);
        if (TOP) bm = fmaxf(bm, lm);
      }
      if (TOP && peak.see(bm, blk)) {
#pragma unroll
        for (int u = 0; u < U; ++u) kept[u * NT + tid] = w[u];
      }
    }
    const int64_t odd = run.odd(tid);
    if (odd >= 0) {
      const float x[2] = {load1<DT>(row, odd), -CUDART_INF_F};
      take<2>(st, x, max_of<2>(x));
      // (a maximum here has no block: every block is looked at if it is chosen)
      if (TOP && x[0] > peak.m) peak.other = peak.m = x[0];
    }

    const bool nan = st.s != st.s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      st = join(st, Stats{__shfl_xor_sync(0xFFFFFFFFu, st.m, o),
                          __shfl_xor_sync(0xFFFFFFFFu, st.s, o),
                          __shfl_xor_sync(0xFFFFFFFFu, st.t, o)});
    unsigned long long best = 0;
    if constexpr (TOP)
      best = alternatives<DT, NT>(run, row, c0, peak, nan, a.top_k, kept, cand, &row_list[0], &n_cand);

    if constexpr (kWarps > 1) {
      if (lane == 0) part_stats[warp] = st;
      __syncthreads();
      if (warp == 0) {
        st = lane < kWarps ? part_stats[lane] : Stats{-CUDART_INF_F, 0.0f, 0.0f};
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
          st = join(st, Stats{__shfl_xor_sync(0xFFFFFFFFu, st.m, o),
                              __shfl_xor_sync(0xFFFFFFFFu, st.s, o),
                              __shfl_xor_sync(0xFFFFFFFFu, st.t, o)});
      }
    }
    if (parts > 1) {  // the row's other parts, through their shared memory
      if (warp == 0) {
        if (lane == 0) {
          row_stats[0] = st.m;
          row_stats[1] = st.s;
          row_stats[2] = st.t;
        }
        if constexpr (TOP) row_list[lane] = best;
      }
      cluster_barrier();
      if (rank == 0 && warp == 0)
        for (uint32_t q = 1; q < parts; ++q) {
          st = join(st, Stats{remote_f32(&row_stats[0], q), remote_f32(&row_stats[1], q),
                              remote_f32(&row_stats[2], q)});
          if constexpr (TOP) best = merge_desc(best, remote_u64(&row_list[lane], q), lane);
        }
      cluster_barrier();
    }
    if (rank == 0 && warp == 0) {
      st.m = __shfl_sync(0xFFFFFFFFu, st.m, 0);
      st.s = __shfl_sync(0xFFFFFFFFu, st.s, 0);
      const float m = st.m, s = st.s;
      const bool bad = s != s, none = !bad && m == -CUDART_INF_F;
      const float ls = logf(s);  // log sum e^(x - m)
      // log probability of a logit
      const auto lp = [&](float x) {
        return bad ? CUDART_NAN_F : none ? -CUDART_INF_F : (x - m) - ls;
      };
      if (lane == 0) {
        if (a.lse) a.lse[r] = bad ? CUDART_NAN_F : none ? m : m + ls;
        if (a.entropy) a.entropy[r] = bad ? CUDART_NAN_F : none ? 0.0f : ls - kLn2 * (st.t / s);
        if (a.logprob) {
          const int64_t at = a.targets[r];
          a.logprob[r] = at >= a.V ? CUDART_NAN_F
                         : at < 0  ? 0.0f
                                   : lp(load1<DT>(a.logits, r * a.ld + at));
        }
      }
      if constexpr (TOP) {
        if (lane < a.top_k) {
          a.top_ids[r * a.top_k + lane] = (int32_t)(0xFFFFFFFFu - (uint32_t)best);
          a.top_logprob[r * a.top_k + lane] = lp(key_value((uint32_t)(best >> 32)));
        }
      }
    }
    __syncthreads();  // the shared arrays are free for the next row
  }
}

cudaError_t launch_token_logprob(const void* logits, int64_t ld, int dtype, int64_t R, int64_t V,
                                 const int64_t* targets, float* logprob, float* lse,
                                 float* entropy, int top_k, int32_t* top_ids, float* top_logprob,
                                 cudaStream_t stream) {
  // CTAs of a row: as few as fill the device once (five CTAs per SM), none
  // with less than 4096 columns.  512 rows of 128256 bf16 with 8 alternatives
  // take 43 us so, 51 us with the device filled twice over.
  const int64_t want = (int64_t)sm_count() * 5;
  int parts = 1;
  while (parts < kLossCluster && R * parts < want && V / (2 * parts) >= 4096) parts *= 2;
  const int64_t part = ((V + parts - 1) / parts + 7) / 8 * 8;
  const LogprobArgs a{logits,  ld,  R,       V,     part,    targets,
                      logprob, lse, entropy, top_k, top_ids, top_logprob};
  const int64_t most = (int64_t)1 << 27;  // clusters of a grid; more rows go round
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((R < most ? R : most) * parts));
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)parts;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  // Threads of a CTA: short rows leave most of a wide CTA's time to its
  // joins (16000 rows of 8000 bf16, lse alone: 75 us with 64 threads, 101 with
  // 256); long ones want few joins (4096 x 128256 bf16 with 8 alternatives:
  // 194 us with 256 threads, 210 with 128), but where the rows alone do not
  // fill the device, smaller CTAs spread the joins (512 rows: 42 and 37 us, 100
  // rows: 25 and 19 us; a few rows are again faster with 256, 13 and 15 us).
  const bool few = R >= sm_count() / 2 && R < want;
#define GS_N(DT, NT, CTAS)                                                     \
  (cfg.blockDim = dim3(NT),                                                    \
   top_k ? cudaLaunchKernelEx(&cfg, token_logprob_kernel<DT, NT, CTAS, true>, a) \
         : cudaLaunchKernelEx(&cfg, token_logprob_kernel<DT, NT, CTAS, false>, a))
#define GS_F(DT)                                                              \
  return part <= 1536 ? GS_N(DT, 32, 32)                                      \
         : part <= 12288 ? GS_N(DT, 64, 16)                                   \
         : few ? GS_N(DT, 128, 10) : GS_N(DT, 256, 5)
  if (dtype == GS_F32) GS_F(GS_F32);
  if (dtype == GS_F16) GS_F(GS_F16);
  GS_F(GS_BF16);
#undef GS_F
#undef GS_N
}

// ---- backward --------------------------------------------------------------
// An elementwise pass: each logit is read once, p formed from lse, and the
// gradient written.  HBM-bound (the two tensors; 8192 x 128256 bf16 in 590 us, 7.1
// TB/s); about five instructions per element.  A CTA takes one run of a row and issues its loads before anything
// that waits for the row's scalars.

constexpr int kBwdThreads = 128;

// Columns of a thread's granule: 32 bytes of the wider type.
template <int DT, int OT>
constexpr int kGranule = (DT == GS_F32 || OT == GS_F32) ? 8 : 16;
constexpr int kBwdGranules = 2;  // per thread of a run
template <int DT, int OT>
constexpr int kBwdRun = kBwdThreads * kBwdGranules * kGranule<DT, OT>;

struct LogprobBwdArgs {
  const void* logits;
  int64_t ld, R, V;
  const int64_t* targets;
  const float* lse;
  const float* dlogprob;
  const float* entropy;
  const float* dentropy;
  const float* loss_scale;
  void* dlogits;
  int64_t ld_out;
  int runs;  // runs per row
  bool in_place;
};

// G elements' bits, loaded 16 or 32 bytes at a time or one by one.  Not
// through the read-only path: dlogits may be the logits.
template <int DT, int G>
struct Granule {
  static constexpr int kWords = G * (int)sizeof(typename Elem<DT>::type) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* base, int64_t i, bool vec) {
    const typename Elem<DT>::type* q = static_cast<const typename Elem<DT>::type*>(base) + i;
    if (vec) {
      if constexpr (kWords == 8) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(q));
      } else {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(q));
      }
    } else if constexpr (DT == GS_F32) {
#pragma unroll
      for (int j = 0; j < G; ++j) w[j] = __float_as_uint(q[j]);
    } else {
#pragma unroll
      for (int j = 0; j < G / 2; ++j) w[j] = (uint32_t)q[2 * j] | ((uint32_t)q[2 * j + 1] << 16);
    }
  }
  __device__ __forceinline__ void unpack(float* x) const {
    if constexpr (DT == GS_F32) {
#pragma unroll
      for (int j = 0; j < G; ++j) x[j] = __uint_as_float(w[j]);
    } else {
      using Tag = std::conditional_t<DT == GS_BF16, BF16Tag, F16Tag>;
#pragma unroll
      for (int j = 0; j < G / 2; ++j) {
        x[2 * j] = lo16<Tag>(w[j]);
        x[2 * j + 1] = hi16<Tag>(w[j]);
      }
    }
  }
  __device__ __forceinline__ void pack(const float* x) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (DT == GS_F32) {
        w[j] = __float_as_uint(x[j]);
      } else if constexpr (DT == GS_BF16) {
        w[j] = cvt_f32x2_bf16x2(x[2 * j + 1], x[2 * j]);
      } else {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
      }
    }
  }
  // base + i is aligned to the granule.
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    typename Elem<DT>::type* q = static_cast<typename Elem<DT>::type*>(base) + i;
    if constexpr (kWords == 8) {
      V8 v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v.w[j] = w[j];
      st_stream8(q, v);
    } else {
      st_stream(reinterpret_cast<uint4*>(q), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
};

template <int DT, int OT, bool ENT>
__global__ void __launch_bounds__(kBwdThreads, DT == GS_F32 ? 12 : 10)
    token_logprob_bwd_kernel(const LogprobBwdArgs a) {
  __shared__ float red[kBwdThreads / 32];
  constexpr int G = kGranule<DT, OT>, U = kBwdGranules;
  using In = Granule<DT, G>;
  using Out = Granule<OT, G>;
  const int run = blockIdx.x;
  for (int64_t r = blockIdx.y; r < a.R; r += gridDim.y) {
    const void* in = static_cast<const typename Elem<DT>::type*>(a.logits) + r * a.ld;
    void* out = static_cast<typename Elem<OT>::type*>(a.dlogits) + r * a.ld_out;
    // `head` columns up to the first granule boundary of the output
    constexpr uint32_t kAlign = Out::kWords * 4;
    int64_t head = (int64_t)((kAlign - ((uint32_t)(uintptr_t)out & (kAlign - 1))) & (kAlign - 1)) /
                   (int64_t)sizeof(typename Elem<OT>::type);
    if (head > a.V) head = a.V;
    const int64_t nv = (a.V - head) / G;
    const bool vec = ((uintptr_t)(static_cast<const typename Elem<DT>::type*>(in) + head) &
                      (In::kWords * 4 - 1)) == 0;
    In w[U];
    const auto fetch = [&](int64_t k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t v = (k * U + u) * kBwdThreads + threadIdx.x;
        if (v < nv) w[u].load(in, head + v * G, vec);
      }
    };
    fetch(run);

    const float S = a.loss_scale ? *a.loss_scale : 1.0f;
    const float l = a.lse[r];
    const int64_t at = a.targets[r];
    const bool none = l == -CUDART_INF_F;
    // S dlogprob and S dentropy of the row; a target beyond V makes it NaN
    const float g = at >= a.V ? CUDART_NAN_F : at < 0 || none ? 0.0f : S * a.dlogprob[r];
    const float ge = ENT ? (none ? 0.0f : S * a.dentropy[r]) : 0.0f;
    const float eh = ENT ? a.entropy[r] : 0.0f;
    // log of the row's sum of e^(x - lse), where lse's rounding shows.  In
    // place, the row must not be overwritten by another CTA meanwhile: the
    // first run's CTA then does the whole row.
    float ls = 0.0f;
    int runs = 1;
    if (fabsf(l) > kLseExact && !none) {
      if (a.in_place) {
        if (run > 0) continue;
        runs = a.runs;
      }
      // A granule's terms are summed as a tree, a thread's granules with the
      // rounding carried along (Kahan, "Further remarks on reducing truncation
      // errors", 1965): equal terms round alike, and 1000 of them one after another
      // are off by more than lse is.  (Unrolled, the loops cost the rows that skip
      // them: 1021 x 32003 fp16 with entropy 27.7 us, 27.2 so.)
      float s = 0.0f, lost = 0.0f;
      const auto add = [&](float v) {
        const float y = v - lost, t = s + y;
        lost = (t - s) - y;
        s = t;
      };
#pragma unroll 1
      for (int64_t v = threadIdx.x; v < nv; v += kBwdThreads) {
        float x[G];
        In q;
        q.load(in, head + v * G, vec);
        q.unpack(x);
        uint64_t e[G / 2];
#pragma unroll
        for (int j = 0; j < G; j += 2) {
          float e0, e1;
          upk_f32x2(mul_f32x2(add_f32x2(pk_f32x2(x[j], x[j + 1]), pk_f32x2(-l, -l)),
                              pk_f32x2(kLog2e, kLog2e)), e0, e1);
          e[j / 2] = pk_f32x2(ex2(e0), ex2(e1));
        }
#pragma unroll
        for (int n = G / 4; n > 0; n /= 2)
#pragma unroll
          for (int j = 0; j < n; ++j) e[j] = add_f32x2(e[j], e[j + n]);
        float lo, hi;
        upk_f32x2(e[0], lo, hi);
        add(lo + hi);
      }
#pragma unroll 1
      for (int64_t i = threadIdx.x; i < a.V - nv * G; i += kBwdThreads)
        add(ex2((load1<DT>(in, i < head ? i : nv * G + i) - l) * kLog2e));
      ls = logf(block_sum<kBwdThreads>(s, red));
    }
    const float base = none ? 0.0f : l;
    // gradient of two logits, without the target's own term; d stays above
    // -30000, where p is 0 all the same, so that a masked logit gives 0 and not
    // 0 * Inf
    const uint64_t nbase = pk_f32x2(-base, -base), nls = pk_f32x2(-ls, -ls);
    const uint64_t ng = pk_f32x2(-g, -g), nge = pk_f32x2(-ge, -ge), eh2 = pk_f32x2(eh, eh);
    const auto grad2 = [&](float& x0, float& x1) {
      uint64_t d = add_f32x2(add_f32x2(pk_f32x2(x0, x1), nbase), nls);
      if constexpr (ENT) {
        upk_f32x2(d, x0, x1);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(-30000.0f));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(-30000.0f));
        d = pk_f32x2(x0, x1);
      }
      float e0, e1;
      upk_f32x2(mul_f32x2(d, pk_f32x2(kLog2e, kLog2e)), e0, e1);
      const uint64_t p = pk_f32x2(ex2(e0), ex2(e1));
      upk_f32x2(mul_f32x2(p, ENT ? fma_f32x2(nge, add_f32x2(d, eh2), ng) : ng), x0, x1);
    };
    for (int k = run;; ++k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t v = ((int64_t)k * U + u) * kBwdThreads + threadIdx.x;
        if (v >= nv) continue;
        float x[G];
        w[u].unpack(x);
#pragma unroll
        for (int j = 0; j < G; j += 2) grad2(x[j], x[j + 1]);
        const uint64_t hot = (uint64_t)(at - (head + v * G));
        if (hot < G) {
#pragma unroll
          for (int j = 0; j < G; ++j)
            if (hot == (uint64_t)j) x[j] += g;
        }
        Out o;
        o.pack(x);
        o.store(out, head + v * G);
      }
      if (k + 1 >= run + runs) break;
      fetch(k + 1);
    }
    if (run == 0) {  // the columns outside the granules
      const int64_t odd = a.V - nv * G;
      for (int64_t i = threadIdx.x; i < odd; i += kBwdThreads) {
        const int64_t c = i < head ? i : nv * G + i;
        float x = load1<DT>(in, c), unused = 0.0f;
        grad2(x, unused);
        store1<OT>(out, c, x + (c == at ? g : 0.0f));
      }
    }
    if (gridDim.y < a.R) __syncthreads();  // `red` is free for the next row
  }
}

template <int DT, int OT>
static void bwd_launch(LogprobBwdArgs a, cudaStream_t stream) {
  a.runs = (int)((a.V + kBwdRun<DT, OT> - 1) / kBwdRun<DT, OT>);
  const dim3 grid((unsigned)a.runs, (unsigned)(a.R < 65535 ? a.R : 65535));
  if (a.dentropy)
    token_logprob_bwd_kernel<DT, OT, true><<<grid, kBwdThreads, 0, stream>>>(a);
  else
    token_logprob_bwd_kernel<DT, OT, false><<<grid, kBwdThreads, 0, stream>>>(a);
}

cudaError_t launch_token_logprob_bwd(const void* logits, int64_t ld, int dtype, int64_t R,
                                     int64_t V, const int64_t* targets, const float* lse,
                                     const float* dlogprob, const float* entropy,
                                     const float* dentropy, const float* loss_scale,
                                     void* dlogits, int64_t ld_out, int out_dtype,
                                     cudaStream_t stream) {
  const LogprobBwdArgs a{logits,   ld,         R,       V,      targets, lse, dlogprob, entropy,
                         dentropy, loss_scale, dlogits, ld_out, 0,       dlogits == logits};
#define GS_G(DT)                                                      \
  if (out_dtype == GS_F32) bwd_launch<DT, GS_F32>(a, stream);         \
  else if (out_dtype == GS_F16) bwd_launch<DT, GS_F16>(a, stream);    \
  else bwd_launch<DT, GS_BF16>(a, stream)
  if (dtype == GS_F32) { GS_G(GS_F32); }
  else if (dtype == GS_F16) { GS_G(GS_F16); }
  else { GS_G(GS_BF16); }
#undef GS_G
  return cudaGetLastError();
}

}  // namespace gs

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
// largest of the elements it read, so the k-th largest of the threads' maxima
// is a lower bound of the k-th largest logit (k elements reach it), and only
// the elements of threads whose maximum reaches it can be among the first k:
// about k threads' (a few in a thousand), read again out of L2 by one warp
// each.  A warp holds its k best in lane order and inserts candidates.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gs_elem.cuh"
#include "gs_internal.h"
#include "gs_quant.cuh"

namespace gs {

constexpr int kLossThreads = 512;
constexpr int kLossWarps = kLossThreads / 32;
constexpr int kLossCluster = 8;  // most CTAs of a row

// Beyond this |lse| its rounding to fp32 (2^-24 |lse|, the relative error it
// brings to every p) is no longer small beside the rest, and the gradient
// forms the row's sum anew.
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

// Brings (s, t) from maximum m to the larger M.  m = -Inf (nothing yet, s = 0)
// must not turn into 0 * Inf: the shift is kept finite.
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

// N logits at once (N even).  With ENT, d is kept above -1024, where 2^d is 0
// all the same, so that a masked logit adds 0 and not 0 * Inf to t.
template <bool ENT, int N>
__device__ __forceinline__ void take(Stats& a, const float* x) {
  float lm = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) lm = fmaxf(lm, x[i]);
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
    if constexpr (ENT) {
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(d0) : "f"(-1024.0f));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(d1) : "f"(-1024.0f));
    }
    const uint64_t e = pk_f32x2(ex2(d0), ex2(d1));
    s2 = add_f32x2(s2, e);
    if constexpr (ENT) t2 = fma_f32x2(e, pk_f32x2(d0, d1), t2);
  }
  float lo, hi;
  upk_f32x2(s2, lo, hi);
  a.s = lo + hi;
  if constexpr (ENT) {
    upk_f32x2(t2, lo, hi);
    a.t = lo + hi;
  }
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

// A run of a row: `head` elements up to the first 16-byte boundary, nv
// 16-byte vectors, then `tail` elements (head, tail < kVec).
template <int DT>
struct Run {
  const char* p;  // first element
  int head, tail;
  int64_t nv;
  static constexpr int kSize = sizeof(typename Elem<DT>::type);
  __device__ __forceinline__ Run(const void* base, int64_t n) : p(static_cast<const char*>(base)) {
    const int64_t h = (int64_t)((16u - ((uint32_t)(uintptr_t)p & 15u)) & 15u) / kSize;
    head = (int)(h < n ? h : n);
    nv = (n - head) / kVec<DT>;
    tail = (int)(n - head - nv * kVec<DT>);
  }
  __device__ __forceinline__ const uint4* vec() const {
    return reinterpret_cast<const uint4*>(p + head * kSize);
  }
  // Index of the odd element that thread i holds (the heads, then the
  // tails), or -1.
  __device__ __forceinline__ int64_t odd(int i) const {
    if (i < head) return i;
    return i < head + tail ? nv * kVec<DT> + i : -1;
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
// Merges the warps' lists; warp 0 returns the result.  `buf` holds
// kLossWarps * 32 values that no thread still reads.
template <typename T>
__device__ __forceinline__ T merge_warps(T v, T* buf, int warp, int lane) {
  buf[warp * 32 + lane] = v;
#pragma unroll
  for (int n = kLossWarps / 2; n > 0; n >>= 1) {
    __syncthreads();
    if (warp < n) {
      v = merge_desc(v, buf[(warp + n) * 32 + lane], lane);
      buf[warp * 32 + lane] = v;
    }
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

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// Shared memory of another CTA of the cluster, at the address of p in ours.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(d)
      : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return d;
}
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

template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLossThreads, 2)
    token_logprob_kernel(const LogprobArgs a) {
  __shared__ Stats part_stats[kLossWarps];
  __shared__ float row_stats[3];
  __shared__ unsigned long long lists[TOP ? kLossWarps * 32 : 1];
  __shared__ unsigned long long row_list[TOP ? 32 : 1];
  __shared__ int chosen[TOP ? kLossThreads : 1];
  __shared__ int n_chosen;
  __shared__ uint32_t tau_key;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t parts = cluster_size(), rank = cluster_rank();
  constexpr int N = kVec<DT>, U = 4;

  for (int64_t r = blockIdx.x / parts; r < a.R; r += gridDim.x / parts) {
    const int64_t c0 = a.part * rank < a.V ? a.part * rank : a.V;
    const int64_t n = a.V - c0 < a.part ? a.V - c0 : a.part;
    const char* row = static_cast<const char*>(a.logits) +
                      (r * a.ld + c0) * (int64_t)sizeof(typename Elem<DT>::type);
    const Run<DT> run(row, n);
    Stats st{-CUDART_INF_F, 0.0f, 0.0f};
    const uint4* p = run.vec();
    int64_t v = tid;
    for (; v + (U - 1) * kLossThreads < run.nv; v += U * kLossThreads) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = ld_stream(p + v + u * kLossThreads);
      float x[U * N];
#pragma unroll
      for (int u = 0; u < U; ++u) unpack16<DT>(w[u], x + u * N);
      take<ENT, U * N>(st, x);
    }
    for (; v < run.nv; v += kLossThreads) {
      float x[N];
      unpack16<DT>(ld_stream(p + v), x);
      take<ENT, N>(st, x);
    }
    const int64_t odd = run.odd(tid);
    if (odd >= 0) {
      const float x[2] = {load1<DT>(row, odd), -CUDART_INF_F};
      take<ENT, 2>(st, x);
    }

    unsigned long long best = 0;
    if constexpr (TOP) {
      // the threads' maxima, and the k-th largest of them
      uint32_t key = 0;
      if (st.s != st.s) {  // a NaN or +Inf was read: its key from the elements
        for (int64_t i = tid; i < run.nv; i += kLossThreads) {
          float x[N];
          unpack16<DT>(ld_stream(p + i), x);
#pragma unroll
          for (int j = 0; j < N; ++j) key = max(key, order_key(x[j]));
        }
        if (odd >= 0) key = max(key, order_key(load1<DT>(row, odd)));
      } else if (tid < run.nv || odd >= 0) {
        key = order_key(st.m);
      }
      if (tid == 0) n_chosen = 0;
      uint32_t* keys = reinterpret_cast<uint32_t*>(lists);
      const uint32_t top = merge_warps<uint32_t>(sort_desc(key, lane), keys, warp, lane);
      if (warp == 0 && lane == a.top_k - 1) tau_key = top;
      __syncthreads();
      const uint32_t tau = tau_key;
      if (key != 0 && key >= tau) chosen[atomicAdd(&n_chosen, 1)] = tid;
      __syncthreads();
      Best b{0, (unsigned long long)tau << 32, a.top_k};
      for (int g = warp; g < n_chosen; g += kLossWarps) {
        const int o = chosen[g];
        for (int64_t i0 = o; i0 < run.nv; i0 += (int64_t)32 * kLossThreads) {
          const int64_t i = i0 + (int64_t)lane * kLossThreads;
          const bool have = i < run.nv;
          float x[N];
          unpack16<DT>(have ? ld_stream(p + i) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
          for (int j = 0; j < N; ++j)
            b.offer(order_pair(x[j], (uint32_t)(c0 + run.head + i * N + j)), have, lane);
        }
        const int64_t i = run.odd(o);
        if (i >= 0) b.offer(order_pair(load1<DT>(row, i), (uint32_t)(c0 + i)), lane == 0, lane);
      }
      best = merge_warps<unsigned long long>(b.v, lists, warp, lane);
    }

#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      st = join(st, Stats{__shfl_xor_sync(0xFFFFFFFFu, st.m, o),
                          __shfl_xor_sync(0xFFFFFFFFu, st.s, o),
                          __shfl_xor_sync(0xFFFFFFFFu, st.t, o)});
    if (lane == 0) part_stats[warp] = st;
    __syncthreads();
    if (warp == 0) {
      st = lane < kLossWarps ? part_stats[lane] : Stats{-CUDART_INF_F, 0.0f, 0.0f};
#pragma unroll
      for (int o = kLossWarps / 2; o > 0; o >>= 1)
        st = join(st, Stats{__shfl_xor_sync(0xFFFFFFFFu, st.m, o),
                            __shfl_xor_sync(0xFFFFFFFFu, st.s, o),
                            __shfl_xor_sync(0xFFFFFFFFu, st.t, o)});
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
      const float m = __shfl_sync(0xFFFFFFFFu, st.m, 0), s = __shfl_sync(0xFFFFFFFFu, st.s, 0);
      const bool bad = s != s, none = !bad && m == -CUDART_INF_F;
      const float ls = logf(s);
      // log probability of a logit
      const auto lp = [&](float x) {
        return bad ? CUDART_NAN_F : none ? -CUDART_INF_F : (x - m) - ls;
      };
      if (lane == 0) {
        if (a.lse) a.lse[r] = bad ? CUDART_NAN_F : none ? m : m + ls;
        if (ENT) a.entropy[r] = bad ? CUDART_NAN_F : none ? 0.0f : ls - kLn2 * (st.t / s);
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
  // CTAs of a row: as few as fill the device several times over, none with
  // less than 4096 columns
  const int64_t want = (int64_t)sm_count() * 8;
  int parts = 1;
  while (parts < kLossCluster && R * parts < want && V / (2 * parts) >= 4096) parts *= 2;
  const int64_t part = ((V + parts - 1) / parts + 7) / 8 * 8;
  const LogprobArgs a{logits,  ld,  R,       V,     part,    targets,
                      logprob, lse, entropy, top_k, top_ids, top_logprob};
  const int64_t most = (int64_t)1 << 27;  // clusters of a grid; more rows go round
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((R < most ? R : most) * parts));
  cfg.blockDim = dim3(kLossThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)parts;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
#define GS_F(DT)                                                                               \
  (entropy ? (top_k ? cudaLaunchKernelEx(&cfg, token_logprob_kernel<DT, true, true>, a)        \
                    : cudaLaunchKernelEx(&cfg, token_logprob_kernel<DT, true, false>, a))      \
           : (top_k ? cudaLaunchKernelEx(&cfg, token_logprob_kernel<DT, false, true>, a)       \
                    : cudaLaunchKernelEx(&cfg, token_logprob_kernel<DT, false, false>, a)))
  if (dtype == GS_F32) return GS_F(GS_F32);
  if (dtype == GS_F16) return GS_F(GS_F16);
  return GS_F(GS_BF16);
#undef GS_F
}

// ---- backward --------------------------------------------------------------
// An elementwise pass: each logit is read once, p formed from lse, and the
// gradient written.  HBM-bound (the two tensors); about five instructions per
// element.

constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 4;                              // per thread of a run
constexpr int kBwdRun = kBwdThreads * kBwdVecs * 8;      // columns of a run

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
  int64_t ld_out, runs;  // runs per row
  bool in_place;
};

// Eight elements as fp32, by 16-byte loads or one by one.  Not through the
// read-only path: dlogits may be the logits.
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, bool vec, float* x) {
  const typename Elem<DT>::type* q = static_cast<const typename Elem<DT>::type*>(p) + i;
  if (vec) {
    const uint4* v = reinterpret_cast<const uint4*>(q);
    unpack16<DT>(v[0], x);
    if constexpr (DT == GS_F32) unpack16<DT>(v[1], x + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = Elem<DT>::get(q[j]);
  }
}
// Eight results; p + i is 16-byte aligned.
template <int OT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float* x) {
  uint4* q = reinterpret_cast<uint4*>(static_cast<typename Elem<OT>::type*>(p) + i);
  if constexpr (OT == GS_F32) {
    st_stream(q, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                            __float_as_uint(x[3])));
    st_stream(q + 1, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]),
                                __float_as_uint(x[6]), __float_as_uint(x[7])));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (OT == GS_BF16) {
        w[j] = cvt_f32x2_bf16x2(x[2 * j + 1], x[2 * j]);
      } else {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
      }
    }
    st_stream(q, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

template <int DT, int OT, bool ENT>
__global__ void __launch_bounds__(kBwdThreads)
    token_logprob_bwd_kernel(const LogprobBwdArgs a) {
  __shared__ float red[kBwdThreads / 32];
  const float S = a.loss_scale ? *a.loss_scale : 1.0f;
  for (int64_t w = blockIdx.x; w < a.R * a.runs; w += gridDim.x) {
    const int64_t r = w / a.runs, run = w - r * a.runs;
    const void* in =
        static_cast<const typename Elem<DT>::type*>(a.logits) + r * a.ld;
    void* out = static_cast<typename Elem<OT>::type*>(a.dlogits) + r * a.ld_out;
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
    int64_t last_run = run + 1;
    if (fabsf(l) > kLseExact && !none) {
      if (a.in_place) {
        if (run > 0) continue;
        last_run = a.runs;
      }
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < a.V; c += kBwdThreads)
        s += ex2((load1<DT>(in, c) - l) * kLog2e);
      ls = logf(block_sum<kBwdThreads>(s, red));
    }
    const float base = none ? 0.0f : l;
    // gradient of one logit; d stays above -30000, where p is 0 all the same,
    // so that a masked logit gives 0 and not 0 * Inf
    const auto grad = [&](float x) {
      float d = (x - base) - ls;
      if constexpr (ENT) asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(-30000.0f));
      const float p = ex2(d * kLog2e);
      return ENT ? p * __fmaf_rn(-ge, d + eh, -g) : p * -g;
    };
    // `head` columns up to the first 16-byte boundary of the output
    int64_t head = (int64_t)((16u - ((uint32_t)(uintptr_t)out & 15u)) & 15u) /
                   (int64_t)sizeof(typename Elem<OT>::type);
    if (head > a.V) head = a.V;
    const int64_t nv = (a.V - head) / 8;
    const bool vec =
        ((uintptr_t)(static_cast<const typename Elem<DT>::type*>(in) + head) & 15u) == 0;
    for (int64_t k = run; k < last_run; ++k) {
      const int64_t v0 = k * (kBwdRun / 8);
      float x[kBwdVecs][8];
  #pragma unroll
      for (int u = 0; u < kBwdVecs; ++u) {
        const int64_t v = v0 + u * kBwdThreads + threadIdx.x;
        if (v < nv) load8<DT>(in, head + v * 8, vec, x[u]);
      }
  #pragma unroll
      for (int u = 0; u < kBwdVecs; ++u) {
        const int64_t v = v0 + u * kBwdThreads + threadIdx.x;
        if (v >= nv) continue;
  #pragma unroll
        for (int j = 0; j < 8; ++j) x[u][j] = grad(x[u][j]);
        const uint64_t hot = (uint64_t)(at - (head + v * 8));
        if (hot < 8) {
  #pragma unroll
          for (int j = 0; j < 8; ++j)
            if (hot == (uint64_t)j) x[u][j] += g;
        }
        store8<OT>(out, head + v * 8, x[u]);
      }
    }
    if (run == 0) {  // the columns outside the vectors
      const int64_t odd = a.V - nv * 8;
      for (int64_t i = threadIdx.x; i < odd; i += kBwdThreads) {
        const int64_t c = i < head ? i : nv * 8 + i;
        store1<OT>(out, c, grad(load1<DT>(in, c)) + (c == at ? g : 0.0f));
      }
    }
    __syncthreads();  // `red` is free for the next run
  }
}

cudaError_t launch_token_logprob_bwd(const void* logits, int64_t ld, int dtype, int64_t R,
                                     int64_t V, const int64_t* targets, const float* lse,
                                     const float* dlogprob, const float* entropy,
                                     const float* dentropy, const float* loss_scale,
                                     void* dlogits, int64_t ld_out, int out_dtype,
                                     cudaStream_t stream) {
  const int64_t runs = (V + kBwdRun - 1) / kBwdRun;
  const LogprobBwdArgs a{logits,  ld,       R,          V,       targets, lse, dlogprob,
                         entropy, dentropy, loss_scale, dlogits, ld_out,  runs, dlogits == logits};
  const int64_t most = (int64_t)1 << 30;
  const unsigned grid = (unsigned)(R < most / runs ? R * runs : most);
#define GS_F(DT, OT)                                                               \
  if (dentropy)                                                                    \
    token_logprob_bwd_kernel<DT, OT, true><<<grid, kBwdThreads, 0, stream>>>(a);   \
  else                                                                             \
    token_logprob_bwd_kernel<DT, OT, false><<<grid, kBwdThreads, 0, stream>>>(a)
#define GS_G(DT)                                     \
  if (out_dtype == GS_F32) { GS_F(DT, GS_F32); }     \
  else if (out_dtype == GS_F16) { GS_F(DT, GS_F16); }\
  else { GS_F(DT, GS_BF16); }
  if (dtype == GS_F32) { GS_G(GS_F32) }
  else if (dtype == GS_F16) { GS_G(GS_F16) }
  else { GS_G(GS_BF16) }
#undef GS_G
#undef GS_F
  return cudaGetLastError();
}

}  // namespace gs

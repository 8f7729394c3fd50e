// layernorm.cu -- layer norm of rows and its backward pass, statistics and
// sums in fp32 ("Numerical Precision, Mixed Precision, and Loss Scaling",
// paragraph on autocast: normalisations run in fp32).
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y = (x - mean) rstd gamma + beta
//   d = dy gamma,  xhat = (x - mean) rstd
//   dx = rstd (d - sum d / C - xhat (sum d xhat) / C)
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
//
// xhat is formed from the difference, never as x rstd - mean rstd: where a
// row is nearly constant and eps small, the rounding of mean rstd would stand
// in xhat's place.
//
// Both passes are HBM-bound: forward 2 elements moved per element, backward 3.
//
// Many rows of 16 bits, forward, and rows of any type, backward, go through a
// ring of asynchronous copies in shared memory (below): each thread owns the
// same 16 bytes of every row, so that its weights and its share of dgamma and
// dbeta stay in registers.  Rows wider than 1024 threads' 16 bytes are a
// cluster's, whose CTAs write their sums into each other's shared memory.
// 16384 x 8192 bf16 takes 86 us forward (6.2 TB/s) and 146 us backward (5.5 TB/s);
// with odd rows (8001) 111 and 175 us.  What is left to the copy rate is issue: 65
// to 70 % of the issue slots are taken.
//
// Few rows, and fp32 forward: a row is read once into registers (at most 32
// values per thread), the variance formed about the mean from there (two block
// sums; a one-pass variance would cancel for rows far from zero), and written.  A
// warp takes a short row by itself, a CTA a long one.
//
// Rows that neither can take, element by element: a thread owns columns t + i nt.
// Longer rows than a CTA's registers hold are read again, out of L2 after the
// first time.
//
// dgamma and dbeta: each CTA writes one row of partial sums at its end, which a
// second kernel adds in a fixed order: no atomics, the result depends on the
// sizes and the device alone.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gs_elem.cuh"
#include "gs_internal.h"
#include "gs_quant.cuh"

namespace gs {

// ---- element vectors --------------------------------------------------------
// W consecutive elements as fp32: W = 1, or 16 bytes' worth (a whole vector,
// 16-byte aligned).
template <int DT>
constexpr int kVecElems = DT == GS_F32 ? 4 : 8;

template <int DT>
__device__ __forceinline__ void unpack_vec(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == GS_F32) {
      f[i] = __uint_as_float(w[i]);
    } else {
      using Tag = std::conditional_t<DT == GS_BF16, BF16Tag, F16Tag>;
      f[2 * i] = lo16<Tag>(w[i]);
      f[2 * i + 1] = hi16<Tag>(w[i]);
    }
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack_vec(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == GS_F32) {
      w[i] = __float_as_uint(f[i]);
    } else if constexpr (DT == GS_BF16) {
      w[i] = cvt_f32x2_bf16x2(f[2 * i + 1], f[2 * i]);
    } else {
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes of elements as pairs of fp32 for the packed operations.
template <int DT>
__device__ __forceinline__ void unpack_pairs(const uint4& v, uint64_t* p) {
  float f[kVecElems<DT>];
  unpack_vec<DT>(v, f);
#pragma unroll
  for (int i = 0; i < kVecElems<DT> / 2; ++i) p[i] = pk_f32x2(f[2 * i], f[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ uint4 pack_pairs(const uint64_t* p) {
  float f[kVecElems<DT>];
#pragma unroll
  for (int i = 0; i < kVecElems<DT> / 2; ++i) upk_f32x2(p[i], f[2 * i], f[2 * i + 1]);
  return pack_vec<DT>(f);
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float f) { return pk_f32x2(f, f); }
__device__ __forceinline__ float sum_of(uint64_t p) {
  float lo, hi;
  upk_f32x2(p, lo, hi);
  return lo + hi;
}

// W weights from column c; `missing` where there are none.  `vec`: the array
// is 16-byte aligned.
template <int WT, int W>
__device__ __forceinline__ void load_weights(const void* p, int64_t c, bool vec, float missing,
                                             float* f) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = missing;
  } else if (W * sizeof(typename Elem<WT>::type) >= 16 && vec) {
    const uint4* q =
        reinterpret_cast<const uint4*>(static_cast<const typename Elem<WT>::type*>(p) + c);
#pragma unroll
    for (int i = 0; i < W / kVecElems<WT>; ++i) unpack_vec<WT>(__ldg(q + i), f + i * kVecElems<WT>);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = load1<WT>(p, c + i);
  }
}

// ---- forward ----------------------------------------------------------------

struct NormArgs {
  const void* x;
  int64_t ldx, R, C;
  const void* gamma;
  const void* beta;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  bool w_vec;   // gamma and beta are 16-byte aligned (or absent)
  int classes;  // of rows by alignment
};

// Sum over the NT threads that share a row: a warp's, or the CTA's; `red`
// holds NT / 32 floats that no thread still reads.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (NT > 32) {
    constexpr int kWarps = NT / 32;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < kWarps ? red[lane] : 0.0f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (kWarps < 32) v = __shfl_sync(0xFFFFFFFFu, v, 0);
  }
  return v;
}

// NT threads per row, each with up to VPT vectors of W columns.
template <int DT, int WT, int W, int NT, int VPT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
    layernorm_fwd_kernel(const NormArgs a) {
  __shared__ float red[2][NT / 32];
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t r = NT >= 256 ? (int64_t)blockIdx.x
                              : ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / NT;
  if (r >= a.R) return;  // whole warps: NT < 256 has one row per warp
  static_assert(NT == 32 || NT >= 256, "a row is a warp's or a CTA's");
  const typename Elem<DT>::type* x = static_cast<const typename Elem<DT>::type*>(a.x) + r * a.ldx;
  typename Elem<DT>::type* y = static_cast<typename Elem<DT>::type*>(a.y) + r * a.ldy;
  const int C = (int)a.C;
  float f[VPT][W];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * W;
    if (c < C) {
      if constexpr (W > 1) unpack_vec<DT>(ld_stream(reinterpret_cast<const uint4*>(x + c)), f[i]);
      else f[i][0] = Elem<DT>::get(x[c]);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) f[i][j] = 0.0f;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) s += f[i][j];
  const float mu = __fdiv_rn(row_sum<NT>(s, red[0]), (float)C);
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if ((i * NT + tid) * W < C) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        f[i][j] -= mu;
        s = __fmaf_rn(f[i][j], f[i][j], s);
      }
    }
  const float var = __fdiv_rn(row_sum<NT>(s, red[1]), (float)C);
  const float rs = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * W;
    if (c < C) {
      float g[W], b[W];
      load_weights<WT, W>(a.gamma, c, a.w_vec, 1.0f, g);
      load_weights<WT, W>(a.beta, c, a.w_vec, 0.0f, b);
#pragma unroll
      for (int j = 0; j < W; ++j) f[i][j] = __fmaf_rn(f[i][j] * rs, g[j], b[j]);
      if constexpr (W > 1) st_stream(reinterpret_cast<uint4*>(y + c), pack_vec<DT>(f[i]));
      else y[c] = Elem<DT>::put(f[i][0]);
    }
  }
  if (tid == 0) {
    if (a.mean) a.mean[r] = mu;
    if (a.rstd) a.rstd[r] = rs;
  }
}

// ---- rows through a copy ring ----------------------------------------------
// Thread t owns vector t of every row (its weights stay in registers) and
// copies its part of the next rows into shared memory itself (cp.async), so
// that no thread waits for another's copy and the memory stays busy across
// the barriers.  Two rows (backward) or four (forward) share a barrier: the
// sums' latency, some 800 cycles of shuffles and barrier, would take half the
// time of a row otherwise.  A row is read from the ring again after the barrier:
// held in registers it costs spills (forward 110 us, so 89).
// The grid is planned for 1024 threads per SM with 64 registers each: one CTA per
// SM for rows of more than 512 threads, 32 for the narrowest, of which the shared
// memory of an SM (ring, sums and what the system keeps: some 9.5 KB each) holds 24
// at a time.  One CTA of 513 to 1023 threads leaves a part of the SM unused:
// 16384 x 5120, 6144 and 7168 bf16 take 62, 70 and 79 us forward, 102, 117 and 134 us
// backward, beside 52 and 86 us at 4096 and 89 and 148 us at 8192 columns (timed
// one by one, caches flushed).

// Sums of four values over the warp: lane 8 q and its seven neighbours return
// the sum of s[q].
__device__ __forceinline__ float warp_sum4(const float* s, int lane) {
  const bool hi = lane & 16, mid = lane & 8;
  const float u0 = (hi ? s[2] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? s[0] : s[2], 16);
  const float u1 = (hi ? s[3] : s[1]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? s[1] : s[3], 16);
  float v = (mid ? u1 : u0) + __shfl_xor_sync(0xFFFFFFFFu, mid ? u0 : u1, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Rows that do not begin or end on 16 bytes (EDGE; W elements are 16 bytes): in a
// tensor that begins on 16 bytes, rows W apart stand alike to the boundaries.
// Such rows are a class: each begins e elements behind a boundary, and in the
// other tensors too if their pitches agree modulo W.  A CTA takes rows of one
// class and a thread the W columns between two boundaries, so that all copies and
// stores are of 16 bytes but a row's first and last, whose threads have the
// columns [lo, hi) of their vector only.  A first vector's other bytes belong to
// the row before (or the gap), are read and left out; a last vector's are not
// read.  Only the warps of those two threads run the code that masks.
// Rows wider than a CTA's threads (WIDE) are a cluster's, rank 0 with the first of
// them.
template <int W, bool EDGE, bool WIDE>
struct RowClass {
  int C, K, k, e;          // columns; classes, this CTA's, and its e
  int64_t R, block, blocks;  // rows of the class; this CTA (or cluster) among the class's
  int c, lo, hi;
  bool live, partial;
  __device__ __forceinline__ RowClass(int classes, int64_t rows, int64_t columns, int64_t ld)
      : C((int)columns), K(EDGE ? classes : 1) {
    const uint32_t size = WIDE ? cluster_size() : 1, id = blockIdx.x / size;
    k = EDGE ? (int)(id % (uint32_t)K) : 0;
    e = EDGE ? (int)(k * ld % W) : 0;
    R = EDGE ? (rows - k + K - 1) / K : rows;
    block = EDGE ? id / (uint32_t)K : id;
    blocks = gridDim.x / size / (uint32_t)K;
    c = (int)(threadIdx.x + (WIDE ? cluster_rank() * blockDim.x : 0)) * W - e;
    live = c < C;
    lo = EDGE ? max(-c, 0) : 0;
    hi = EDGE ? min(C - c, W) : W;
    partial = EDGE && live && hi - lo < W;
  }
  __device__ __forceinline__ int64_t row(int64_t i) const { return EDGE ? k + K * i : i; }
  // columns of warp w
  __device__ __forceinline__ int columns_of(int w) const {
    const int from = w * 32 * W - e;
    return max(0, min(C, from + 32 * W) - max(0, from));
  }
  __device__ __forceinline__ bool has(int j) const { return j >= lo && j < hi; }
  template <int WT>
  __device__ __forceinline__ void weights(const void* p, bool vec, float missing, uint64_t* w) const {
    float f[W];
#pragma unroll
    for (int j = 0; j < W; ++j) f[j] = 0.0f;
    if (EDGE) {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (live && has(j)) load_weights<WT, 1>(p, c + j, false, missing, &f[j]);
    } else if (live) {
      load_weights<WT, W>(p, c, vec, missing, f);
    }
#pragma unroll
    for (int j = 0; j < W / 2; ++j) w[j] = pk_f32x2(f[2 * j], f[2 * j + 1]);
  }
  template <int DT>
  __device__ __forceinline__ void copy(uint32_t to, const typename Elem<DT>::type* from) const {
    if constexpr (EDGE) {
      const int bytes = hi * (int)sizeof(*from);  // the rest of the 16 is zeroed
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                   : "memory");
    } else {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
  }
  // The columns of the warp's partial vectors, which are in their slots of the
  // ring, to their places in an output row: a lane each, so that it is one store
  // instruction and not W.
  template <int DT>
  __device__ __forceinline__ void store_partial(typename Elem<DT>::type* to, const uint4* slot) const {
    const uint32_t edges = __ballot_sync(0xFFFFFFFFu, partial);
    const int lane = threadIdx.x & 31, first = __ffs(edges) - 1, last = 31 - __clz(edges);
    const int from = lane < W ? first : last, col = c + (from - lane) * W + lane % W;
    if ((lane < W || (lane < 2 * W && first != last)) && col >= 0 && col < C)
      to[col - c] = reinterpret_cast<const typename Elem<DT>::type*>(slot + (from - lane))[lane % W];
  }
};
// The bits of a vector that are the thread's own, as in memory and as fp32
// pairs: of a row's first thread, its last, and any other.
template <int DT>
struct EdgeMasks {
  static constexpr int W = kVecElems<DT>;
  uint4 raw[3];
  uint64_t pair[3][W / 2];
  __device__ __forceinline__ static int kind(bool partial, int c) { return !partial ? 2 : c > 0; }
  // By threads of one kind alike.
  __device__ __forceinline__ void make(int kind, int lo, int hi) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t keep = kind == 2 || (j >= lo && j < hi) ? 0xFFFFFFFFu : 0;
      w[j * 4 / W] |= W == 4 ? keep : keep & (j & 1 ? 0xFFFF0000u : 0x0000FFFFu);
      reinterpret_cast<uint32_t*>(pair[kind])[j] = keep;
    }
    raw[kind] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
__device__ __forceinline__ uint4 and4(const uint4& a, const uint4& b) {
  return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}
// Classes of rows `ld` elements apart.
static int row_classes(int64_t ld, int W) { return ld % W == 0 ? 1 : W; }

// CTAs of a ring kernel's grid, 1024 threads per SM, whole numbers of every
// class; `size` CTAs per row.  None if a row is too wide.
constexpr int kRingCluster = 8, kFwdCluster = 4;  // most CTAs of a row, backward and forward
struct RingPlan {
  int threads, size;
  int64_t ctas;
};
static RingPlan ring_plan(int64_t C, int W, int classes, bool edge, int most) {
  const int64_t vectors = std::max<int64_t>((C + (edge ? W - 1 : 0) + W - 1) / W, 1);
  int size = 1;
  while (size < most && vectors > 1024 * size) size *= 2;
  const int64_t threads = ((vectors + size - 1) / size + 31) / 32 * 32;
  if (threads > 1024) return RingPlan{0, 0, 0};
  const int64_t ctas = (int64_t)sm_count() * (1024 / threads) / (classes * size) * (classes * size);
  return RingPlan{(int)threads, size, ctas};
}

// Launches a ring kernel for R rows, `each` 16-byte words of ring per thread; the
// grid's CTAs (or clusters) of a row to *ctas.
template <typename Args>
static cudaError_t launch_ring(void (*kernel)(Args), const Args& a, const RingPlan& p, int classes,
                               int each, cudaStream_t stream, int64_t* ctas) {
  const void* const f = reinterpret_cast<const void*>(kernel);
  int per_sm = 0;  // (raises the kernel's shared-memory limit to the widest rows' need)
  cudaError_t e = kernel_blocks_per_sm(f, 1024, each * 1024 * 16, &per_sm);
  if (e != cudaSuccess) return e;
  const int smem = each * p.threads * 16;
  int64_t n = p.ctas / p.size;
  if (p.size > 1) {  // only resident clusters share the rows evenly
    int clusters = 0;
    e = kernel_clusters(f, p.threads, smem, p.size, &clusters);
    if (e != cudaSuccess) return e;
    if (clusters < n) n = std::max(clusters / classes, 1) * classes;
  }
  n = std::min(a.R, n);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n * p.size));
  cfg.blockDim = dim3((unsigned)p.threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)p.size;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = p.size > 1 ? 1 : 0;
  *ctas = n;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

constexpr int kFwdRows = 4, kFwdGroups = 3;  // forward: rows that share a barrier, groups in the ring
constexpr int kBwdGroups = 3;                // backward: pairs of rows in the ring

template <int DT, int WT, bool EDGE, bool WIDE>
__global__ void __launch_bounds__(1024, 1) layernorm_fwd_ring_kernel(const NormArgs a) {
  constexpr int W = kVecElems<DT>, P = W / 2, D = kFwdGroups, Q = kFwdRows;
  constexpr int S = WIDE ? kFwdCluster : 1;
  static_assert(Q == 4, "the joins below are of four rows");
  extern __shared__ uint4 ring[];  // [D][Q][blockDim.x]
  // Of each CTA of the row, per row of the group: the warps' means, and their
  // squared deviations; every CTA of the cluster has them all.
  __shared__ float4 part_mean[2][S][Q][8], part_dev[2][S][Q][8];
  __shared__ float4 columns[S][8];  // of the row, each warp's
  const uint32_t ranks = WIDE ? cluster_size() : 1, rank = WIDE ? cluster_rank() : 0;
  __shared__ EdgeMasks<DT> masks;
  const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, warp = tid >> 5, lane = tid & 31;
  const RowClass<W, EDGE, WIDE> own(a.classes, a.R, a.C, a.ldx);
  const int c = own.c, row8 = lane >> 3;  // row8: the group's row that this lane joins
  const bool live = own.live;
  const int64_t ldx = own.K * a.ldx, ldy = own.K * a.ldy;
  const typename Elem<DT>::type* x =
      static_cast<const typename Elem<DT>::type*>(a.x) + own.k * a.ldx + c;
  typename Elem<DT>::type* y = static_cast<typename Elem<DT>::type*>(a.y) + own.k * a.ldy + c;
  uint64_t g[P], b[P];
  own.template weights<WT>(a.gamma, a.w_vec, 1.0f, g);
  own.template weights<WT>(a.beta, a.w_vec, 0.0f, b);
  const int kind = EdgeMasks<DT>::kind(own.partial, c);
  if (EDGE && live) masks.make(kind, own.lo, own.hi);
  const bool edge_warp = EDGE && __any_sync(0xFFFFFFFFu, own.partial);
  const float n_own = EDGE ? (float)max(own.hi - own.lo, 1) : (float)W;
  const float inv_own = EDGE ? __frcp_rn(n_own) : 1.0f / W;
  if (tid < 32)
    for (int q = 0; q < S; ++q)
      reinterpret_cast<float*>(columns[q])[tid] =
          tid < warps ? (float)own.columns_of(q * warps + tid) : 0.0f;
  const float inv = __fdiv_rn(1.0f, (float)a.C);
  for (int i = tid; i < 2 * S * Q * 8; i += nt)  // of warps that do not exist
    (&part_mean[0][0][0][0])[i] = (&part_dev[0][0][0][0])[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
  if constexpr (WIDE) cluster_barrier();  // before another CTA's sums arrive
  const float inv_warp = __fdiv_rn(1.0f, fmaxf(reinterpret_cast<float*>(columns[rank])[warp], 1.0f));

  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(ring + tid);
  const int64_t stride = own.blocks * Q, first = own.block * Q;
  // the rows left from the group to copy next, and from the group in hand
  int64_t ahead = own.R - first, rows = own.R - first;
  const typename Elem<DT>::type* from = x + first * ldx;
  typename Elem<DT>::type* to = y + first * ldy;
  const auto copy_group = [&](int slot) {
    const uint32_t at = slot0 + slot * Q * nt * 16;
#pragma unroll
    for (int i = 0; i < Q; ++i)
      if (live && ahead > i) own.template copy<DT>(at + i * nt * 16, from + i * ldx);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead -= stride;
    from += stride * ldx;
  };
#pragma unroll
  for (int i = 0; i < D; ++i) copy_group(i);
  int slot = 0, side = 0;
  for (; rows > 0; rows -= stride, to += stride * ldy) {
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    uint4* mine = ring + slot * Q * nt + tid;
    // this thread's sums, and its squared deviations from its own means
    float s[Q], dev[Q];
    const auto sums = [&](auto edge) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        uint4 raw = live && rows > i ? mine[i * nt] : make_uint4(0, 0, 0, 0);
        if constexpr (edge.value) raw = and4(raw, masks.raw[kind]);
        uint64_t f[P], t = 0;
        unpack_pairs<DT>(raw, f);
        uint64_t sum = f[0];
#pragma unroll
        for (int j = 1; j < P; ++j) sum = add_f32x2(sum, f[j]);
        s[i] = sum_of(sum);
        const uint64_t m2 = both(-s[i] * (edge.value ? inv_own : 1.0f / W));
#pragma unroll
        for (int j = 0; j < P; ++j) {
          f[j] = add_f32x2(f[j], m2);
          if constexpr (edge.value) f[j] &= masks.pair[kind][j];
          t = fma_f32x2(f[j], f[j], t);
        }
        dev[i] = sum_of(t);
      }
    };
    if (EDGE && edge_warp) sums(std::integral_constant<bool, EDGE>());
    else sums(std::false_type());
    // this warp's means, and the squared deviations from them
    const float wm = warp_sum4(s, lane) * inv_warp;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const float d = __fmaf_rn(s[i], inv_own, -__shfl_sync(0xFFFFFFFFu, wm, 8 * i));
      s[i] = live ? __fmaf_rn(n_own * d, d, dev[i]) : 0.0f;
    }
    const float wq = warp_sum4(s, lane);
    float mu, var;  // of row `row8` of the group, in this lane
    if (WIDE || warps > 1) {
      if ((lane & 7) == 0) {
        float* const at_mean = reinterpret_cast<float*>(part_mean[side][rank][row8]) + warp;
        float* const at_dev = reinterpret_cast<float*>(part_dev[side][rank][row8]) + warp;
        if constexpr (WIDE) {
          for (uint32_t q = 0; q < ranks; ++q) {
            store_remote_f32(at_mean, q, wm);
            store_remote_f32(at_dev, q, wq);
          }
        } else {
          *at_mean = wm;
          *at_dev = wq;
        }
      }
      if constexpr (WIDE) {
        __syncwarp();
        cluster_barrier();
      } else {
        __syncthreads();
      }
      // four warps' sums, each with its columns (fewer in the last one)
      float t = 0.0f;
#pragma unroll 1  // (unrolled, the other CTAs' sums cost spills)
      for (uint32_t q = 0; q < ranks; ++q) {
        const float4 m = part_mean[side][q][row8][lane & 7], n = columns[q][lane & 7];
        t += __fmaf_rn(n.x, m.x, n.y * m.y) + __fmaf_rn(n.z, m.z, n.w * m.w);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
      mu = t * inv;
      t = 0.0f;
#pragma unroll 1  // (unrolled, the other CTAs' sums cost spills)
      for (uint32_t q = 0; q < ranks; ++q) {
        const float4 m = part_mean[side][q][row8][lane & 7], n = columns[q][lane & 7];
        const float4 v = part_dev[side][q][row8][lane & 7];
        const float d0 = m.x - mu, d1 = m.y - mu, d2 = m.z - mu, d3 = m.w - mu;
        t += (__fmaf_rn(n.x * d0, d0, v.x) + __fmaf_rn(n.y * d1, d1, v.y)) +
             (__fmaf_rn(n.z * d2, d2, v.z) + __fmaf_rn(n.w * d3, d3, v.w));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
      var = t * inv;
      side ^= 1;  // free again: every thread passes the next barrier after these reads
    } else {
      mu = wm;
      var = wq * inv;
    }
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
    if (rank == 0 && warp == 0 && (lane & 7) == 0 && rows > row8) {
      const int64_t at = own.row(own.R - rows + row8);
      if (a.mean) a.mean[at] = mu;
      if (a.rstd) a.rstd[at] = rs;
    }
    const auto finish = [&](auto edge) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const uint64_t scale2 = both(__shfl_sync(0xFFFFFFFFu, rs, 8 * i));
        const uint64_t m2 = both(-__shfl_sync(0xFFFFFFFFu, mu, 8 * i));
        if (!(live && rows > i)) continue;
        uint64_t f[P];
        unpack_pairs<DT>(mine[i * nt], f);
#pragma unroll
        for (int j = 0; j < P; ++j)
          f[j] = fma_f32x2(mul_f32x2(add_f32x2(f[j], m2), scale2), g[j], b[j]);
        if (edge.value && own.partial) mine[i * nt] = pack_pairs<DT>(f);
        else st_stream(reinterpret_cast<uint4*>(to + i * ldy), pack_pairs<DT>(f));
      }
      if constexpr (edge.value) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < Q; ++i)
          if (rows > i) own.template store_partial<DT>(to + i * ldy, mine + i * nt);
        __syncwarp();  // before the slots' next copies
      }
    };
    if (EDGE && edge_warp) finish(std::integral_constant<bool, EDGE>());
    else finish(std::false_type());
    copy_group(slot);
    slot = slot + 1 < D ? slot + 1 : 0;
  }
}

// Rows of any alignment, element by element: thread t of a CTA just wide
// enough holds columns t + i blockDim.x, their weights for all of the CTA's
// rows.
template <int DT, int WT, int EPT>
__global__ void __launch_bounds__(1024) layernorm_fwd_elem_kernel(const NormArgs a) {
  __shared__ float red[2][2][32];
  const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, lane = tid & 31;
  const int left = (int)a.C - tid;  // columns i with i nt < left are this thread's
  const float inv = __fdiv_rn(1.0f, (float)a.C);
  constexpr uint32_t kSize = sizeof(typename Elem<DT>::type);
  float g[EPT], b[EPT];
  uint32_t at[EPT];  // byte offsets in a row; beyond it the last column's, so that every
                     // load is in bounds without a condition
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    at[i] = (uint32_t)min(tid + i * nt, (int)a.C - 1) * kSize;
    g[i] = b[i] = 0.0f;
    if (i * nt < left) {
      load_weights<WT, 1>(a.gamma, tid + i * nt, false, 1.0f, &g[i]);
      load_weights<WT, 1>(a.beta, tid + i * nt, false, 0.0f, &b[i]);
    }
  }
  const auto row_sum = [&](float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps > 1) {
      if (lane == 0) part[tid >> 5] = v;
      __syncthreads();
      v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    return v;
  };
  int side = 0;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + r * a.ldx * (int64_t)kSize;
    char* y = static_cast<char*>(a.y) + r * a.ldy * (int64_t)kSize;
    typename Elem<DT>::type raw[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      raw[i] = *reinterpret_cast<const typename Elem<DT>::type*>(x + at[i]);
    float f[EPT], s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      f[i] = Elem<DT>::get(raw[i]);
      s += i * nt < left ? f[i] : 0.0f;
    }
    const float mu = row_sum(s, red[side][0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      f[i] = i * nt < left ? f[i] - mu : 0.0f;
      s = __fmaf_rn(f[i], f[i], s);
    }
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fmaf_rn(row_sum(s, red[side][1]), inv, a.eps)));
    side ^= 1;  // free again: every thread passes two barriers after these reads
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      if (i * nt < left)
        *reinterpret_cast<typename Elem<DT>::type*>(y + at[i]) =
            Elem<DT>::put(__fmaf_rn(f[i] * rs, g[i], b[i]));
    if (tid == 0) {
      if (a.mean) a.mean[r] = mu;
      if (a.rstd) a.rstd[r] = rs;
    }
  }
}

// Rows of any length, read three times.
constexpr int kLongThreads = 1024;
template <int DT, int WT>
__global__ void __launch_bounds__(kLongThreads) layernorm_fwd_long_kernel(const NormArgs a) {
  __shared__ float red[2][kLongThreads / 32];
  const int64_t r = blockIdx.x, xo = r * a.ldx, yo = r * a.ldy;
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < a.C; c += kLongThreads) s += load1<DT>(a.x, xo + c);
  const float mu = __fdiv_rn(row_sum<kLongThreads>(s, red[0]), (float)a.C);
  s = 0.0f;
  for (int64_t c = threadIdx.x; c < a.C; c += kLongThreads) {
    const float d = load1<DT>(a.x, xo + c) - mu;
    s = __fmaf_rn(d, d, s);
  }
  const float var = __fdiv_rn(row_sum<kLongThreads>(s, red[1]), (float)a.C);
  const float rs = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
  for (int64_t c = threadIdx.x; c < a.C; c += kLongThreads) {
    float g, b;
    load_weights<WT, 1>(a.gamma, c, false, 1.0f, &g);
    load_weights<WT, 1>(a.beta, c, false, 0.0f, &b);
    store1<DT>(a.y, yo + c, __fmaf_rn((load1<DT>(a.x, xo + c) - mu) * rs, g, b));
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[r] = mu;
    if (a.rstd) a.rstd[r] = rs;
  }
}

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

template <int DT, int WT>
static cudaError_t fwd_launch(const NormArgs& a, cudaStream_t stream) {
  constexpr int V = kVecElems<DT>;
  const bool vec = aligned16(a.x) && aligned16(a.y) && a.C % V == 0 && a.ldx % V == 0 &&
                   a.ldy % V == 0;
  const unsigned rows = (unsigned)a.R, warps = (unsigned)((a.R + 7) / 8);
#define GS_L(W, NT, VPT)                                                                      \
  layernorm_fwd_kernel<DT, WT, W, NT, VPT>                                                    \
      <<<NT == 32 ? warps : rows, NT == 32 ? 256 : NT, 0, stream>>>(a)
  // The ring where a CTA gets a group of rows at least (8192 columns of
  // bf16 on alignment: 608 rows 9.6 us, 8.7 from registers; 1216 rows 11 and 15;
  // 16384 rows 87 and 132), and the rows of no alignment are not narrow
  // (16384 x 4097 fp16 82 us, 109 element by element; 16384 x 1001: 21 and 26; 100000
  // x 501: 69 and 67).  fp32 has enough bytes in flight without (16384 x 4096: 81
  // us from registers, 98 through the ring).
  if constexpr (DT != GS_F32) {
    const bool edge = !vec && aligned16(a.x) && aligned16(a.y) && (a.ldx - a.ldy) % V == 0;
    const int classes = edge ? a.classes : 1;
    // Wide rows: a cluster's ring against the next paths below (8192 x 16384 bf16,
    // two CTAs: 124 and 142 us; 4096 x 32768, four: 150 and 179; 2048 x 65536, eight:
    // 249 and 217; off alignment, 4000 x 12001, two: 66 and 98; 8192 x 16383, four: 240
    // and 222).
    const RingPlan p = ring_plan(a.C, V, classes, edge, edge ? 2 : kFwdCluster);
    if ((vec || (edge && a.C > 512)) && p.ctas > 0 && a.R >= p.ctas / p.size * kFwdRows) {
      void (*const kernel)(NormArgs) =
          edge ? (p.size > 1 ? layernorm_fwd_ring_kernel<DT, WT, true, true>
                             : layernorm_fwd_ring_kernel<DT, WT, true, false>)
               : (p.size > 1 ? layernorm_fwd_ring_kernel<DT, WT, false, true>
                             : layernorm_fwd_ring_kernel<DT, WT, false, false>);
      int64_t ctas = 0;
      return launch_ring(kernel, a, p, classes, kFwdGroups * kFwdRows, stream, &ctas);
    }
  }
  if (vec) {
    // A row's threads: a warp while it holds the row in four vectors a lane (fp32,
    // 262144 x 128: 57 us with one vector each, 71 with a warp of four; 65536 x 512: 44,
    // 99 with 256 threads), then CTAs with as many vectors a thread as keep several of
    // them on an SM (16384 x 4096: 81 us with 256 threads, 95 with 512; 8192 x 8192: 85
    // with 512, 106 with 1024).
    const int64_t nv = a.C / V;
    if (nv <= 32) GS_L(V, 32, 1);
    else if (nv <= 128) GS_L(V, 32, 4);
    else if (nv <= 512) GS_L(V, 256, 2);
    else if (nv <= 1024) GS_L(V, 256, 4);
    else if (nv <= 2048) GS_L(V, 512, 4);
    else if (nv <= 4096) GS_L(V, 1024, 4);
    else layernorm_fwd_long_kernel<DT, WT><<<rows, kLongThreads, 0, stream>>>(a);
  } else {
    // A warp per row up to 128 columns (262144 x 100 bf16 64 us, 66 by the next), then
    // CTAs of eight columns per thread, 8192 threads per SM: several rounds of them.
    // (Sixteen columns per thread for twice the width: 4000 x 15000 117 us, 124 by the
    // last, but 4000 x 10000 93 and 90.)
    constexpr int kEach = 8;
    const unsigned nt = (unsigned)((a.C + kEach * 32 - 1) / (kEach * 32) * 32);
    if (a.C <= 128) GS_L(1, 32, 4);
    else if (a.C <= 1024 * kEach)
      layernorm_fwd_elem_kernel<DT, WT, kEach>
          <<<(unsigned)std::min<int64_t>(a.R, (int64_t)sm_count() * (8192 / nt)), nt, 0, stream>>>(a);
    else layernorm_fwd_long_kernel<DT, WT><<<rows, kLongThreads, 0, stream>>>(a);
  }
#undef GS_L
  return cudaGetLastError();
}

// Runs `f` with the two type codes as template arguments: w_dtype is GS_F32
// or dtype.
#define GS_NORM_TYPES(dtype, w_dtype, F)                        \
  if (dtype == GS_F32) { F(GS_F32, GS_F32) }                    \
  else if (dtype == GS_F16) {                                   \
    if (w_dtype == GS_F32) { F(GS_F16, GS_F32) }                \
    else { F(GS_F16, GS_F16) }                                  \
  } else {                                                      \
    if (w_dtype == GS_F32) { F(GS_BF16, GS_F32) }               \
    else { F(GS_BF16, GS_BF16) }                                \
  }

cudaError_t launch_layernorm_fwd(const void* x, int64_t ldx, int dtype, int64_t R, int64_t C,
                                 const void* gamma, const void* beta, int w_dtype, float eps,
                                 void* y, int64_t ldy, float* mean, float* rstd,
                                 cudaStream_t stream) {
  const int64_t esz = dtype == GS_F32 ? 4 : 2, most = (int64_t)1 << 30;
  for (int64_t r0 = 0; r0 < R; r0 += most) {  // rows of one grid
    const NormArgs a{static_cast<const char*>(x) + r0 * ldx * esz, ldx,
                     std::min(most, R - r0), C, gamma, beta, eps,
                     static_cast<char*>(y) + r0 * ldy * esz, ldy,
                     mean ? mean + r0 : nullptr, rstd ? rstd + r0 : nullptr,
                     aligned16(gamma) && aligned16(beta), row_classes(ldx, dtype == GS_F32 ? 4 : 8)};
    cudaError_t e = cudaSuccess;
#define GS_F(DT, WT) e = fwd_launch<DT, WT>(a, stream);
    GS_NORM_TYPES(dtype, w_dtype, GS_F)
#undef GS_F
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ---- backward ---------------------------------------------------------------

struct NormBwdArgs {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx, R, C;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  int64_t lddx;
  float* ws;  // [2, gridDim.x, C] partial sums, or nullptr
  bool w_vec;
  int classes;  // of rows by alignment
};

// The two sums of a row over the CTA, the same in every thread; `red` holds
// one float2 per warp that no thread still reads.
__device__ __forceinline__ float2 row_sum2(float s1, float s2, float2* red, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
    s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
  }
  if (warps > 1) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = make_float2(s1, s2);
    __syncthreads();
    const float2 p = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    s1 = p.x;
    s2 = p.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
      s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
    }
  }
  return make_float2(s1, s2);
}

// Rows 16 bytes at a time, two per barrier; registers hold the weights and both
// sums' accumulators.
template <int DT, int WT, bool EDGE, bool WIDE>
__global__ void __launch_bounds__(1024, 1) layernorm_bwd_ring_kernel(const NormBwdArgs a) {
  constexpr int W = kVecElems<DT>, D = kBwdGroups, S = WIDE ? kRingCluster : 1;
  extern __shared__ uint4 ring[];  // [D][2][x, dy][blockDim.x]
  // Of each CTA of the row, per value of the pair's four: the warps' sums, four a
  // float4; every CTA of the cluster has them all.
  __shared__ float4 part4[2][S][32];
  float* const part = reinterpret_cast<float*>(part4);  // [2][S][4][32]
  const uint32_t ranks = WIDE ? cluster_size() : 1, rank = WIDE ? cluster_rank() : 0;
  __shared__ float4 stats[D][32];  // a pair's means and rstd, one copy per warp
  __shared__ EdgeMasks<DT> masks;
  const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, warp = tid >> 5, lane = tid & 31;
  const RowClass<W, EDGE, WIDE> own(a.classes, a.R, a.C, a.ldx);
  const int c = own.c;
  const bool live = own.live;
  const int64_t ldx = own.K * a.ldx, lddy = own.K * a.lddy, lddx = own.K * a.lddx;
  const typename Elem<DT>::type* x =
      static_cast<const typename Elem<DT>::type*>(a.x) + own.k * a.ldx + c;
  const typename Elem<DT>::type* dy =
      static_cast<const typename Elem<DT>::type*>(a.dy) + own.k * a.lddy + c;
  typename Elem<DT>::type* dx = static_cast<typename Elem<DT>::type*>(a.dx) + own.k * a.lddx + c;
  constexpr int P = W / 2;  // pairs of columns
  uint64_t g[P], ag[P], ab[P];
#pragma unroll
  for (int j = 0; j < P; ++j) ag[j] = ab[j] = 0;
  own.template weights<WT>(a.gamma, a.w_vec, 1.0f, g);
  const int kind = EdgeMasks<DT>::kind(own.partial, c);
  if (EDGE && live) masks.make(kind, own.lo, own.hi);
  const bool edge_warp = EDGE && __any_sync(0xFFFFFFFFu, own.partial);
  const float inv = __fdiv_rn(1.0f, (float)a.C);
  for (int i = tid; i < 256 * S; i += nt) part[i] = 0.0f;  // of warps that do not exist
  __syncthreads();
  if constexpr (WIDE) cluster_barrier();  // before another CTA's sums arrive

  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(ring + tid);
  const uint32_t stat0 = (uint32_t)__cvta_generic_to_shared(&stats[0][warp]);
  const int64_t stride = own.blocks * 2, first = own.block * 2;
  // the rows left from the pair to copy next, and from the pair in hand
  int64_t ahead = own.R - first, rows = own.R - first;
  const typename Elem<DT>::type* from_x = x + first * ldx;
  const typename Elem<DT>::type* from_dy = dy + first * lddy;
  typename Elem<DT>::type* to_dx = dx + first * lddx;
  const auto copy_pair = [&](int slot) {
    const uint32_t at = slot0 + slot * 4 * nt * 16;
    if (live && ahead > 0) {
      own.template copy<DT>(at, from_x);
      own.template copy<DT>(at + nt * 16, from_dy);
    }
    if (live && ahead > 1) {
      own.template copy<DT>(at + nt * 32, from_x + ldx);
      own.template copy<DT>(at + nt * 48, from_dy + lddy);
    }
    // the rows' statistics, for the warp: lanes 0, 1 the means, 2, 3 rstd
    if (lane < 4 && ahead > (lane & 1))
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(stat0 + slot * 512 + lane * 4),
                   "l"((lane < 2 ? a.mean : a.rstd) + own.row(own.R - ahead + (lane & 1)))
                   : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead -= stride;
    from_x += stride * ldx;
    from_dy += stride * lddy;
  };
#pragma unroll
  for (int i = 0; i < D; ++i) copy_pair(i);
  int slot = 0, side = 0;
  for (; rows > 0; rows -= stride, to_dx += stride * lddx) {
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    __syncwarp();  // the statistics are other lanes' copies
    const float4 st = stats[slot][warp];
    const float mu[2] = {st.x, st.y}, rs[2] = {st.z, st.w};
    uint4* mine = ring + slot * 4 * nt + tid;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const auto sums = [&](auto edge) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (!(live && rows > q)) continue;
        uint4 rx = mine[2 * q * nt], rd = mine[(2 * q + 1) * nt];
        if constexpr (edge.value) {
          rx = and4(rx, masks.raw[kind]);
          rd = and4(rd, masks.raw[kind]);
        }
        uint64_t h[P], d[P], s1 = 0, s2 = 0;
        unpack_pairs<DT>(rx, h);
        unpack_pairs<DT>(rd, d);
        const uint64_t scale = both(rs[q]), m2 = both(-mu[q]);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          h[j] = mul_f32x2(add_f32x2(h[j], m2), scale);
          ab[j] = add_f32x2(ab[j], d[j]);
          ag[j] = fma_f32x2(d[j], h[j], ag[j]);
          d[j] = mul_f32x2(d[j], g[j]);
          s1 = add_f32x2(s1, d[j]);
          s2 = fma_f32x2(d[j], h[j], s2);
        }
        s[2 * q] = sum_of(s1);
        s[2 * q + 1] = sum_of(s2);
      }
    };
    if (EDGE && edge_warp) sums(std::integral_constant<bool, EDGE>());
    else sums(std::false_type());
    float t = warp_sum4(s, lane);
    if (WIDE || warps > 1) {
      if ((lane & 7) == 0) {
        float* const at = part + ((side * S + rank) * 4 + (lane >> 3)) * 32 + warp;
        if constexpr (WIDE) {
          for (uint32_t q = 0; q < ranks; ++q) store_remote_f32(at, q, t);
        } else {
          *at = t;
        }
      }
      if constexpr (WIDE) {
        __syncwarp();
        cluster_barrier();
      } else {
        __syncthreads();
      }
      t = 0.0f;
#pragma unroll
      for (int q = 0; q < S; ++q) {
        const float4 p = part4[side][q][lane];  // value lane / 8, four warps of it
        t += (p.x + p.y) + (p.z + p.w);
      }
      side ^= 1;  // free again: every thread passes the next barrier after these reads
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    t *= inv;
    const auto finish = [&](auto edge) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float c1 = __shfl_sync(0xFFFFFFFFu, t, 16 * q);
        const float c2 = __shfl_sync(0xFFFFFFFFu, t, 16 * q + 8);
        if (!(live && rows > q)) continue;
        uint64_t h[P], d[P];
        unpack_pairs<DT>(mine[2 * q * nt], h);
        unpack_pairs<DT>(mine[(2 * q + 1) * nt], d);
        const uint64_t scale = both(rs[q]), m2 = both(-mu[q]);
        const uint64_t n1 = both(-c1), n2 = both(-c2 * rs[q]);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          h[j] = add_f32x2(h[j], m2);
          d[j] = mul_f32x2(fma_f32x2(h[j], n2, fma_f32x2(d[j], g[j], n1)), scale);
        }
        if (edge.value && own.partial) mine[2 * q * nt] = pack_pairs<DT>(d);
        else st_stream(reinterpret_cast<uint4*>(to_dx + (q ? lddx : 0)), pack_pairs<DT>(d));
      }
      if constexpr (edge.value) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (rows > q) own.template store_partial<DT>(to_dx + (q ? lddx : 0), mine + 2 * q * nt);
        __syncwarp();  // before the slots' next copies
      }
    };
    if (EDGE && edge_warp) finish(std::integral_constant<bool, EDGE>());
    else finish(std::false_type());
    copy_pair(slot);
    slot = slot + 1 < D ? slot + 1 : 0;
  }
  asm volatile("griddepcontrol.launch_dependents;");  // the join may take this SM next
  if (!a.ws) return;
  float* pg = a.ws + (int64_t)(blockIdx.x / ranks) * a.C;
  float* pb = pg + (int64_t)(gridDim.x / ranks) * a.C;
  if constexpr (EDGE) {  // through the ring, all of its copies done and read
    float* sum = reinterpret_cast<float*>(ring);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
      if (live) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          float v[2];
          upk_f32x2(side ? ab[j / 2] : ag[j / 2], v[0], v[1]);
          if (own.has(j)) sum[tid * W + j] = v[j & 1];
        }
      }
      __syncthreads();
      const int from = c - tid * W;  // the first thread's
      for (int i = tid; i < nt * W; i += nt)
        if (from + i >= 0 && from + i < a.C) (side ? pb : pg)[from + i] = sum[i];
    }
  } else if (live) {
    pg += c;
    pb += c;
#pragma unroll
    for (int j = 0; j < P; j += 2) {  // C is a multiple of 4: the rows of ws are aligned
      *reinterpret_cast<ulonglong2*>(pg + 2 * j) = make_ulonglong2(ag[j], ag[j + 1]);
      *reinterpret_cast<ulonglong2*>(pb + 2 * j) = make_ulonglong2(ab[j], ab[j + 1]);
    }
  }
}

// Rows of any alignment, element by element: thread t owns columns t + i nt.
// The next row's elements are loaded before this row's barrier.
template <int DT, int WT, int EPT, int NT, int CTAS>
__global__ void __launch_bounds__(NT, CTAS) layernorm_bwd_elem_kernel(const NormBwdArgs a) {
  __shared__ float2 red[2][32];
  const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, C = (int)a.C;
  constexpr uint32_t kSize = sizeof(typename Elem<DT>::type);
  float g[EPT], ag[EPT], ab[EPT];
  // Byte offsets in a row; beyond it the last column's, so that every load is in
  // bounds without a condition (its weight here is 0 and its sums are not kept).
  uint32_t at[EPT];
  typename Elem<DT>::type nx[EPT], nd[EPT];  // the next row's
  float nmu = 0.0f, nrs = 0.0f;
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int c = tid + i * nt;
    at[i] = (uint32_t)min(c, C - 1) * kSize;
    ag[i] = ab[i] = 0.0f;
    g[i] = 0.0f;
    if (c < C) load_weights<WT, 1>(a.gamma, c, false, 1.0f, &g[i]);
  }
  const float inv = __fdiv_rn(1.0f, (float)C);
  const auto fetch = [&](int64_t r) {
    if (r >= a.R) return;
    const char* rx = static_cast<const char*>(a.x) + r * a.ldx * (int64_t)kSize;
    const char* rd = static_cast<const char*>(a.dy) + r * a.lddy * (int64_t)kSize;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      nx[i] = *reinterpret_cast<const typename Elem<DT>::type*>(rx + at[i]);
      nd[i] = *reinterpret_cast<const typename Elem<DT>::type*>(rd + at[i]);
    }
    nmu = a.mean[r];
    nrs = a.rstd[r];
  };
  fetch(blockIdx.x);
  int side = 0;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const float rs = nrs, mu = nmu;
    float h[EPT], d[EPT];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      h[i] = (Elem<DT>::get(nx[i]) - mu) * rs;
      d[i] = Elem<DT>::get(nd[i]);
      ab[i] += d[i];
      ag[i] = __fmaf_rn(d[i], h[i], ag[i]);
      d[i] *= g[i];
      s1 += d[i];
      s2 = __fmaf_rn(d[i], h[i], s2);
    }
    fetch(r + gridDim.x);
    const float2 s = row_sum2(s1, s2, red[side], warps);
    side ^= 1;  // free again: every thread passes the next barrier after these reads
    const float c1 = s.x * inv, c2 = s.y * inv;
    char* out = static_cast<char*>(a.dx) + r * a.lddx * (int64_t)kSize;
#pragma unroll
    for (int i = 0; i < EPT; ++i)
      if (tid + i * nt < C)
        *reinterpret_cast<typename Elem<DT>::type*>(out + at[i]) =
            Elem<DT>::put(rs * __fmaf_rn(-h[i], c2, d[i] - c1));
  }
  asm volatile("griddepcontrol.launch_dependents;");
  if (a.ws) {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = tid + i * nt;
      if (c < C) {
        a.ws[(int64_t)blockIdx.x * C + c] = ag[i];
        a.ws[((int64_t)gridDim.x + blockIdx.x) * C + c] = ab[i];
      }
    }
  }
}

// Rows of any length: dx alone, the row read twice.
template <int DT, int WT>
__global__ void __launch_bounds__(kLongThreads) layernorm_dx_long_kernel(const NormBwdArgs a) {
  __shared__ float2 red[32];
  const int64_t r = blockIdx.x;
  const float mu = a.mean[r], rs = a.rstd[r];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = threadIdx.x; c < a.C; c += kLongThreads) {
    float g;
    load_weights<WT, 1>(a.gamma, c, false, 1.0f, &g);
    const float h = (load1<DT>(a.x, r * a.ldx + c) - mu) * rs;
    const float d = load1<DT>(a.dy, r * a.lddy + c) * g;
    s1 += d;
    s2 = __fmaf_rn(d, h, s2);
  }
  const float2 s = row_sum2(s1, s2, red, kLongThreads / 32);
  const float inv = __fdiv_rn(1.0f, (float)a.C), c1 = s.x * inv, c2 = s.y * inv;
  for (int64_t c = threadIdx.x; c < a.C; c += kLongThreads) {
    float g;
    load_weights<WT, 1>(a.gamma, c, false, 1.0f, &g);
    const float h = (load1<DT>(a.x, r * a.ldx + c) - mu) * rs;
    const float d = load1<DT>(a.dy, r * a.lddy + c) * g;
    store1<DT>(a.dx, r * a.lddx + c, rs * __fmaf_rn(-h, c2, d - c1));
  }
}

// Partial sums of dgamma and dbeta for those: CTA (i, j) adds rows i, i + P,
// ... of columns [256 j, 256 j + 256) and writes row i of ws [2, P, C].
constexpr int kDwThreads = 256;
template <int DT>
__global__ void __launch_bounds__(kDwThreads) layernorm_dw_long_kernel(const NormBwdArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kDwThreads + threadIdx.x, P = gridDim.y;
  if (c >= a.C) return;
  float sg = 0.0f, sb = 0.0f;
  for (int64_t r = blockIdx.y; r < a.R; r += P) {
    const float d = load1<DT>(a.dy, r * a.lddy + c);
    sg = __fmaf_rn(d, (load1<DT>(a.x, r * a.ldx + c) - a.mean[r]) * a.rstd[r], sg);
    sb += d;
  }
  a.ws[blockIdx.y * a.C + c] = sg;
  a.ws[(P + blockIdx.y) * a.C + c] = sb;
}

// Adds the P partial sums of each column: eight columns per CTA (a 32-byte
// sector of each row of ws), four rows per warp at a time, so that a few
// loads per thread, all in flight, cover every row; joined in a fixed order.
constexpr int kJoinCols = 8;
template <int OT>
__global__ void __launch_bounds__(1024)
    layernorm_join_kernel(const float* ws, int64_t P, int64_t C, void* dgamma, void* dbeta) {
  __shared__ float part[32][kJoinCols + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are written
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int step = warps * 4;  // rows of a step of the CTA
  const int64_t c = (int64_t)blockIdx.x * kJoinCols + (lane & 7);
  void* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (!out) return;
  ws += blockIdx.y * P * C;
  float s = 0.0f;
  if (c < C)
    for (int64_t i = warp * 4 + (lane >> 3); i < P; i += 8 * step) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = i + k * step < P ? ws[(i + k * step) * C + c] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  if (lane < kJoinCols) part[warp][lane] = s;
  __syncthreads();
  if (warp >= kJoinCols) return;
  s = lane < warps ? part[lane][warp] : 0.0f;  // warp w joins column w
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int64_t oc = (int64_t)blockIdx.x * kJoinCols + warp;
  if (lane == 0 && oc < C) store1<OT>(out, oc, s);
}

constexpr int kElems = 8;  // columns per thread of the element path
struct NormBwdPlan {
  int threads;
  int64_t ctas;
};
// One CTA's threads and the CTAs of the grid, where a thread owns `each`
// columns: 1024 threads per SM at most (64 registers each).
static NormBwdPlan bwd_plan(int64_t R, int64_t C, int64_t each, int64_t sm_threads = 1024) {
  const int64_t threads = ((C + each - 1) / each + 31) / 32 * 32;
  const int64_t per_sm = std::min<int64_t>(32, sm_threads / threads);
  return NormBwdPlan{(int)threads, std::min<int64_t>(R, sm_count() * per_sm)};
}
static int64_t long_partials(int64_t R) { return R < 128 ? R : 128; }

// Upper bound over the paths a call with these sizes may take (the alignment
// decides which).
int64_t layernorm_partials(int64_t R, int64_t C) {
  if (C == 0) return 0;
  int64_t most = long_partials(R);
  for (int64_t each : {8, 4})
    if (C <= 1024 * each) most = std::max(most, bwd_plan(R, C, each).ctas);
    else if (C <= 1024 * each * kRingCluster) most = std::max(most, std::min<int64_t>(R, sm_count()));
  return most;
}

template <int DT, int WT>
static cudaError_t bwd_launch(const NormBwdArgs& a, int64_t* partials, cudaStream_t stream) {
  constexpr int V = kVecElems<DT>;
  const bool vec = aligned16(a.x) && aligned16(a.dy) && aligned16(a.dx) && a.C % V == 0 &&
                   a.ldx % V == 0 && a.lddy % V == 0 && a.lddx % V == 0;
  // Through the ring, up to eight CTAs a row (8192 x 16384 bf16, two: 194 us, 450
  // with each row read twice and thrice; 2048 x 65536, eight: 290), on alignment
  // always; with rows of no alignment where a CTA gets a dozen of them and more
  // than 1024 columns (bf16, through the ring and element by element: 16384 x 8001
  // 175 and 391 us, 8000 x 2001 36 and 37, 4000 x 2001 27 and 23, 65536 x 1023 125
  // and 117; fp32, whose elements are twice as wide: 16384 x 2001 78 and 80).
  const bool edge = DT != GS_F32 && !vec && aligned16(a.x) && aligned16(a.dy) && aligned16(a.dx) &&
                    (a.ldx - a.lddy) % V == 0 && (a.ldx - a.lddx) % V == 0;
  const int classes = edge ? a.classes : 1;
  const RingPlan ring = ring_plan(a.C, V, classes, edge, kRingCluster);
  if (ring.ctas > 0 && (vec || (edge && a.C > 1024 && a.R >= 12 * ring.ctas / ring.size))) {
    void (*kernel)(NormBwdArgs) = ring.size > 1 ? layernorm_bwd_ring_kernel<DT, WT, false, true>
                                                : layernorm_bwd_ring_kernel<DT, WT, false, false>;
    if constexpr (DT != GS_F32)
      if (edge)
        kernel = ring.size > 1 ? layernorm_bwd_ring_kernel<DT, WT, true, true>
                               : layernorm_bwd_ring_kernel<DT, WT, true, false>;
    int64_t ctas = 0;
    const cudaError_t e = launch_ring(kernel, a, ring, classes, kBwdGroups * 4, stream, &ctas);
    if (e != cudaSuccess) return e;
    *partials = ctas;
  } else if (a.C <= 1024 * kElems) {
    // As many registers as the width leaves: 16384 x 4001 fp16 takes 117 us with
    // 512 threads of 128 registers, 189 us with 1024 of 64 that own four
    // columns each.
    const NormBwdPlan p = bwd_plan(a.R, a.C, kElems, a.C <= 2048 ? 768 : 1024);
    const unsigned ctas = (unsigned)p.ctas;
    if (a.C <= 2048)
      layernorm_bwd_elem_kernel<DT, WT, kElems, 256, 3><<<ctas, p.threads, 0, stream>>>(a);
    else if (a.C <= 4096)
      layernorm_bwd_elem_kernel<DT, WT, kElems, 512, 1><<<ctas, p.threads, 0, stream>>>(a);
    else if (a.C <= 6144)
      layernorm_bwd_elem_kernel<DT, WT, kElems, 768, 1><<<ctas, p.threads, 0, stream>>>(a);
    else
      layernorm_bwd_elem_kernel<DT, WT, kElems, 1024, 1><<<ctas, p.threads, 0, stream>>>(a);
    *partials = p.ctas;
  } else {
    const int64_t most = (int64_t)1 << 30;
    for (int64_t r0 = 0; r0 < a.R; r0 += most) {
      NormBwdArgs b = a;
      b.x = static_cast<const typename Elem<DT>::type*>(a.x) + r0 * a.ldx;
      b.dy = static_cast<const typename Elem<DT>::type*>(a.dy) + r0 * a.lddy;
      b.dx = static_cast<typename Elem<DT>::type*>(a.dx) + r0 * a.lddx;
      b.mean += r0;
      b.rstd += r0;
      b.R = std::min(most, a.R - r0);
      layernorm_dx_long_kernel<DT, WT><<<(unsigned)b.R, kLongThreads, 0, stream>>>(b);
    }
    if (a.ws) {
      *partials = long_partials(a.R);
      const dim3 grid((unsigned)((a.C + kDwThreads - 1) / kDwThreads), (unsigned)*partials);
      layernorm_dw_long_kernel<DT><<<grid, kDwThreads, 0, stream>>>(a);
    }
  }
  return cudaGetLastError();
}

cudaError_t launch_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                 int dtype, int64_t R, int64_t C, const void* gamma, int w_dtype,
                                 const float* mean, const float* rstd, void* dx, int64_t lddx,
                                 void* dgamma, void* dbeta, int dw_dtype, float* ws,
                                 cudaStream_t stream) {
  int64_t P = 0;
  if (R > 0) {
    const NormBwdArgs a{dy,   lddy, x,  ldx,  R,  C, gamma, mean, rstd, dx,
                        lddx, ws,   aligned16(gamma), row_classes(ldx, dtype == GS_F32 ? 4 : 8)};
    cudaError_t e = cudaSuccess;
#define GS_F(DT, WT) e = bwd_launch<DT, WT>(a, &P, stream);
    GS_NORM_TYPES(dtype, w_dtype, GS_F)
#undef GS_F
    if (e != cudaSuccess) return e;
  }
  if (!dgamma && !dbeta) return cudaSuccess;
  // launched while the sums' kernel ends; it waits for them on the device
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((C + kJoinCols - 1) / kJoinCols), 2);
  cfg.blockDim = dim3(P <= 256 ? 256 : 1024);  // one step of eight loads per thread
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const float* cws = ws;
  if (dw_dtype == GS_F32)
    return cudaLaunchKernelEx(&cfg, layernorm_join_kernel<GS_F32>, cws, P, C, dgamma, dbeta);
  if (dw_dtype == GS_F16)
    return cudaLaunchKernelEx(&cfg, layernorm_join_kernel<GS_F16>, cws, P, C, dgamma, dbeta);
  return cudaLaunchKernelEx(&cfg, layernorm_join_kernel<GS_BF16>, cws, P, C, dgamma, dbeta);
}

}  // namespace gs

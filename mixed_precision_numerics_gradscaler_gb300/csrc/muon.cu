// muon.cu -- the update of weight matrices by their orthogonalised momentum
// (K. Jordan, "Muon: an optimizer for hidden layers in neural networks", 2024):
//   m = mu m + g,  u = g + mu m (nesterov) or m,  X = u / |u|_F,
//   steps times:  G = X X^T,  P = (a - 1) I + b G + c G G,  X = X + P X
//                 (for more rows than columns: G = X^T X, X = X + X P),
//   w = w (1 - lr weight_decay) - lr scale X,
// (a, b, c) = (3.4445, -4.7750, 2.0315), a quintic in the singular values that
// takes (0, 1] to near 1.
//
// The products take s^2 (l + s) operations each way of G and P with their
// symmetric halves left out, 2 s^2 l for X (twice, see below): all on the tensor cores.  Operands
// are fp16, not bf16: every value is bounded (singular values of X stay below
// 1.21, of G below 1.46, of P below 2.45), so that a power of two per matrix
// keeps them in fp16's normal range with three more bits than bf16 has, at the
// same rate.  Sums are fp32 in tensor memory and round to fp16 once per product;
// the last product's go into w unrounded.  One X is left out of P: where singular
// values are near 1, P is then the small difference between X and the result,
// and its rounding counts for as much.
// X is kept as two fp16 numbers, x and what it leaves, up to the last step, and P is
// applied to both.  A rounding of X is relative to its strongest directions and lies in
// all of them, and five steps raise weak ones up to 3.44^5 = 485 times: with x alone
// a matrix of 256 x 768 ended 9e-4 of its norm off where its spectrum was flat, 2.1e-2
// with one direction 1000 times the rest and 0.12 with one of 1e4; with both parts
// 9e-4, 5e-4 and 1.6e-3.  G and
// P need no second part: their roundings multiply X and lie in its own directions.
// The sum of P's product with the second part is another one as long: five steps take
// 1.4 to 1.5 times the operations (two of 14336 x 4096 5500 to 5850 us without, 7500 to
// 8300 with it).
// The last step's X is short of it: nothing raises its rounding any more.
//
// One cooperative launch takes every product of every step and matrix of the
// list: persistent pairs of CTAs walk the tiles of 256 x 256, half as wide where a
// list has few (every G, every P, every X of a step; longest sums first).  A tile waits until the matrix's tiles
// of the products before are stored, told by a count per matrix, so that one
// matrix's product fills the gap at the end of another's and nothing waits for
// a launch.  Pairs take their tiles in the common order, so the first tile that
// is not done never waits for one behind it.  A pair shares an MMA of
// 256 x 256 x 16, each CTA loading half of either operand (TMA, 64 x 64 boxes, five
// stages of 64 of the sum, or six narrow ones); operands lie with the sum along
// their rows or across them, which the MMA's descriptors tell.  Two accumulators:
// eight warps store one while the other is formed, each a quarter's rows of half the
// columns: what the sum is added to comes and what it becomes goes by TMA (stores
// by lanes took 13000 cycles a tile, these 4700).  Tiles above the diagonal of G
// and P are stored transposed from the ones below.
// Two matrices of 14336 x 4096 (7.9e12 operations, 11.7e12 with X's second part): the
// products 6.8 to 7.0 ms by themselves, 1.7 PFLOP/s, the tensor cores under the power
// cap; momentum and scaling 0.40 ms at the copy rate.  Twelve of 256 x 768: 164 us,
// fifteen products in a chain.
// Every wait is bounded and reports GS_ERR_TIMEOUT.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "gs_internal.h"
#include "gs_muon.h"
#include "gs_tcgen05.cuh"

namespace gs {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr int kMThreads = 384;               // warps 0-3: loads, MMA, two idle; 4-11 store
constexpr int kMEThreads = 256;              // of the element-wise steps
constexpr int kMRuns = (int)(kMuonChunk / (4 * kMEThreads));  // of four elements, per thread
constexpr int kMBox = 64 * 128;              // bytes of a 64 x 64 box
constexpr int kMPiece = 32 * 128;            // bytes of a warp's 32 rows x 64 columns of fp16
constexpr int kMKeys = 128;                  // matrices whose first tiles are kept in shared memory
// Sizes for tiles of 256 x BN.
template <int BN>
struct Mu {
  static constexpr int kBBoxes = BN / 128;               // a CTA's half of B's columns
  static constexpr int kStage = (2 + kBBoxes) * kMBox;   // and 128 rows of A
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kGroups = BN / 128;               // of 64 columns, per storing warp
  static constexpr int kSmem = kStages * kStage + 8 * 2 * kMPiece + 8 * kMKeys + 1024 + 512;
  static_assert(kSmem <= 232448, "dynamic shared memory above the per-CTA limit");
};

// The matrix that holds item t: the last one whose first is not above t.
template <typename T>
__device__ __forceinline__ int mat_of(const MuonMat* mats, int n, T t, T MuonMat::*first) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mats[mid].*first <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float clip_of(const MuonArgs& a) {
  if (!(a.max_norm > 0.0f)) return 1.0f;
  const float n = *a.grad_norm;
  return n > a.max_norm ? __fdiv_rn(a.max_norm, n) : 1.0f;
}

// Four elements from p + i; whole and aligned, or up to n.
template <int DT>
__device__ __forceinline__ void get4(const void* p, int64_t i, int64_t n, bool vec, float (&v)[4]) {
  using T = typename Elem<DT>::type;
  if (vec && i + 4 <= n) {
    if constexpr (DT == GS_F32) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const T*>(p) + i);
      v[0] = Elem<DT>::get((T)(w.x & 0xFFFFu)), v[1] = Elem<DT>::get((T)(w.x >> 16));
      v[2] = Elem<DT>::get((T)(w.y & 0xFFFFu)), v[3] = Elem<DT>::get((T)(w.y >> 16));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? load1<DT>(p, i + j) : 0.0f;
  }
}

// m = mu m + clip g, and the sum of squares of u.  CTAs take chunks by turns (runs
// of chunks, a few hundred KB apart at any time, took 1.7 times as long); what one
// has of a matrix is one part of its sum, and the last part to arrive forms the
// factor sx / |u| from all of them in their order.
template <int DT>
__global__ void __launch_bounds__(kMEThreads) muon_momentum_kernel(MuonTable t, MuonArgs a) {
  if (*a.found_inf) return;
  __shared__ double red[kMEThreads / 32];
  __shared__ bool last;
  const float clip = clip_of(a);
  float sum = 0.0f;
  int64_t begun = -1;  // this CTA's first chunk of the matrix
  int64_t chunks = 0;
  int id = 0;
  MuonMat mat = {};    // (a copy: what is stored could be the table, to the compiler)
  bool vec_m = false, vec_g = false;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    if (c >= mat.first_chunk + chunks) {
      id = mat_of(t.mats, t.n, c, &MuonMat::first_chunk);
      mat = t.mats[id];
      chunks = ((int64_t)mat.rows * mat.cols + kMuonChunk - 1) / kMuonChunk;
      vec_m = (uintptr_t)mat.m % 16 == 0;
      vec_g = (uintptr_t)mat.g % 16 == 0;
    }
    const int64_t n = (int64_t)mat.rows * mat.cols, base = (c - mat.first_chunk) * kMuonChunk;
    const int64_t end = min(n, base + kMuonChunk);
    if (base == 0 && threadIdx.x == 0) t.done[id] = 0;  // for the products' launch
    // everything is loaded before anything is stored: the loads do not wait for
    // one another
    float g[kMRuns][4], m[kMRuns][4];
#pragma unroll
    for (int j = 0; j < kMRuns; ++j) {
      const int64_t i = base + (j * kMEThreads + threadIdx.x) * 4;
      if (i < end) {
        get4<DT>(mat.g, i, end, vec_g, g[j]);
        get4<GS_F32>(mat.m, i, end, vec_m, m[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kMRuns; ++j) {
      const int64_t i = base + (j * kMEThreads + threadIdx.x) * 4;
      if (i >= end) continue;
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gc = __fmul_rn(g[j][e], clip);
        m[j][e] = __fmaf_rn(a.mu, m[j][e], gc);
        const float u = a.nesterov ? __fmaf_rn(a.mu, m[j][e], gc) : m[j][e];
        sq = __fmaf_rn(u, u, sq);
      }
      sum = __fadd_rn(sum, sq);
      if (vec_m && i + 4 <= end) {
        *reinterpret_cast<float4*>(mat.m + i) = make_float4(m[j][0], m[j][1], m[j][2], m[j][3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < end) mat.m[i + e] = m[j][e];
      }
    }
    if (begun < 0) begun = c;
    if (c + gridDim.x < mat.first_chunk + chunks) continue;
    // this CTA's part of the matrix's sum.  A thread's is of groups of four squares in
    // fp32, all positive: 200 additions for 32 M elements and 3400 for 2^31, 2^-24 of
    // the sum each at most (1.2e-5, 2e-4; half of that in the norm); fp64 from there
    double part = (double)sum;
    sum = 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_down_sync(0xFFFFFFFFu, part, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = part;
    __syncthreads();
    const int64_t parts = min(chunks, (int64_t)gridDim.x);  // their places: the first chunks
    if (threadIdx.x == 0) {
      part = red[0];
      for (int w = 1; w < kMEThreads / 32; ++w) part += red[w];
      t.partials[begun] = part;
      __threadfence();
      last = atomicAdd(&t.arrived[id], 1u) == (unsigned)parts - 1;
      __threadfence();
    }
    __syncthreads();
    if (last) {
      double all = 0.0;
      for (int64_t k = threadIdx.x; k < parts; k += kMEThreads)
        all += __ldcg(&t.partials[mat.first_chunk + k]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_down_sync(0xFFFFFFFFu, all, o);
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = all;
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int w = 1; w < kMEThreads / 32; ++w) all += red[w];
        // a momentum of zeros stays one; one whose squares have no sum shows as NaN
        t.factor[id] = all == 0.0 ? 0.0f
                       : all < (double)INFINITY ? (float)((double)mat.sx / sqrt(all))
                                                : __uint_as_float(0x7FFFFFFFu);
        t.arrived[id] = 0;
      }
    }
    __syncthreads();
    begun = -1;
  }
}

// x[0] = fp16(u sx / |u|), and what that leaves.
template <int DT>
__global__ void __launch_bounds__(kMEThreads) muon_scale_kernel(MuonTable t, MuonArgs a) {
  if (*a.found_inf) return;
  const float clip = clip_of(a);
  int64_t chunks = 0;
  MuonMat mat = {};
  bool vec_m = false, vec_g = false;
  float f = 0.0f;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    if (c >= mat.first_chunk + chunks) {
      const int id = mat_of(t.mats, t.n, c, &MuonMat::first_chunk);
      mat = t.mats[id];
      chunks = ((int64_t)mat.rows * mat.cols + kMuonChunk - 1) / kMuonChunk;
      vec_m = (uintptr_t)mat.m % 16 == 0;
      vec_g = (uintptr_t)mat.g % 16 == 0;
      f = t.factor[id];
    }
    const int64_t n = (int64_t)mat.rows * mat.cols, base = (c - mat.first_chunk) * kMuonChunk;
    const int64_t end = min(n, base + kMuonChunk);
    const bool rows4 = mat.cols % 4 == 0;  // four elements lie in one row
    float g[kMRuns][4], m[kMRuns][4];
#pragma unroll
    for (int j = 0; j < kMRuns; ++j) {
      const int64_t i = base + (j * kMEThreads + threadIdx.x) * 4;
      if (i < end) {
        get4<GS_F32>(mat.m, i, end, vec_m, m[j]);
        if (a.nesterov) get4<DT>(mat.g, i, end, vec_g, g[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kMRuns; ++j) {
      const int64_t i = base + (j * kMEThreads + threadIdx.x) * 4;
      if (i >= end) continue;
      uint16_t h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = a.nesterov ? __fmaf_rn(a.mu, m[j][e], __fmul_rn(g[j][e], clip)) : m[j][e];
        const float x = __fmul_rn(u, f);
        h[e] = Elem<GS_F16>::put(x);
        l[e] = Elem<GS_F16>::put(__fsub_rn(x, Elem<GS_F16>::get(h[e])));
      }
      unsigned row = (unsigned)i / (unsigned)mat.cols, col = (unsigned)i - row * (unsigned)mat.cols;
      if (rows4) {  // i + 4 <= end: the matrix is a multiple of 4
        *reinterpret_cast<uint2*>(mat.x[0] + (int64_t)row * mat.ldx + col) =
            make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        if (a.steps > 1)
          *reinterpret_cast<uint2*>(mat.x_lo[0] + (int64_t)row * mat.ldx + col) =
              make_uint2(l[0] | (uint32_t)l[1] << 16, l[2] | (uint32_t)l[3] << 16);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (i + e < end) {
            mat.x[0][(int64_t)row * mat.ldx + col] = h[e];
            if (a.steps > 1) mat.x_lo[0][(int64_t)row * mat.ldx + col] = l[e];
          }
          if (++col == (unsigned)mat.cols) col = 0, ++row;
        }
      }
    }
  }
}

// ---- products -----------------------------------------------------------------
enum { kGram, kPoly, kApply, kLast };

// Instruction descriptor: fp16 operands, fp32 sums, 256 x n; t: the operand's sum
// dimension runs across its rows.
__device__ __forceinline__ uint32_t idesc16(int n, bool ta, bool tb) {
  return (1u << 4) | (ta ? 1u << 15 : 0u) | (tb ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kMuonTile >> 4) << 24);
}
__device__ __forceinline__ void mma16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Step kk (16 of the sum) of a stage's 128 x 64 operand.  Sum along the rows: two
// boxes of 64 rows, 32 bytes a step.  Across: boxes of 64 (of 128) x 64 of the
// sum, a step is 16 rows of 128 bytes, the boxes 8192 bytes apart.
__device__ __forceinline__ uint64_t desc16(uint32_t base, int kk, bool across) {
  if (!across) return tc_desc_k(base + 32 * kk);
  return (uint64_t)(((base + 2048 * kk) >> 4) & 0x3FFFu) | ((uint64_t)(kMBox >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// One tile of a step's products: where it lies and what it takes.
struct Product {
  int kind, turn;        // turn: which of x[0], x[1] the step reads
  int id;                // matrix
  int m0, n0;            // first row and column of the result
  int M, N, K;
  bool ta, tb;           // operand with its sum across the rows
  int map_a, map_b;      // of the matrix's maps
  bool lo_in, lo_out;    // x's low part takes part, is stored
  int map_a_lo, map_b_lo;  // with lo_in: the operands of the sum's second half
  bool mirror;           // a tile below the diagonal
  unsigned need;         // sixteenths of the matrix's tiles to be stored before
};
// The step's tiles in their order: every matrix's G, every P, every X.
// keys: the matrices' first tiles of either kind, or null to read them from memory.
template <int BN>
__device__ __forceinline__ Product product(const MuonTable& t, const int* keys, int at, int steps) {
  Product p;
  const int per = 2 * t.sym_tiles + t.app_tiles, step = at / per;
  at -= step * per;
  p.turn = step & 1;
  const bool sym = at < 2 * t.sym_tiles;
  if (sym) {
    p.kind = at < t.sym_tiles ? kGram : kPoly;
    if (p.kind == kPoly) at -= t.sym_tiles;
  } else {
    p.kind = step + 1 < steps ? kApply : kLast;
    at -= 2 * t.sym_tiles;
  }
  if (keys) {
    const int* k = keys + (sym ? 0 : kMKeys);
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (k[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    p.id = lo;
  } else {
    p.id = mat_of(t.mats, t.n, at, sym ? &MuonMat::first_sym : &MuonMat::first_app);
  }
  const MuonMat& mat = t.mats[p.id];
  at -= sym ? mat.first_sym : mat.first_app;
  const int done = step * (2 * mat.syms + mat.apps);
  p.need = 16u * (unsigned)(done + (p.kind == kGram ? 0 : p.kind == kPoly ? mat.syms : 2 * mat.syms));
  int mt, nt;
  if (sym) {  // row mt of a triangle holds squares mt (mt + 1) / 2 ..., of one or two tiles
    constexpr int kW = kMuonTile / BN;
    const int sq = at / kW;
    mt = (int)((sqrtf(8.0f * (float)sq + 1.0f) - 1.0f) * 0.5f);
    while ((mt + 1) * (mt + 2) / 2 <= sq) ++mt;
    while (mt * (mt + 1) / 2 > sq) --mt;
    nt = at - kW * (mt * (mt + 1) / 2);
    p.M = p.N = mat.s;
    p.mirror = nt < kW * mt;
  } else {
    const int tm = (mat.rows + kMuonTile - 1) / kMuonTile, tn = (mat.cols + BN - 1) / BN;
    tc_tile(at, 8, tm, tn, mt, nt);
    p.M = mat.rows;
    p.N = mat.cols;
    p.mirror = false;
  }
  p.m0 = mt * kMuonTile;
  p.n0 = nt * BN;
  p.lo_in = p.kind == kApply;
  p.lo_out = p.lo_in && step + 2 < steps;
  if (p.kind == kGram) {
    p.K = mat.tall ? mat.rows : mat.cols;
    p.ta = p.tb = mat.tall;
    p.map_a = p.map_b = p.turn;
  } else if (p.kind == kPoly) {
    p.K = mat.s;
    p.ta = p.tb = false;
    p.map_a = p.map_b = 2;
  } else {
    p.K = mat.s;
    p.ta = false;
    p.tb = !mat.tall;
    p.map_a = mat.tall ? p.turn : 3;
    p.map_b = mat.tall ? 3 : p.turn;
  }
  p.map_a_lo = mat.tall ? 4 + p.turn : p.map_a;
  p.map_b_lo = mat.tall ? p.map_b : 4 + p.turn;
  return p;
}

// Before a CTA's first use of a tensor map in global memory.
__device__ __forceinline__ void map_fence(const CUtensorMap* m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.sys [%0], 128;" ::"l"(m) : "memory");
}
__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Bounded wait for *p >= need; a whole warp goes on or gives up together.
__device__ __forceinline__ bool wait_done(const unsigned* p, unsigned need, volatile int* abort_flag,
                                          int32_t* status) {
  bool ok = true;
  if (load_acquire(p) < need) {
    const uint64_t t0 = tc_now();
    while (load_acquire(p) < need) {
      if (*abort_flag) ok = false;
      if (tc_now() - t0 > kTcWaitNs) {
        *abort_flag = 1;
        atomicExch(status, (int32_t)GS_ERR_TIMEOUT);
        ok = false;
      }
      if (!ok) break;
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// Two fp32 values -> two fp16 (round to nearest even), hi in the high half.
__device__ __forceinline__ uint32_t cvt_f32x2_f16x2(float hi, float lo) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// w = w decay - to_w o and its bf16 copy, of 32 rows (one per lane's o) and 32
// columns from (row0, col): by way of buf (4096 bytes), so that neighbouring
// lanes take neighbouring columns.
__device__ __forceinline__ void update_weights(const MuonMat& mat, float* buf, const float* o, int row0,
                                               int col, float decay, float to_w) {
  if (col >= mat.cols) return;
  const int lane = threadIdx.x & 31;
  const auto piece = [&](int r, int j) { return buf + 32 * r + 4 * (j ^ (r & 7)); };
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(piece(lane, j)) = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  __syncwarp();
  const bool vec = mat.cols % 4 == 0 && (uintptr_t)mat.w % 16 == 0 && (uintptr_t)mat.wb % 8 == 0;
  if (vec) {  // eight lanes to a row
    const int c4 = col + 4 * (lane & 7), r0 = row0 + (lane >> 3);
    float* wp = mat.w + (int64_t)r0 * mat.cols + c4;
    float4 f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + 4 * i < mat.rows && c4 < mat.cols)
        f[i] = *reinterpret_cast<const float4*>(wp + (int64_t)4 * i * mat.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + 4 * i < mat.rows && c4 < mat.cols) {
        const float4 u = *reinterpret_cast<const float4*>(piece(4 * i + (lane >> 3), lane & 7));
        f[i].x = __fmaf_rn(-to_w, u.x, __fmul_rn(f[i].x, decay));
        f[i].y = __fmaf_rn(-to_w, u.y, __fmul_rn(f[i].y, decay));
        f[i].z = __fmaf_rn(-to_w, u.z, __fmul_rn(f[i].z, decay));
        f[i].w = __fmaf_rn(-to_w, u.w, __fmul_rn(f[i].w, decay));
        *reinterpret_cast<float4*>(wp + (int64_t)4 * i * mat.cols) = f[i];
        if (mat.wb)
          *reinterpret_cast<uint2*>(mat.wb + (int64_t)(r0 + 4 * i) * mat.cols + c4) =
              make_uint2(cvt_f32x2_bf16x2(f[i].y, f[i].x), cvt_f32x2_bf16x2(f[i].w, f[i].z));
      }
    }
  } else if (col + lane < mat.cols) {  // any address: a row's columns by lanes
    const int rows = min(32, mat.rows - row0);
    for (int r = 0; r < rows; ++r) {
      const int64_t at = (int64_t)(row0 + r) * mat.cols + col + lane;
      const float f = __fmaf_rn(-to_w, piece(r, lane >> 2)[lane & 3], __fmul_rn(mat.w[at], decay));
      mat.w[at] = f;
      if (mat.wb) mat.wb[at] = Elem<GS_BF16>::put(f);
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(kMThreads, 1) __cluster_dims__(2, 1, 1)
    muon_products_kernel(MuonTable t, MuonArgs a) {
  using S = Mu<BN>;
  constexpr int kMStages = S::kStages, kMStage = S::kStage;
  if (*a.found_inf) return;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (tc_smem(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;
  uint8_t* pieces = stages + kMStages * kMStage;  // two per storing warp
  int* key_space = reinterpret_cast<int*>(pieces + 8 * 2 * kMPiece);
  uint64_t* full = reinterpret_cast<uint64_t*>(key_space + 2 * kMKeys);
  uint64_t* empty = full + kMStages;
  uint64_t* tfull = empty + kMStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* loaded = drain + 1;                   // a storing warp's pieces of old
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(loaded + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int* keys = t.n <= kMKeys ? key_space : nullptr;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int first = (int)blockIdx.x / 2, step = (int)gridDim.x / 2;
  const int tiles = a.steps * (2 * t.sym_tiles + t.app_tiles);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMStages; ++s) {
      tc_bar_init(&full[s], 1);
      tc_bar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc_bar_init(&tfull[b], 1);
      tc_bar_init(&tempty[b], 16);
    }
    tc_bar_init(drain, 1);
    for (int w = 0; w < 8; ++w) tc_bar_init(&loaded[w], 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tc_alloc<2>(tmem_slot, 2 * BN);
  if (keys && threadIdx.x >= 64 && threadIdx.x - 64 < t.n) {
    key_space[threadIdx.x - 64] = t.mats[threadIdx.x - 64].first_sym;
    key_space[kMKeys + threadIdx.x - 64] = t.mats[threadIdx.x - 64].first_app;
  }
  // the tensor maps lie in global memory: once per CTA before their use
  for (int i = threadIdx.x; i < 2 * kMuonMaps * t.n; i += kMThreads) map_fence(t.maps + i);
  tc_before();
  __syncthreads();
  cluster_barrier();
  tc_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {  // loads
    uint32_t s = 0, ph = 0, used = 0;
    bool go = !a.stall;
    for (int tile = first; go && tile < tiles; tile += step) {
      const Product p = product<BN>(t, keys, tile, a.steps);
      const CUtensorMap* maps = t.maps + 2 * kMuonMaps * p.id;
      if (!wait_done(t.done + p.id, p.need, abort_flag, a.status)) break;
      // what other CTAs stored is read by TMA from here on
      asm volatile("fence.proxy.async;" ::: "memory");
      const CUtensorMap *ma = maps + p.map_a, *mb = maps + p.map_b;
      const int m0 = p.m0 + 128 * (int)rank, n0 = p.n0 + BN / 2 * (int)rank;
      const int parts = (p.K + 63) / 64, all = p.lo_in ? 2 * parts : parts;
      for (int i = 0; i < all; ++i) {
        if (!tc_wait_warp(&empty[s], ph ^ 1u, abort_flag, a.status)) {
          go = false;
          break;
        }
        if (i == parts) ma = maps + p.map_a_lo, mb = maps + p.map_b_lo;
        const int k = 64 * (i < parts ? i : i - parts);
        uint8_t* st = stages + s * kMStage;
        if (tc_elect()) {
          const uint32_t bar = tc_leader<2>(&full[s]);
          if (rank == 0) tc_expect(&full[s], 2 * kMStage);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tc_load2<2>(ma, bar, st + h * kMBox, p.ta ? m0 + 64 * h : k, p.ta ? k : m0 + 64 * h);
#pragma unroll
          for (int h = 0; h < S::kBBoxes; ++h) {
            tc_load2<2>(mb, bar, st + (2 + h) * kMBox, p.tb ? n0 + 64 * h : k, p.tb ? k : n0 + 64 * h);
          }
        }
        __syncwarp();
        used |= 1u << s;
        if (++s == kMStages) s = 0, ph ^= 1u;
      }
    }
    // the MMAs that read the last stages, and with them the loads, are done
    for (int j = 0; j < kMStages; ++j) {
      if (s == 0) s = kMStages, ph ^= 1u;
      --s;
      if (used >> s & 1u) tc_drain(&empty[s], ph);
    }
  } else if (warp == 1 && rank == 0) {  // MMA
    uint32_t s = 0, ph = 0, b = 0, tph = 0;
    bool go = true;
    for (int tile = first; go && tile < tiles; tile += step) {
      const Product p = product<BN>(t, keys, tile, a.steps);
      if (!tc_wait_warp(&tempty[b], tph ^ 1u, abort_flag, a.status)) break;
      tc_after();
      const uint32_t idesc = idesc16(BN, p.ta, p.tb);
      const int all = (p.lo_in ? 2 : 1) * ((p.K + 63) / 64);
      for (int i = 0; i < all; ++i) {
        if (!tc_wait_warp(&full[s], ph, abort_flag, a.status)) {
          go = false;
          break;
        }
        tc_after();
        const uint32_t a0 = tc_smem(stages) + s * kMStage, b0 = a0 + 2 * kMBox;
        if (tc_elect()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma16(tmem + b * BN, desc16(a0, kk, p.ta), desc16(b0, kk, p.tb), idesc,
                  i > 0 || kk > 0 ? 1u : 0u);
          tc_commit<2>(&empty[s]);
          if (i == all - 1) tc_commit<2>(&tfull[b]);
        }
        __syncwarp();
        if (++s == kMStages) s = 0, ph ^= 1u;
      }
      b ^= 1u;
      if (b == 0) tph ^= 1u;
    }
    if (tc_elect()) tc_commit<2>(drain);
    __syncwarp();
    tc_drain(drain, 0);
  } else if (warp >= 4) {  // store
    const int q = warp & 3, h = (warp - 4) >> 2;
    uint8_t* const mine = pieces + (warp - 4) * 2 * kMPiece;
    uint64_t* const bar = &loaded[warp - 4];
    uint32_t b = 0, tph = 0, lph = 0;
    for (int tile = first; tile < tiles; tile += step) {
      const Product p = product<BN>(t, keys, tile, a.steps);
      const MuonMat& mat = t.mats[p.id];
      // result = alpha acc + beta old, old in the result's shape
      float alpha, beta = 0.0f, one = 0.0f, decay = 1.0f, to_w = 0.0f;
      int map_old = 0, map_out = 0;
      if (p.kind == kGram) {
        alpha = __fdiv_rn(mat.sa, __fmul_rn(mat.sx, mat.sx));
        map_out = 2;
      } else if (p.kind == kPoly) {
        alpha = __fdiv_rn(0.25f * kNsC, mat.sa);  // gram gram is by sa^2, poly by sa / 4
        beta = 0.25f * kNsB;
        one = __fmul_rn(0.25f * (kNsA - 1.0f), mat.sa);
        map_old = 2;
        map_out = 3;
      } else {
        alpha = __fdiv_rn(4.0f, mat.sa);
        beta = 1.0f;
        map_old = p.turn;
        map_out = p.turn ^ 1;
        if (p.kind == kLast) {
          const float big = (float)max(mat.rows, mat.cols);
          const float scale = a.scale_mode == GS_MUON_SCALE_RMS
                                  ? 0.2f * sqrtf(big)
                                  : sqrtf(fmaxf(1.0f, __fdiv_rn((float)mat.rows, (float)mat.cols)));
          decay = __fsub_rn(1.0f, __fmul_rn(a.lr, a.weight_decay));
          to_w = __fdiv_rn(__fmul_rn(a.lr, scale), mat.sx);
        }
      }
      const int row0 = p.m0 + 128 * (int)rank + 32 * q, row = row0 + lane, col0 = p.n0 + BN / 2 * h;
      const CUtensorMap* maps = t.maps + 2 * kMuonMaps * p.id + kMuonMaps;  // boxes of 32 rows
      const bool some = row0 < p.M && col0 < p.N;
      // what the sum is added to, of 64 columns and both parts (one lane)
      const auto old_pair = [&](int g) {
        tc_expect(bar, 2 * kMPiece);
        tc_load2<1>(maps + map_old, tc_smem(bar), mine, col0 + 64 * g, row0);
        tc_load2<1>(maps + map_old + 4, tc_smem(bar), mine + kMPiece, col0 + 64 * g, row0);
      };
      if (p.kind != kGram && some) {
        if (!wait_done(t.done + p.id, p.need, abort_flag, a.status)) break;
        // what other CTAs stored is read by TMA; this warp's own uses of its
        // pieces are over
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncwarp();
        if (tc_elect()) {
          if (p.lo_in) {
            old_pair(0);
          } else {
            tc_expect(bar, S::kGroups * kMPiece);
#pragma unroll
            for (int i = 0; i < S::kGroups; ++i)
              tc_load2<1>(maps + map_old, tc_smem(bar), mine + i * kMPiece, col0 + 64 * i, row0);
          }
        }
        __syncwarp();
      }
      bool got = tc_wait(&tfull[b], tph, abort_flag, a.status);
      if (p.kind != kGram && some) {
        // (also where the tile is given up: the loads have to land)
        tc_drain(bar, lph);
        lph ^= 1u;
      }
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      tc_after();
      const bool mirror = p.mirror && row < p.M;
      uint4 later[4] = {};
#pragma unroll 1
      for (int c = 0; c < BN / 64; ++c) {
        const int col = col0 + 32 * c;
        uint8_t* const buf = mine + (p.lo_in ? 0 : c >> 1) * kMPiece;
        uint8_t* const buf_lo = mine + kMPiece;
        float o[32];
        uint32_t* const v = reinterpret_cast<uint32_t*>(o);
        tc_ld32(tmem + ((uint32_t)(32 * q) << 16) + b * BN + BN / 2 * h + 32 * c, v);
        tc_wait_ld<32>(v);
        if (c == BN / 64 - 1) {
          tc_before();
          __syncwarp();
          if (lane == 0) tc_arrive_at(&tempty[b], 0);
        }
        // (the second half of a piece is stored with the first)
        if (row0 >= p.M || col0 + 64 * (c >> 1) >= p.N) continue;
        if (p.lo_in && c > 0 && (c & 1) == 0) {  // the next 64 columns, where the last are on their way
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          asm volatile("fence.proxy.async;" ::: "memory");
          __syncwarp();
          if (tc_elect()) old_pair(c >> 1);
          __syncwarp();
          tc_drain(bar, lph);
          lph ^= 1u;
        }
        // 16 bytes j of row r lie at j ^ (r % 8)
        const auto place = [&](int j) {
          return reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4));
        };
        const auto place_lo = [&](int j) {
          return reinterpret_cast<uint4*>(buf_lo + lane * 128 + ((j ^ (lane & 7)) << 4));
        };
        uint4 was[4];  // both halves are read before the piece is written
#pragma unroll
        for (int j = 0; j < 4; ++j) was[j] = later[j];
        if (p.kind != kGram && (c & 1) == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) was[j] = *place(j), later[j] = *place(4 + j);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __fmul_rn(o[j], alpha);
        if (p.lo_in) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 w = *place_lo(4 * (c & 1) + j);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[8 * j + 2 * e] = __fadd_rn(lo_f16(ww[e]), o[8 * j + 2 * e]);
              o[8 * j + 2 * e + 1] = __fadd_rn(hi_f16(ww[e]), o[8 * j + 2 * e + 1]);
            }
          }
        }
        if (p.kind != kGram) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t ww[4] = {was[j].x, was[j].y, was[j].z, was[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[8 * j + 2 * e] = __fmaf_rn(beta, lo_f16(ww[e]), o[8 * j + 2 * e]);
              o[8 * j + 2 * e + 1] = __fmaf_rn(beta, hi_f16(ww[e]), o[8 * j + 2 * e + 1]);
            }
          }
          if (p.kind == kPoly && row0 < col + 32 && col < row0 + 32) {  // the diagonal is in it
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col + j == row) o[j] = __fadd_rn(o[j], one);
          }
        }
        if (p.kind != kLast) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = cvt_f32x2_f16x2(o[8 * j + 2 * e + 1], o[8 * j + 2 * e]);
            *place(4 * (c & 1) + j) = make_uint4(w[0], w[1], w[2], w[3]);
            if (p.lo_out) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = cvt_f32x2_f16x2(__fsub_rn(o[8 * j + 2 * e + 1], hi_f16(w[e])),
                                       __fsub_rn(o[8 * j + 2 * e], lo_f16(w[e])));
              *place_lo(4 * (c & 1) + j) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (c & 1) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (tc_elect()) {  // clipped at the matrix's edges
              tc_store2(maps + map_out, buf, col - 32, row0);
              if (p.lo_out) tc_store2(maps + map_out + 4, buf_lo, col - 32, row0);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            __syncwarp();
          }
          if (mirror) {
            uint16_t* const out = (p.kind == kGram ? mat.gram : mat.poly) + row;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col + j < p.N) out[(int64_t)(col + j) * mat.lds] = Elem<GS_F16>::put(o[j]);
          }
        } else {
          update_weights(mat, reinterpret_cast<float*>(buf), o, row0, col, decay, to_w);
        }
      }
      // this warp's part is stored: for loads of either kind by other CTAs.  (Each
      // warp counts for itself: one that gave up holds no other.)
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      __threadfence();
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      if (lane == 0)
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(t.done + p.id) : "memory");
      b ^= 1u;
      if (b == 0) tph ^= 1u;
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  cluster_barrier();
  tc_after();
  if (warp == 1) tc_dealloc<2>(tmem, 2 * BN);
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) ==
            cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool muon_encode(CUtensorMap* map, uint16_t* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  if (!encode_fn()) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
static cudaError_t launch_products(const MuonTable& t, const MuonArgs& a, cudaStream_t st) {
  auto k = muon_products_kernel<BN>;
  int occ = 0, pairs = 0;  // also raises the shared-memory limit in this context
  cudaError_t e = kernel_blocks_per_sm((const void*)k, kMThreads, Mu<BN>::kSmem, &occ);
  if (e == cudaSuccess) e = kernel_clusters((const void*)k, kMThreads, Mu<BN>::kSmem, 2, &pairs);
  if (e != cudaSuccess) return e;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)std::min(std::max(t.sym_tiles, t.app_tiles), pairs));
  cfg.blockDim = dim3(kMThreads);
  cfg.dynamicSmemBytes = Mu<BN>::kSmem;
  cfg.stream = st;
  // CTAs wait for one another's tiles: all of them have to be resident
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeCooperative;
  at.val.cooperative = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, t, a);
}

template <int DT>
static cudaError_t muon_dt(const MuonTable& t, const MuonArgs& a, cudaStream_t st) {
  const unsigned wave = (unsigned)std::min<int64_t>(t.chunks, (int64_t)sm_count() * 4);
  muon_momentum_kernel<DT><<<wave, kMEThreads, 0, st>>>(t, a);
  const unsigned grid = (unsigned)std::min<int64_t>(t.chunks, (int64_t)sm_count() * 32);
  muon_scale_kernel<DT><<<grid, kMEThreads, 0, st>>>(t, a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return t.tile_n == kMuonTile ? launch_products<kMuonTile>(t, a, st)
                               : launch_products<kMuonTile / 2>(t, a, st);
}

cudaError_t launch_master_update_muon(const MuonTable& t, const MuonArgs& a, cudaStream_t st) {
  if (t.n == 0) return cudaSuccess;
  if (a.grad_dtype == GS_F32) return muon_dt<GS_F32>(t, a, st);
  if (a.grad_dtype == GS_F16) return muon_dt<GS_F16>(t, a, st);
  return muon_dt<GS_BF16>(t, a, st);
}

}  // namespace gs

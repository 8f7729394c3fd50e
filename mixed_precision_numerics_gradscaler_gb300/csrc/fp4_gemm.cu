// fp4_gemm.cu -- products of microscaled 4-bit tensors on the tensor cores:
//   D[m][n] = ta tb sum_k A[m][k] sa[m][k / block] B[n][k] sb[n][k / block],
// A [M, K] and B [N, K] e2m1 codes, block scales E8M0 per 32 (MXFP4) or E4M3 per
// 16 (NVFP4) in tiles of 128 rows x 4 scales, D fp32 or bf16.
//
// tcgen05.mma takes 64 elements of K with their scales from tensor memory:
// products and scales are exact, sums fp32.  Nothing is promoted between, so a
// tile's whole sum stays in tensor memory.
//
// Persistent clusters of CG CTAs (a pair shares one MMA of 256 rows: each CTA
// loads half of either operand, which halves what shared memory has to take and
// give per operation) walk tiles of 128 CG x BN of D.  Roles of a CTA:
//   warp 0             TMA loads, 256 elements of K a stage: codes in the
//                      128-byte swizzle, scale tiles as they lie;
//   warp 1 (of the leading CTA)  copies a stage's scales to tensor memory and
//                      issues its four MMAs, in order in one pipe;
//   warps 4-11         read the sum from tensor memory into registers, hand the
//                      accumulator back at once and store while the next tile's
//                      MMAs run.  A sum of 256 columns and the scales leave no
//                      room for a second one.
// Few rows of A (TRANS): the operands change places, the weight's rows become
// the 128 rows of a tile and the few rows its BN columns, and a tile is stored
// transposed, 32 lanes to 32 neighbours of a row of D.
// 16384 x 28672 x 8192, NVFP4, bf16 out: 1.26 to 1.31 ms, 5.9 to 6.1 PFLOP/s under
// the power cap (without the copies of scales, twelve a stage in the MMAs' pipe,
// 1.14 ms; two sets of columns for them change nothing).  One row by 28672 x 8192:
// 29 us, 26 from a graph (30 with cold caches), 19.8 at the copy rate.
// Every wait is bounded and reports GS_ERR_TIMEOUT.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "gs_fp4.h"
#include "gs_internal.h"
#include "gs_tcgen05.cuh"

namespace gs {

constexpr int kQThreads = 384;      // warps 0-3: loads, MMA, two idle; 4-11 store
constexpr int kQRow = 128;          // bytes of a row of a stage: 256 elements
constexpr int kQK = 256;

// One configuration's sizes.
// SLOTS: sums of other CTAs of a cluster that the leading one takes in.
template <int CG, int BN, int FMT, int SLOTS>
struct Q4 {
  static constexpr int kBRows = BN / CG;                   // of B that a CTA loads
  static constexpr int kTiles = FMT == GS_NVFP4 ? 4 : 2;   // scale tiles per stage and 128 rows
  static constexpr int kBTiles = BN <= 128 ? 1 : BN / 128; // of 128 rows of B's scales
  static constexpr int kA = 128 * kQRow, kB = kBRows * kQRow;
  static constexpr int kSA = kTiles * 512, kSB = kBTiles * kTiles * 512;
  static constexpr int kStage = ((kA + kB + kSA + kSB + 1023) / 1024) * 1024;
  static constexpr int kBytes = kA + kB + kSA + kSB;       // a CTA's loads per stage
  static constexpr int kSlot = 128 * BN * 4;
  // store staging of 8 warps, or the other CTAs' sums
  static constexpr int kOut = SLOTS ? SLOTS * kSlot : 8 * 32 * 128;
  static constexpr int kMost = (232448 - 1024 - 512 - kOut) / kStage;
  static constexpr int kStages = kMost > 8 ? 8 : kMost;
  static constexpr int kAccs = BN <= 128 ? 2 : 1;
  static constexpr int kSfCol = kAccs * BN;                // columns of the scales
  static constexpr int kSbCol = kSfCol + 4 * kTiles;
  static constexpr int kCols = kSbCol + 4 * kTiles * kBTiles;
  static constexpr int kAlloc = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kSmem = kStages * kStage + kOut + 1024 + 512;
  static_assert(kCols <= 512 && kStages >= 3 && kSmem <= 232448, "sizes");
};

struct Gemm4Args {
  const float *ta, *tb;   // null: 1
  int64_t M, N, K;        // of the tile space (operands changed over for TRANS)
  void* d;
  int64_t ldd;
  int32_t* status;
  int group;              // tile rows of a raster group
  int split;              // CTAs that share a tile's sum (TRANS)
  int stall;
};

// Instruction descriptor: e2m1 operands with the sum dimension along their rows,
// E4M3 or E8M0 scales; sf: which scales of a 32-bit word an MMA takes.
template <int FMT>
__device__ __forceinline__ uint32_t idesc4(int m, int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         (FMT == GS_MXFP4 ? 1u << 23 : 0u) | ((uint32_t)(m >> 4) << 24) | (sf << 29);
}

template <int CG, int FMT>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                     uint32_t sb, uint32_t accumulate) {
#define GS_MMA4(cg, kind)                                                                       \
  asm volatile(                                                                                 \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                         \
      "tcgen05.mma.cta_group::" cg "." kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),  \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                             \
      : "memory")
  if constexpr (FMT == GS_NVFP4) {
    if constexpr (CG == 2) GS_MMA4("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else GS_MMA4("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if constexpr (CG == 2) GS_MMA4("2", "kind::mxf4.block_scale.scale_vec::2X");
    else GS_MMA4("1", "kind::mxf4.block_scale.scale_vec::2X");
  }
#undef GS_MMA4
}
// 32 rows of 16 bytes of shared memory -> 4 columns of tensor memory, the same
// in each of its four lane quarters (in both CTAs of a pair).
template <int CG>
__device__ __forceinline__ void cp_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// TRANS: 0, or the operands have changed places and TRANS + 1 CTAs of a cluster at
// most share a tile's sum, split along K: CTA r takes its part of the stages, CTAs
// 1 .. split - 1 write their fp32 sums to the leading CTA's shared memory, which
// adds them in their order.  There is one tile of columns then (N <= BN): one further
// on would begin inside its 128 rows' scales, and an MMA takes scales from multiples
// of four columns of tensor memory alone.
template <int CG, int BN, int FMT, int OUT, int TRANS, bool TMA_STORE>
__global__ void __launch_bounds__(kQThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
                    const __grid_constant__ CUtensorMap map_d, Gemm4Args a) {
  using S = Q4<CG, BN, FMT, TRANS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (tc_smem(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;  // the same offset in both CTAs of a pair
  uint8_t* out_stage = stages + S::kStages * S::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + S::kOut);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* joined = drain + 1;    // the other CTAs' sums are in the leading CTA
  uint64_t* taken = joined + 1;    // ... and this CTA's has been read there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(taken + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const uint32_t part = TRANS ? cluster_rank() : 0;
  const int parts = TRANS ? a.split : CG;             // CTAs of a cluster
  const int all_kb = (int)((a.K + kQK - 1) / kQK);
  // this CTA's stages (split <= all_kb: none has no stage)
  const int kb0 = TRANS ? (int)((int64_t)all_kb * part / a.split) : 0;
  const int kb1 = TRANS ? (int)((int64_t)all_kb * (part + 1) / a.split) : all_kb;
  const int tiles_m = (int)((a.M + 128 * CG - 1) / (128 * CG)), tiles_n = (int)((a.N + BN - 1) / BN);
  const int n_tiles = tiles_m * tiles_n;
  const int first = (int)blockIdx.x / parts, step = (int)gridDim.x / parts;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      tc_bar_init(&full[s], 1);
      tc_bar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc_bar_init(&tfull[b], 1);
      tc_bar_init(&tempty[b], 8 * CG);
    }
    tc_bar_init(drain, 1);
    tc_bar_init(joined, TRANS ? 4 * (a.split > 1 ? a.split - 1 : 1) : 1);
    tc_bar_init(taken, 4);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tc_alloc<CG>(tmem_slot, S::kAlloc);
  tc_before();
  __syncthreads();
  if constexpr (CG == 2 || TRANS) cluster_barrier();  // the cluster's barriers are there
  tc_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {  // loads
    uint32_t s = 0, ph = 0, used = 0;
    bool go = !a.stall;
    for (int t = first; go && t < n_tiles; t += step) {
      int mt, nt;
      tc_tile(t, a.group, tiles_m, tiles_n, mt, nt);
      const int row_a = (mt * CG + (int)rank) * 128, row_b = nt * BN + (int)rank * S::kBRows;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!tc_wait_warp(&empty[s], ph ^ 1u, abort_flag, a.status)) {
          go = false;
          break;
        }
        uint8_t* st = stages + s * S::kStage;
        if (tc_elect()) {
          const uint32_t bar = tc_leader<CG>(&full[s]);
          if (rank == 0) tc_expect(&full[s], CG * S::kBytes);
          tc_load2<CG>(&map_a, bar, st, kb * kQRow, row_a);
          tc_load2<CG>(&map_b, bar, st + S::kA, kb * kQRow, row_b);
          tc_load3<CG>(&map_sa, bar, st + S::kA + S::kB, 0, kb * S::kTiles, row_a / 128);
          tc_load3<CG>(&map_sb, bar, st + S::kA + S::kB + S::kSA, 0, kb * S::kTiles, nt * BN / 128);
        }
        __syncwarp();
        used |= 1u << s;
        if (++s == S::kStages) s = 0, ph ^= 1u;
      }
    }
    // the MMAs that read the last stages, and with them the loads, are done
    for (int j = 0; j < S::kStages; ++j) {
      if (s == 0) s = S::kStages, ph ^= 1u;
      --s;
      if (used >> s & 1u) tc_drain(&empty[s], ph);
    }
  } else if (warp == 1 && rank == 0) {  // MMA
    uint32_t s = 0, ph = 0, b = 0, tph = 0;
    bool go = true;
    for (int t = first; go && t < n_tiles; t += step) {
      int mt, nt;
      tc_tile(t, a.group, tiles_m, tiles_n, mt, nt);
      if (!tc_wait_warp(&tempty[b], tph ^ 1u, abort_flag, a.status)) break;
      tc_after();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!tc_wait_warp(&full[s], ph, abort_flag, a.status)) {
          go = false;
          break;
        }
        tc_after();
        const uint32_t a0 = tc_smem(stages) + s * S::kStage, b0 = a0 + S::kA;
        const uint32_t sa0 = b0 + S::kB, sb0 = sa0 + S::kSA;
        const int steps = (int)min((int64_t)4, (a.K - (int64_t)kb * kQK + 63) / 64);
        if (tc_elect()) {
#pragma unroll
          for (int j = 0; j < S::kTiles; ++j) {
            cp_scales<CG>(tmem + S::kSfCol + 4 * j, tc_desc_scales(sa0 + 512 * j));
#pragma unroll
            for (int r = 0; r < S::kBTiles; ++r)
              cp_scales<CG>(tmem + S::kSbCol + 4 * (j * S::kBTiles + r),
                            tc_desc_scales(sb0 + 512 * (r * S::kTiles + j)));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk < steps) {
              // NVFP4: a scale tile per 64 elements; MXFP4: one per 128, in halves
              const int j = FMT == GS_NVFP4 ? kk : kk >> 1;
              const uint32_t sf = FMT == GS_NVFP4 ? 0u : 2u * (kk & 1);
              mma4<CG, FMT>(tmem + b * BN, tc_desc_k(a0 + 32 * kk), tc_desc_k(b0 + 32 * kk),
                            idesc4<FMT>(128 * CG, BN, sf), tmem + S::kSfCol + 4 * j,
                            tmem + S::kSbCol + 4 * j * S::kBTiles, kb > kb0 || kk > 0 ? 1u : 0u);
            }
          }
          tc_commit<CG>(&empty[s]);
          if (kb == kb1 - 1) tc_commit<CG>(&tfull[b]);
        }
        __syncwarp();
        if (++s == S::kStages) s = 0, ph ^= 1u;
      }
      if (++b == S::kAccs) b = 0, tph ^= 1u;
    }
    if (tc_elect()) tc_commit<CG>(drain);
    __syncwarp();
    tc_drain(drain, 0);
  } else if (warp >= 4) {  // store
    const int q = warp & 3;            // the lanes of tensor memory this warp reads
    const int h = (warp - 4) >> 2;     // which half of the columns
    constexpr int kCols = BN >= 64 ? BN / 2 : BN;  // per warp (the first four alone below 64)
    const bool mine = BN >= 64 || h == 0;
    uint8_t* const buf = out_stage + (warp - 4) * 32 * 128;
    float alpha = 1.0f, beta = 1.0f;
    if (a.ta) alpha = __fmul_rn(*a.ta, *a.tb);
    // A product of the two that fp32 does not hold is applied a factor at a time: the
    // larger one first where it is small, the smaller one first where it is large, so
    // that nothing on the way leaves fp32 but where the result does (a sum is 0 or at
    // least 2^-20).
    if (a.ta && !(fabsf(alpha) >= 0x1p-126f && fabsf(alpha) < INFINITY)) {
      const float x = *a.ta, y = *a.tb;
      const bool x_first = fabsf(alpha) < 1.0f ? fabsf(x) > fabsf(y) : fabsf(x) < fabsf(y);
      alpha = x_first ? x : y;
      beta = x_first ? y : x;
    }
    uint32_t n = 0;
    for (int t = first; t < n_tiles; t += step, ++n) {
      int mt, nt;
      tc_tile(t, a.group, tiles_m, tiles_n, mt, nt);
      const uint32_t b = n % S::kAccs, tph = (n / S::kAccs) & 1u;
      const bool got = tc_wait(&tfull[b], tph, abort_flag, a.status);
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      tc_after();
      uint32_t v[kCols];
      if (mine) {
#pragma unroll
        for (int c = 0; c < kCols; c += 32)
          tc_ld32(tmem + ((uint32_t)(32 * q) << 16) + b * BN + h * kCols + c, v + c);
        tc_wait_ld<kCols>(v);
      }
      tc_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) tc_arrive_at(&tempty[b], 0);
        else tc_arrive(&tempty[b]);
      }
      if (!mine) continue;
      const int64_t row = ((int64_t)mt * CG + rank) * 128 + 32 * q;  // this warp's first
      const int64_t col = (int64_t)nt * BN + h * kCols;
      if constexpr (TRANS) {
        // every CTA of the cluster comes to the same tiles with its part of the sum
        if (a.split > 1) {
          static_assert(BN == 32, "a slot is four warps' 32 columns");
          float4* const slot = reinterpret_cast<float4*>(out_stage) + q * 256 + lane;
          if (part > 0) {
            // (n-th tile of this cluster: its sum before has been read)
            if (!__all_sync(0xFFFFFFFFu, tc_wait_cluster(taken, (n & 1u) ^ 1u, abort_flag, a.status))) break;
            const uint32_t to = remote(slot + (part - 1) * (S::kSlot / 16), 0);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + 512 * c), "r"(v[4 * c]),
                           "r"(v[4 * c + 1]), "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                           : "memory");
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc_arrive_at(joined, 0);
            continue;
          }
          if (!__all_sync(0xFFFFFFFFu, tc_wait_cluster(joined, n & 1u, abort_flag, a.status))) break;
          for (int p = 1; p < a.split; ++p) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 f = slot[(p - 1) * (S::kSlot / 16) + 32 * c];
              v[4 * c] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * c]), f.x));
              v[4 * c + 1] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * c + 1]), f.y));
              v[4 * c + 2] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * c + 2]), f.z));
              v[4 * c + 3] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * c + 3]), f.w));
            }
          }
          __syncwarp();
          if (lane > 0 && lane < a.split) tc_arrive_at(taken, lane);
        }
      }
      if (row >= a.M || col >= a.N) continue;
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[c] = __float_as_uint(__fmul_rn(__uint_as_float(v[c]), alpha));
      if (beta != 1.0f) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) v[c] = __float_as_uint(__fmul_rn(__uint_as_float(v[c]), beta));
      }
      if constexpr (TRANS) {
        const int64_t to = col * a.ldd + row + lane;
        if (row + lane < a.M) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (col + c < a.N) {
              if constexpr (OUT == GS_F32) static_cast<float*>(a.d)[to + c * a.ldd] = __uint_as_float(v[c]);
              else static_cast<uint16_t*>(a.d)[to + c * a.ldd] = Elem<GS_BF16>::put(__uint_as_float(v[c]));
            }
        }
      } else {
        // 32 columns at any address: through shared memory, rows by turns
        const auto by_rows = [&](int c) {
          float* const f = reinterpret_cast<float*>(buf);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 32; ++j) f[lane * 32 + ((j + lane) & 31)] = __uint_as_float(v[c + j]);
          __syncwarp();
          const int rows = (int)min((int64_t)32, a.M - row);
          if (col + c + lane < a.N) {
            for (int r = 0; r < rows; ++r) {
              const float o = f[r * 32 + ((lane + r) & 31)];
              const int64_t to = (row + r) * a.ldd + col + c + lane;
              if constexpr (OUT == GS_F32) static_cast<float*>(a.d)[to] = o;
              else static_cast<uint16_t*>(a.d)[to] = Elem<GS_BF16>::put(o);
            }
          }
        };
        if constexpr (TMA_STORE) {
          constexpr int kChunk = OUT == GS_F32 ? 32 : 64;  // columns of 128 bytes
          // (a TMA store clips a row's end to 16 bytes)
          const bool whole_end = a.N % (OUT == GS_F32 ? 4 : 8) == 0;
#pragma unroll
          for (int c = 0; c < kCols; c += kChunk) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
            if (!whole_end && col + c + kChunk > a.N) {
#pragma unroll
              for (int i = 0; i < kChunk; i += 32) by_rows(c + i);
              continue;
            }
#pragma unroll
            for (int p = 0; p < 8; ++p) {  // 16-byte piece p of row r lies at p ^ (r % 8)
              uint4 w;
              if constexpr (OUT == GS_F32) {
                w = make_uint4(v[c + 4 * p], v[c + 4 * p + 1], v[c + 4 * p + 2], v[c + 4 * p + 3]);
              } else {
                const float* f = reinterpret_cast<const float*>(v) + c + 8 * p;
                w = make_uint4(cvt_f32x2_bf16x2(f[1], f[0]), cvt_f32x2_bf16x2(f[3], f[2]),
                               cvt_f32x2_bf16x2(f[5], f[4]), cvt_f32x2_bf16x2(f[7], f[6]));
              }
              *reinterpret_cast<uint4*>(buf + lane * 128 + ((p ^ (lane & 7)) << 4)) = w;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0 && col + c < a.N) {
              tc_store2(&map_d, buf, (int32_t)(col + c), (int32_t)row);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 32) by_rows(c);
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  if constexpr (CG == 2 || TRANS) cluster_barrier();  // nothing of the cluster is under way
  tc_after();
  if (warp == 1) tc_dealloc<CG>(tmem, S::kAlloc);
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

// rows x K codes, boxes of 128 bytes x box_rows.
static bool encode_codes(CUtensorMap* m, const uint8_t* q, int64_t rows, int64_t K, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t box[2] = {kQRow, box_rows}, one[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Scale tiles [row tile][scale tile][128 words]: boxes of `tiles` scale tiles of
// `row_tiles` row tiles; zeros past the edges.
static bool encode_scales(CUtensorMap* m, const uint8_t* s, int64_t rows, int64_t K, int fmt,
                          uint32_t tiles, uint32_t row_tiles) {
  const int64_t kt = div_up(K, fmt == GS_NVFP4 ? 64 : 128), rt = div_up(rows, 128);
  const cuuint64_t dims[3] = {128, (cuuint64_t)kt, (cuuint64_t)rt};
  const cuuint64_t strides[2] = {512, (cuuint64_t)kt * 512};
  const cuuint32_t box[3] = {128, tiles, row_tiles}, one[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(s), dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
  const uint8_t *q, *s;
  int64_t rows;
};

template <int CG, int BN, int FMT, int OUT, int TRANS, bool TMA_STORE>
static cudaError_t gemm4_run(const Operand& x, const Operand& y, Gemm4Args a, cudaStream_t st) {
  using S = Q4<CG, BN, FMT, TRANS>;
  auto k = gemm_fp4_kernel<CG, BN, FMT, OUT, TRANS, TMA_STORE>;
  int occ = 0;  // also raises the shared-memory limit in this context
  cudaError_t e = kernel_blocks_per_sm((const void*)k, kQThreads, S::kSmem, &occ);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  CUtensorMap ma, mb, msa, msb, md;
  memset(&md, 0, sizeof(md));
  if (!encode_codes(&ma, x.q, x.rows, a.K, 128) || !encode_codes(&mb, y.q, y.rows, a.K, S::kBRows) ||
      !encode_scales(&msa, x.s, x.rows, a.K, FMT, S::kTiles, 1) ||
      !encode_scales(&msb, y.s, y.rows, a.K, FMT, S::kTiles, S::kBTiles))
    return cudaErrorInvalidValue;
  if (TMA_STORE) {
    const size_t esz = OUT == GS_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M};
    const cuuint64_t strides[1] = {(cuuint64_t)a.ldd * esz};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / esz), 32}, one[2] = {1, 1};
    if (encode_fn()(&md, OUT == GS_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    2, a.d, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int64_t tiles = div_up(a.M, 128 * CG) * div_up(a.N, BN);
  const int per = TRANS ? a.split : CG;
  const int64_t clusters = std::min<int64_t>(tiles, sm_count() / per);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * per));
  cfg.blockDim = dim3(kQThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)per;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = per > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, ma, mb, msa, msb, md, a);
}

// Time of a shape's tiles on all SMs, in units of a stage of the large tile
// (0.4 us): rounds of tiles times stages and the store.  128 x 128 and 256 x 256, bf16:
// 33 x 4096 x 4096 11.0 and 13.1 us, 128 x 4096 x 4096 12.1 and 14.9,
// 1111 x 4099 x 4128 21.4 and 26.5, 1024 x 4096 x 4096 18.9 and 14.9,
// 512 x 8192 x 8192 29.6 and 20.8, 300 x 28672 x 8192 63.8 and 47.7,
// 4096 x 4096 x 14336 145 and 91; the faster one is taken in each.
static double rounds(int64_t M, int64_t N, int64_t K, int tm, int tn, int ctas, double stage, double store) {
  const int64_t tiles = div_up(M, tm) * div_up(N, tn), slots = sm_count() / ctas;
  return (double)div_up(tiles, slots) * ((double)div_up(K, kQK) * stage + store);
}

template <int FMT, int OUT>
static cudaError_t gemm4_pick(const Operand& x, const Operand& y, Gemm4Args a, bool tma, cudaStream_t st) {
  // few rows of A: they become a tile's columns, one tile of 32.  One to 32 rows by
  // 4096 x 14336 15 us, 25 in tiles of 128 rows; by 28672 x 8192 30, 33 to 51
  if (a.M <= 32) {
    std::swap(a.M, a.N);
    // the split that leaves the fewest stages to the busiest SM
    const int64_t tiles = div_up(a.M, 128), kb = div_up(a.K, kQK);
    int64_t best = INT64_MAX;
    for (int s = 1; s <= 4 && s <= kb; s *= 2) {
      const int64_t cost = div_up(tiles, sm_count() / s) * (div_up(kb, s) + 2);
      if (cost < best) best = cost, a.split = s;
    }
    // (room for fewer sums is room for more stages)
    return a.split <= 2 ? gemm4_run<1, 32, FMT, OUT, 1, false>(y, x, a, st)
                        : gemm4_run<1, 32, FMT, OUT, 3, false>(y, x, a, st);
  }
  if (rounds(a.M, a.N, a.K, 128, 128, 1, 0.6, 3.0) < rounds(a.M, a.N, a.K, 256, 256, 2, 1.0, 5.0))
    return tma ? gemm4_run<1, 128, FMT, OUT, 0, true>(x, y, a, st)
               : gemm4_run<1, 128, FMT, OUT, 0, false>(x, y, a, st);
  return tma ? gemm4_run<2, 256, FMT, OUT, 0, true>(x, y, a, st)
             : gemm4_run<2, 256, FMT, OUT, 0, false>(x, y, a, st);
}

cudaError_t launch_gemm_fp4(const uint8_t* qa, const uint8_t* sa, const float* ta, const uint8_t* qb,
                            const uint8_t* sb, const float* tb, int64_t M, int64_t N, int64_t K,
                            int fmt, int out_dtype, void* d, int64_t ldd, int32_t* status,
                            cudaStream_t st) {
  if (M == 0 || N == 0) return cudaSuccess;
  const size_t esz = out_dtype == GS_F32 ? 4 : 2;
  if (K == 0)  // empty sums
    return cudaMemset2DAsync(d, (size_t)ldd * esz, 0, (size_t)N * esz, (size_t)M, st);
  if (!encode_fn()) return cudaErrorNotSupported;
  const Operand x = {qa, sa, M}, y = {qb, sb, N};
  const Gemm4Args a = {ta, tb, M, N, K, d, ldd, status, 16, 1, test_stall()};
  const bool tma = (uintptr_t)d % 16 == 0 && ((size_t)ldd * esz) % 16 == 0;
  if (fmt == GS_NVFP4)
    return out_dtype == GS_F32 ? gemm4_pick<GS_NVFP4, GS_F32>(x, y, a, tma, st)
                               : gemm4_pick<GS_NVFP4, GS_BF16>(x, y, a, tma, st);
  return out_dtype == GS_F32 ? gemm4_pick<GS_MXFP4, GS_F32>(x, y, a, tma, st)
                             : gemm4_pick<GS_MXFP4, GS_BF16>(x, y, a, tma, st);
}

}  // namespace gs

// fp4.cu -- microscaled 4-bit tensors: quantisation of a matrix as it lies and
// of its transpose, and dequantisation.
//
// A block of 32 (MXFP4) or 16 (NVFP4) consecutive elements of a row shares a
// scale; elements are e2m1 (sign, two bits of exponent, one of mantissa: 0,
// 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the even element in the low half.
//   MXFP4: scale 2^e, e = floor(log2 amax) - 2 in [-127, 127] (2 is the
//          exponent of the largest element), stored as the byte e + 127;
//          q = e2m1(x 2^-e).
//   NVFP4: a tensor scale t = max(amax of the tensor, 1e-12) / (448 * 6) in
//          fp32, block scales s = e4m3(amax / (6 t)), q = e2m1(x r) with
//          r = fp32(1 / (s t)), or zeros where s is 0.
// All roundings are to nearest, ties to even; e2m1 saturates at 6 (the cvt
// instruction's rule).  The reciprocal is formed once per block: the quotient
// x / (s t) would cost a division per element for a value that is rounded to
// four bits.
//
// Scales lie as the tensor cores' block-scaled products take them: tiles of 128
// rows and 4 scales, 512 bytes each, [row tile][scale tile], the byte of row r
// and scale k at 16 (r % 32) + 4 (r % 128 / 32) + k % 4.  Bytes past the
// matrix's edges are zero.
//
// One CTA takes tiles of 128 x 128 elements, which hold whole scale tiles both
// ways.  A thread takes one block of 16 of a row at a time, in registers; for
// the transpose the tile goes through shared memory, a thread taking the same
// 16 rows of two columns (of one for fp32).  Both directions read x once; the
// tensor's scale needs a pass over x before, and the second pass runs from the
// last tile to the first, so that what L2 still holds of the first pass is read
// from there.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gs_elem.cuh"
#include "gs_fp4.h"
#include "gs_internal.h"

namespace gs {

constexpr int kFTile = 128;
constexpr int kFThreads = 256;
constexpr int kFBlock = 16;  // elements per thread and step
constexpr float kFMax = 6.0f;

// Two e2m1 codes: lo in the low four bits.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float hi, float lo) {
  uint32_t d;
  asm("{\n\t.reg .b8 c;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\t"
      "cvt.u32.u8 %0, c;\n\t}"
      : "=r"(d)
      : "f"(hi), "f"(lo));
  return d;
}
// Two codes of one byte as two f16 (exact), the low four bits' in the low half.
__device__ __forceinline__ uint32_t cvt_e2m1x2_f16x2(uint32_t codes) {
  uint32_t d;
  asm("{\n\t.reg .b8 c;\n\t"
      "cvt.u8.u32 c, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
      : "=r"(d)
      : "r"(codes));
  return d;
}

__device__ __forceinline__ int scale_place(int r, int k) {
  return ((r & 31) << 4) + ((r >> 5 & 3) << 2) + (k & 3);
}

// The tensor scale as a block takes it.
struct Tensor4 {
  float t, t6;
  bool ok;
};
__device__ __forceinline__ Tensor4 tensor4(float t) {
  // outside, r could not be a number below the largest (or the scale is no number)
  return Tensor4{t, __fmul_rn(6.0f, t), t >= 0x1p-100f && t <= 0x1p120f};
}

// A block's scale byte and the factor of its elements from its largest
// magnitude: codes are zero where `ok` is false.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale4(float amax, const Tensor4& ts, float& r, bool& ok) {
  if constexpr (FMT == GS_MXFP4) {
    const uint32_t b = __float_as_uint(amax);
    ok = b < 0x7F800000u;
    // floor(log2 amax) - 2 + 127: the exponent field less 2 (0 for an amax
    // below 2^-124, subnormal ones among them: e = -127 and no less)
    const int c = max((int)(b >> 23) - 2, 0);
    // 2^-e = 2^(127 - c): normal for c in [0, 253] (c is at most 252)
    r = __uint_as_float((uint32_t)(254 - c) << 23);
    return ok ? (uint32_t)c : 255u;
  } else {
    ok = ts.ok && amax < __uint_as_float(0x7F800000u);
    if (!ok) {
      r = 0.0f;
      return kFp8NaN;
    }
    const uint32_t c = cvt_f32x2_fp8x2<GS_E4M3>(0.0f, __fdiv_rn(amax, ts.t6)) & 0xFFu;
    const float s = lo_f16(cvt_fp8x2_f16x2<GS_E4M3>((uint16_t)c));
    r = c ? __fdiv_rn(1.0f, __fmul_rn(s, ts.t)) : 0.0f;
    return c;
  }
}

// 16 consecutive elements as fp32.
template <int DT>
struct Load16;
template <typename Tag>
struct Load16Half {
  static __device__ __forceinline__ void get(const void* p, float (&v)[16]) {
    const uint4 a = ld_stream(static_cast<const uint4*>(p));
    const uint4 b = ld_stream(static_cast<const uint4*>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = lo16<Tag>(w[i]);
      v[2 * i + 1] = hi16<Tag>(w[i]);
    }
  }
};
template <>
struct Load16<GS_BF16> : Load16Half<BF16Tag> {};
template <>
struct Load16<GS_F16> : Load16Half<F16Tag> {};
template <>
struct Load16<GS_F32> {
  static __device__ __forceinline__ void get(const void* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 a = ld_stream(static_cast<const uint4*>(p) + i);
      v[4 * i] = __uint_as_float(a.x);
      v[4 * i + 1] = __uint_as_float(a.y);
      v[4 * i + 2] = __uint_as_float(a.z);
      v[4 * i + 3] = __uint_as_float(a.w);
    }
  }
};

// NaN-propagating largest magnitude: the order of magnitudes' bit patterns.
__device__ __forceinline__ uint32_t amax16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ uint2 codes16(const float (&v)[16], float r, bool ok) {
  uint32_t c[2] = {0, 0};
  if (ok) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i >> 2] |= cvt_e2m1x2(__fmul_rn(v[2 * i + 1], r), __fmul_rn(v[2 * i], r)) << (8 * (i & 3));
  }
  return make_uint2(c[0], c[1]);
}

// A tile's scale bytes, both formats: 128 rows x 128 / block scales.
template <int FMT>
constexpr int kFScales = kFTile / (FMT == GS_NVFP4 ? 16 : 32);
template <int FMT>
constexpr int kFScaleBytes = kFTile * kFScales<FMT>;

// Quantises one block of 16 (half a block of 32: the partner is the lane 1
// away) into its codes, and its scale byte into `sc`.
template <int FMT>
__device__ __forceinline__ uint2 quant16(const float (&v)[16], const Tensor4& ts, uint8_t* sc, int row,
                                         int blk16) {
  uint32_t m = amax16(v);
  if constexpr (FMT == GS_MXFP4) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  float r;
  bool ok;
  const uint32_t s = block_scale4<FMT>(__uint_as_float(m), ts, r, ok);
  const int k = FMT == GS_NVFP4 ? blk16 : blk16 >> 1;
  if (FMT == GS_NVFP4 || (blk16 & 1) == 0) sc[(k >> 2) * 512 + scale_place(row, k)] = (uint8_t)s;
  return codes16(v, r, ok);
}

// Copies a tile's staged scale tiles to the matrix's; k_tiles: scale tiles per row tile.
template <int FMT>
__device__ __forceinline__ void put_scales(const uint8_t* sc, uint8_t* scales, int64_t row_tile,
                                           int64_t col_tile, int64_t k_tiles) {
  constexpr int kPer = kFScales<FMT> / 4;  // scale tiles side by side
#pragma unroll
  for (int i = threadIdx.x; i < kFScaleBytes<FMT> / 4; i += kFThreads) {
    const int64_t kt = col_tile * kPer + i / 128;
    if (kt < k_tiles)
      reinterpret_cast<uint32_t*>(scales)[(row_tile * k_tiles + kt) * 128 + i % 128] =
          reinterpret_cast<const uint32_t*>(sc)[i];
  }
}

struct Quant4Args {
  const void* x;
  int64_t ldx, R, C;
  uint8_t *q, *scales, *qt, *scales_t;
  const float* ts;         // null for MXFP4
  int64_t tiles_r, tiles_c;
};

// ROW, COL: the directions wanted.  VEC: rows start on 16-byte boundaries.
template <int DT, int FMT, bool ROW, bool COL, bool VEC>
__global__ void __launch_bounds__(kFThreads) quant4_kernel(Quant4Args a) {
  using T = typename Elem<DT>::type;
  // a pitch of 130 words of 32 bits (66 of two 16-bit elements) keeps columns'
  // reads and rows' writes to different banks
  constexpr int kPitch = DT == GS_F32 ? kFTile + 1 : kFTile + 2;
  extern __shared__ __align__(16) uint8_t fsmem[];
  T* tile = reinterpret_cast<T*>(fsmem);
  __shared__ __align__(16) uint8_t sc[kFScaleBytes<FMT>];
  __shared__ __align__(16) uint8_t sct[COL ? kFScaleBytes<FMT> : 16];
  const int tid = threadIdx.x;
  const int64_t n_tiles = a.tiles_r * a.tiles_c;
  const Tensor4 ts = FMT == GS_NVFP4 ? tensor4(*a.ts) : Tensor4{1.0f, 6.0f, true};
  const int64_t k_tiles = (a.C + 16 * (FMT == GS_NVFP4 ? 4 : 8) - 1) / (16 * (FMT == GS_NVFP4 ? 4 : 8));
  const int64_t kt_tiles = (a.R + 16 * (FMT == GS_NVFP4 ? 4 : 8) - 1) / (16 * (FMT == GS_NVFP4 ? 4 : 8));
  for (int64_t i = blockIdx.x; i < n_tiles; i += gridDim.x) {
    const int64_t at = n_tiles - 1 - i;
    const int64_t tr = at / a.tiles_c, tc = at % a.tiles_c;
    const int64_t r0 = tr * kFTile, c0 = tc * kFTile;
    // 128 x 8 blocks of 16: a warp takes 4 rows, lanes along the row
#pragma unroll
    for (int j = 0; j < kFTile * 8 / kFThreads; ++j) {
      const int row = j * (kFThreads / 8) + tid / 8, blk = tid % 8;
      const int64_t r = r0 + row, c = c0 + blk * kFBlock;
      const bool in = r < a.R && c < a.C;
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.0f;
      if (in) {
        const int64_t off = r * a.ldx + c;
        if constexpr (VEC) {
          Load16<DT>::get(static_cast<const T*>(a.x) + off, v);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = load1<DT>(a.x, off + e);
        }
      }
      if constexpr (COL) {
#pragma unroll
        for (int e = 0; e < 16; ++e) tile[row * kPitch + blk * kFBlock + e] = Elem<DT>::put(v[e]);
      }
      if constexpr (ROW) {
        const uint2 c16 = quant16<FMT>(v, ts, sc, row, blk);
        // past the edges: zeros in the padding of the scale tiles
        if (!in) {
          const int k = FMT == GS_NVFP4 ? blk : blk >> 1;
          if (FMT == GS_NVFP4 || (blk & 1) == 0) sc[(k >> 2) * 512 + scale_place(row, k)] = 0;
        } else {
          uint8_t* to = a.q + r * (a.C / 2) + c / 2;
          *reinterpret_cast<uint2*>(to) = c16;
        }
      }
    }
    if constexpr (COL) {
      __syncthreads();
      // columns: a thread takes 16 rows of a column; 8 such runs per column
#pragma unroll
      for (int j = 0; j < kFTile * 8 / kFThreads; ++j) {
        const int run = tid % 8, col = j * (kFThreads / 8) + tid / 8;
        const int64_t c = c0 + col, r = r0 + run * kFBlock;
        const bool in = c < a.C && r < a.R;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = Elem<DT>::get(tile[(run * kFBlock + e) * kPitch + col]);
        const uint2 c16 = quant16<FMT>(v, ts, sct, col, run);
        if (!in) {
          const int k = FMT == GS_NVFP4 ? run : run >> 1;
          if (FMT == GS_NVFP4 || (run & 1) == 0) sct[(k >> 2) * 512 + scale_place(col, k)] = 0;
        } else {
          *reinterpret_cast<uint2*>(a.qt + c * (a.R / 2) + r / 2) = c16;
        }
      }
    }
    __syncthreads();
    if constexpr (ROW) put_scales<FMT>(sc, a.scales, tr, tc, k_tiles);
    if constexpr (COL) put_scales<FMT>(sct, a.scales_t, tc, tr, kt_tiles);
    __syncthreads();
  }
}

// ---- the tensor scale -----------------------------------------------------------
// The largest magnitude of R rows: one partial per CTA.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kFThreads)
    amax_rows_kernel(const void* __restrict__ x, int64_t ldx, int64_t R, int64_t C,
                     uint32_t* __restrict__ partials) {
  __shared__ uint32_t red[kFThreads / 32];
  using T = typename Elem<DT>::type;
  uint32_t m = 0;
  const int64_t per_row = C / kFBlock;  // C is a multiple of 32
  const int64_t n = R * per_row, step = (int64_t)gridDim.x * kFThreads;
  for (int64_t i = (int64_t)blockIdx.x * kFThreads + threadIdx.x; i < n; i += step) {
    const int64_t off = i / per_row * ldx + i % per_row * kFBlock;
    float v[16];
    if constexpr (VEC) {
      Load16<DT>::get(static_cast<const T*>(x) + off, v);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = load1<DT>(x, off + e);
    }
    m = max(m, amax16(v));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kFThreads / 32; ++w) m = max(m, red[w]);
    partials[blockIdx.x] = m;
  }
}

__global__ void __launch_bounds__(kFThreads)
    tensor_scale_kernel(const uint32_t* __restrict__ partials, int n, float* __restrict__ ts) {
  __shared__ uint32_t red[kFThreads / 32];
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n; i += kFThreads) m = max(m, partials[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kFThreads / 32; ++w) m = max(m, red[w]);
    const float amax = __uint_as_float(m);
    // Inf or NaN in the tensor: no scale, and every block's is NaN
    *ts = m >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu)
                           : __fdiv_rn(fmaxf(amax, kAmaxFloor), Fp8Max<GS_E4M3>::value * kFMax);
  }
}

template <int DT, int FMT, bool ROW, bool COL, bool VEC>
static cudaError_t quant4_t(const Quant4Args& a, cudaStream_t st) {
  auto k = quant4_kernel<DT, FMT, ROW, COL, VEC>;
  constexpr int kPitch = DT == GS_F32 ? kFTile + 1 : kFTile + 2;
  constexpr int smem = COL ? kFTile * kPitch * (DT == GS_F32 ? 4 : 2) : 0;
  int occ = 0;
  const cudaError_t e = kernel_blocks_per_sm((const void*)k, kFThreads, smem, &occ);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  const int64_t tiles = a.tiles_r * a.tiles_c;
  k<<<(unsigned)std::min<int64_t>(tiles, (int64_t)sm_count() * 64), kFThreads, smem, st>>>(a);
  return cudaGetLastError();
}
template <int DT, int FMT, bool ROW, bool COL>
static cudaError_t quant4_v(const Quant4Args& a, bool vec, cudaStream_t st) {
  return vec ? quant4_t<DT, FMT, ROW, COL, true>(a, st) : quant4_t<DT, FMT, ROW, COL, false>(a, st);
}
template <int DT, int FMT>
static cudaError_t quant4_d(const Quant4Args& a, bool vec, cudaStream_t st) {
  if (!a.qt) return quant4_v<DT, FMT, true, false>(a, vec, st);
  if (!a.q) return quant4_v<DT, FMT, false, true>(a, vec, st);
  return quant4_v<DT, FMT, true, true>(a, vec, st);
}
template <int DT>
static cudaError_t quant4_dt(Quant4Args a, int fmt, float* ts, uint32_t* partials, cudaStream_t st) {
  using T = typename Elem<DT>::type;
  const bool vec = (uintptr_t)a.x % 16 == 0 && (a.ldx * sizeof(T)) % 16 == 0;
  if (partials) {
    const int64_t n = a.R * (a.C / kFBlock);
    const unsigned grid = (unsigned)std::max<int64_t>(
        1, std::min<int64_t>({(n + kFThreads - 1) / kFThreads, (int64_t)kMaxAmaxBlocks,
                              (int64_t)sm_count() * 8}));
    if (vec) amax_rows_kernel<DT, true><<<grid, kFThreads, 0, st>>>(a.x, a.ldx, a.R, a.C, partials);
    else amax_rows_kernel<DT, false><<<grid, kFThreads, 0, st>>>(a.x, a.ldx, a.R, a.C, partials);
    tensor_scale_kernel<<<1, kFThreads, 0, st>>>(partials, (int)grid, ts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.R == 0 || a.C == 0) return cudaSuccess;
  return fmt == GS_MXFP4 ? quant4_d<DT, GS_MXFP4>(a, vec, st) : quant4_d<DT, GS_NVFP4>(a, vec, st);
}

cudaError_t launch_quant4(const void* x, int64_t ldx, int dtype, int64_t R, int64_t C, int fmt,
                          uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t, float* ts,
                          uint32_t* partials, cudaStream_t st) {
  const Quant4Args a = {x, ldx, R, C, q, scales, qt, scales_t, ts, (R + kFTile - 1) / kFTile,
                        (C + kFTile - 1) / kFTile};
  if (dtype == GS_F32) return quant4_dt<GS_F32>(a, fmt, ts, partials, st);
  if (dtype == GS_F16) return quant4_dt<GS_F16>(a, fmt, ts, partials, st);
  return quant4_dt<GS_BF16>(a, fmt, ts, partials, st);
}

// ---- dequantisation ---------------------------------------------------------------
// y = fp32(v s) t: the first product is exact (2 bits of e2m1 times 4 of e4m3,
// or a power of two), the second rounds; then to the output's type.
template <int DT, int FMT, bool VEC>
__global__ void __launch_bounds__(kFThreads)
    dequant4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                    const float* __restrict__ tsp, int64_t R, int64_t C, void* __restrict__ y,
                    int64_t ldy) {
  const float t = FMT == GS_NVFP4 ? *tsp : 1.0f;
  constexpr int kBlk = FMT == GS_NVFP4 ? 16 : 32;
  const int64_t k_tiles = (C + 4 * kBlk - 1) / (4 * kBlk);
  const int64_t per_row = C / kFBlock, n = R * per_row;
  for (int64_t i = (int64_t)blockIdx.x * kFThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kFThreads) {
    const int64_t r = i / per_row, b = i % per_row, k = b * kFBlock / kBlk;
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(q) + i);
    const uint32_t sb = scales[(r / 128 * k_tiles + k / 4) * 512 + scale_place((int)(r & 127), (int)(k & 3))];
    float s;
    if constexpr (FMT == GS_NVFP4) s = lo_f16(cvt_fp8x2_f16x2<GS_E4M3>((uint16_t)sb));
    else s = sb == 0 ? 0x1p-127f : __uint_as_float(sb == 255u ? 0x7FC00000u : sb << 23);
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = cvt_e2m1x2_f16x2((j < 4 ? c.x : c.y) >> (8 * (j & 3)) & 0xFFu);
      v[2 * j] = __fmul_rn(__fmul_rn(lo_f16(h), s), t);
      v[2 * j + 1] = __fmul_rn(__fmul_rn(hi_f16(h), s), t);
    }
    const int64_t off = r * ldy + b * kFBlock;
    if constexpr (VEC) {
      if constexpr (DT == GS_F32) {
        uint4* to = reinterpret_cast<uint4*>(static_cast<float*>(y) + off);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_stream(to + j, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                       __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
      } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = (uint32_t)Elem<DT>::put(v[2 * j]) | (uint32_t)Elem<DT>::put(v[2 * j + 1]) << 16;
        uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + off);
        st_stream(to, make_uint4(w[0], w[1], w[2], w[3]));
        st_stream(to + 1, make_uint4(w[4], w[5], w[6], w[7]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) store1<DT>(y, off + j, v[j]);
    }
  }
}

template <int DT, int FMT>
static cudaError_t dequant4_t(const uint8_t* q, const uint8_t* scales, const float* ts, int64_t R,
                              int64_t C, void* y, int64_t ldy, cudaStream_t st) {
  const int64_t n = R * (C / kFBlock);
  const unsigned grid =
      (unsigned)std::min<int64_t>((n + kFThreads - 1) / kFThreads, (int64_t)sm_count() * 64);
  if ((uintptr_t)y % 16 == 0 && (ldy * (DT == GS_F32 ? 4 : 2)) % 16 == 0)
    dequant4_kernel<DT, FMT, true><<<grid, kFThreads, 0, st>>>(q, scales, ts, R, C, y, ldy);
  else
    dequant4_kernel<DT, FMT, false><<<grid, kFThreads, 0, st>>>(q, scales, ts, R, C, y, ldy);
  return cudaGetLastError();
}

cudaError_t launch_dequant4(const uint8_t* q, const uint8_t* scales, const float* ts, int64_t R,
                            int64_t C, int fmt, int out_dtype, void* y, int64_t ldy, cudaStream_t st) {
  if (fmt == GS_NVFP4) {
    if (out_dtype == GS_F32) return dequant4_t<GS_F32, GS_NVFP4>(q, scales, ts, R, C, y, ldy, st);
    if (out_dtype == GS_F16) return dequant4_t<GS_F16, GS_NVFP4>(q, scales, ts, R, C, y, ldy, st);
    return dequant4_t<GS_BF16, GS_NVFP4>(q, scales, ts, R, C, y, ldy, st);
  }
  if (out_dtype == GS_F32) return dequant4_t<GS_F32, GS_MXFP4>(q, scales, ts, R, C, y, ldy, st);
  if (out_dtype == GS_F16) return dequant4_t<GS_F16, GS_MXFP4>(q, scales, ts, R, C, y, ldy, st);
  return dequant4_t<GS_BF16, GS_MXFP4>(q, scales, ts, R, C, y, ldy, st);
}

}  // namespace gs

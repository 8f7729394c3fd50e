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
// ways.  A thread takes runs of 16 of a row in registers; for the transpose the
// tile goes through shared memory, a thread taking a block's rows of two columns
// (of one for fp32), and the codes go through it again so that a column's 64 bytes
// are stored together; the next tile is loaded meanwhile (16384 x 8192 bf16 both
// ways: 137 us without, 129 with it and three CTAs per SM).  Both directions read x
// once; the tensor's scale needs a pass over x before, and the second pass runs from the last tile to the first, so
// that what L2 still holds of the first pass is read from there.  Small tensors
// are one cluster's, which reads its own part twice.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gs_elem.cuh"
#include "gs_fp4.h"
#include "gs_internal.h"

namespace gs {

constexpr int kFTile = 128;
constexpr int kFThreads = 256;
constexpr int kFBlock = 16;  // elements per thread and step
// Elements up to which one cluster takes a tensor's scale and codes in one
// launch (a second launch costs the host 4 us), and its most CTAs.
constexpr int64_t kFOneElems = 1 << 17;
constexpr int kFOneCtas = 8;
constexpr float kFMax = 6.0f;

// Eight values times r as e2m1 codes, the first in the low four bits.
__device__ __forceinline__ uint32_t codes8(const uint64_t (&v)[4], uint64_t r) {
  uint32_t d;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(v[i]), "l"(r));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "l"(p));
  }
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
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
  float t6, r6;        // 6 t and its reciprocal
  const float* table;  // 1 / (s t) of every s, 0 for 0
  bool ok;
};
// Fills the table (one entry per thread from 128 on) and gives the rest.
__device__ __forceinline__ Tensor4 tensor4(float t, float* table) {
  if (threadIdx.x < 128) {
    const float s = lo_f16(cvt_fp8x2_f16x2<GS_E4M3>((uint16_t)threadIdx.x));
    table[threadIdx.x] = threadIdx.x ? __fdiv_rn(1.0f, __fmul_rn(s, t)) : 0.0f;
  }
  __syncthreads();
  const float t6 = __fmul_rn(6.0f, t);
  // outside, 1 / (s t) could not be a number (or t is none)
  return Tensor4{t6, __fdiv_rn(1.0f, t6), table, t >= 0x1p-100f && t <= 0x1p120f};
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
    // the quotient as IEEE division rounds it wherever it is not 0 in e4m3, or
    // far beyond its range (where the residuals could overflow)
    ok = ts.ok && amax < __uint_as_float(0x7F800000u);
    const float q = exact_quotient<2>(amax, ts.t6, ts.r6);
    const float u = __fmul_rn(amax, ts.r6) < 1024.0f ? q : 1024.0f;
    const uint32_t k = cvt_f32x2_fp8x2<GS_E4M3>(0.0f, u) & 0x7Fu;
    const uint32_t c = ok ? k : kFp8NaN;
    r = ts.table[c];
    return c;
  }
}

// N consecutive or strided elements of a block as loaded, their largest magnitude
// (NaN counts as the largest: the order of magnitudes' bit patterns) and their
// values.  16-bit elements stay in pairs until they are scaled.
template <int DT>
struct Half {
  static __device__ __forceinline__ float lo(uint32_t w) {
    if constexpr (DT == GS_BF16) return lo_bf16(w);
    else return lo_f16(w);
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    if constexpr (DT == GS_BF16) return hi_bf16(w);
    else return hi_f16(w);
  }
};
template <int DT>
__device__ __forceinline__ float mag16(uint32_t m) {  // of a 16-bit pattern without its sign
  if constexpr (DT == GS_BF16) return __uint_as_float(m << 16);
  else return Half<DT>::lo(m);
}

// The larger magnitudes of m and w (for 16 bits of either half), NaN the largest
// of all; signs in the result mean nothing.
template <int DT>
__device__ __forceinline__ uint32_t max_mag(uint32_t m, uint32_t w) {
  uint32_t d;
  if constexpr (DT == GS_F32) d = max(m, w & 0x7FFFFFFFu);
  else if constexpr (DT == GS_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  return d;
}
// What max_mag left, as the bit pattern of one fp32 magnitude.
template <int DT>
__device__ __forceinline__ uint32_t mag_of(uint32_t m) {
  if constexpr (DT == GS_F32) return m;
  else return __float_as_uint(mag16<DT>(max(m & 0x7FFFu, m >> 16 & 0x7FFFu)));
}

// 16 consecutive elements of a row in registers.
template <int DT>
struct Run16 {
  static constexpr int kWords = DT == GS_F32 ? 16 : 8;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // From element off of x, ALIGN: bytes every run begins at a multiple of (32, 16,
  // or less).
  template <int ALIGN>
  __device__ __forceinline__ void load(const void* x, int64_t off) {
    const typename Elem<DT>::type* p = static_cast<const typename Elem<DT>::type*>(x) + off;
    if constexpr (ALIGN == 32) {
#pragma unroll
      for (int i = 0; i < kWords / 8; ++i) {
        const V8 a = ld_stream8(reinterpret_cast<const uint32_t*>(p) + 8 * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * i + e] = a.w[e];
      }
    } else if constexpr (ALIGN == 16) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 a = ld_stream(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (DT == GS_F32) w[i] = __float_as_uint(p[i]);
        else w[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
      }
    }
  }
  // The same with the alignment as a number, the same for all threads.
  __device__ __forceinline__ void load(const void* x, int64_t off, int align) {
    if (align == 32) load<32>(x, off);
    else if (align == 16) load<16>(x, off);
    else load<1>(x, off);
  }
  // Takes the elements into a running maximum of magnitudes (start: 0), in the
  // elements' own type and, of 16 bits, by halves; see mag_of.
  __device__ __forceinline__ void fold(uint32_t& m) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) m = max_mag<DT>(m, w[i]);
  }
  // Bit pattern of the largest magnitude as fp32.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
    fold(m);
    return mag_of<DT>(m);
  }
  __device__ __forceinline__ uint2 codes(float r, bool ok) const {
    uint32_t c[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint64_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == GS_F32)
          v[i] = pair(__uint_as_float(w[8 * g + 2 * i]), __uint_as_float(w[8 * g + 2 * i + 1]));
        else v[i] = pair(Half<DT>::lo(w[4 * g + i]), Half<DT>::hi(w[4 * g + i]));
      }
      c[g] = codes8(v, pair(r, r)) & (ok ? 0xFFFFFFFFu : 0u);
    }
    return make_uint2(c[0], c[1]);
  }
};

// A tile's scale bytes: 128 rows x 128 / block scales.
template <int FMT>
constexpr int kFBlk = FMT == GS_NVFP4 ? 16 : 32;
template <int FMT>
constexpr int kFScales = kFTile / kFBlk<FMT>;
template <int FMT>
constexpr int kFScaleBytes = kFTile * kFScales<FMT>;

// Copies a tile's staged scale tiles to the matrix's, where they lie together;
// k_tiles: scale tiles per row tile.
template <int FMT>
__device__ __forceinline__ void put_scales(const uint8_t* sc, uint8_t* scales, int64_t row_tile,
                                           int64_t col_tile, int64_t k_tiles) {
  constexpr int kPer = kFScales<FMT> / 4;  // scale tiles side by side
  static_assert(kPer * 32 <= kFThreads, "16 bytes a thread");
  const int64_t kt = col_tile * kPer;
  const int n = 32 * (int)min((int64_t)kPer, k_tiles - kt);
  if ((int)threadIdx.x < n)
    reinterpret_cast<uint4*>(scales + (row_tile * k_tiles + kt) * 512)[threadIdx.x] =
        reinterpret_cast<const uint4*>(sc)[threadIdx.x];
}

struct Quant4Args {
  const void* x;
  int64_t ldx, R, C;
  uint8_t *q, *scales, *qt, *scales_t;
  float* ts;                 // null for MXFP4
  const uint32_t* partials;  // of the pass before, or null: ts is read
  int n_partials;
  int align;                 // of the runs of 16 (see Run16)
  int64_t tiles_r, tiles_c;
};

// The block's largest of every thread's m, in all threads.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int w = 1; w < kFThreads / 32; ++w) m = max(m, red[w]);
  __syncthreads();
  return m;
}
__device__ __forceinline__ float scale_of_amax(uint32_t m) {
  // Inf or NaN in the tensor: no scale, and every block's is NaN
  return m >= 0x7F800000u
             ? __uint_as_float(0x7FFFFFFFu)
             : __fdiv_rn(fmaxf(__uint_as_float(m), kAmaxFloor), Fp8Max<GS_E4M3>::value * kFMax);
}

// ROW, COL: the directions wanted.  ONE: a single cluster forms the tensor scale
// too.
template <int DT, int FMT, bool ROW, bool COL, bool ONE>
__global__ void __launch_bounds__(kFThreads, DT == GS_F32 ? 2 : COL ? 3 : 5) quant4_kernel(Quant4Args a) {
  constexpr int kBlk = kFBlk<FMT>;
  constexpr int kRuns = kFTile * 8 / kFThreads;  // per thread and tile
  static_assert(kFThreads == 256 && kRuns == 4, "a thread's runs are 32 rows apart");
  // Words per row of the tile kept for the transpose: odd, so that a column of
  // words and a row of them go to different banks.
  constexpr int kPitch = DT == GS_F32 ? kFTile + 1 : kFTile / 2 + 1;
  constexpr int kOutPitch = 72;                  // bytes per column of its codes, 64 and 8
  extern __shared__ __align__(16) uint32_t tile[];
  uint8_t* const out_t = reinterpret_cast<uint8_t*>(tile + kFTile * kPitch);
  __shared__ __align__(16) uint8_t sc[kFScaleBytes<FMT>];
  __shared__ __align__(16) uint8_t sct[COL ? kFScaleBytes<FMT> : 16];
  __shared__ uint32_t red[kFThreads / 32];
  __shared__ uint32_t peers[ONE ? kFOneCtas : 1];
  __shared__ float table[FMT == GS_NVFP4 ? 128 : 1];
  const int tid = threadIdx.x;
  const int64_t n_tiles = a.tiles_r * a.tiles_c;
  const int64_t k_tiles = (a.C + 4 * kBlk - 1) / (4 * kBlk), kt_tiles = (a.R + 4 * kBlk - 1) / (4 * kBlk);

  Tensor4 ts = {6.0f, 1.0f, table, true};
  if constexpr (FMT == GS_NVFP4) {
    float t;
    if (ONE || a.partials) {
      uint32_t m = 0;
      if constexpr (ONE) {
        const int64_t per_row = a.C / kFBlock;
        for (int64_t at = blockIdx.x * kFThreads + tid; at < a.R * per_row; at += gridDim.x * kFThreads) {
          Run16<DT> v;
          v.load(a.x, at / per_row * a.ldx + at % per_row * kFBlock, a.align);
          v.fold(m);
        }
        m = mag_of<DT>(m);
        m = block_max(m, red);
        cluster_barrier();  // every CTA of the cluster has begun
        if (tid < (int)cluster_size())
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(&peers[cluster_rank()], (uint32_t)tid)),
                       "r"(m)
                       : "memory");
        cluster_barrier();
        for (uint32_t i = 0; i < cluster_size(); ++i) m = max(m, peers[i]);
      } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are there
        for (int i = tid; i < a.n_partials; i += kFThreads) m = max(m, __ldcg(a.partials + i));
        m = block_max(m, red);
      }
      t = scale_of_amax(m);
      if (blockIdx.x == 0 && tid == 0) *a.ts = t;
    } else {
      t = *a.ts;
    }
    ts = tensor4(t, table);
  }

  // Tile i, last tile first: what L2 holds of a pass over x before is read from
  // there.
  const auto place = [&](int64_t i, int64_t& tr, int64_t& tc) {
    const unsigned at = (unsigned)(n_tiles - 1 - i), across = (unsigned)a.tiles_c;
    tr = at / across;
    tc = at % across;
  };
  // rows tid / 8 + 32 j: eight lanes to a row, a run of 16 each
  const int blk = tid & 7, row0 = tid >> 3 & 31;
  Run16<DT> v[kRuns];
  const auto load = [&](int64_t tr, int64_t tc) {
    const int64_t c = tc * kFTile + blk * kFBlock, r = tr * kFTile;
    const int rows = c < a.C ? (int)min((int64_t)kFTile, a.R - r) : 0;
    const int64_t first = (r + row0) * a.ldx + c;
    const auto all = [&](auto align) {
#pragma unroll
      for (int j = 0; j < kRuns; ++j) {
        v[j].zero();
        if (row0 + 32 * j < rows) v[j].template load<decltype(align)::value>(a.x, first + 32 * j * a.ldx);
      }
    };
    if (a.align == 32) all(std::integral_constant<int, 32>());
    else if (a.align == 16) all(std::integral_constant<int, 16>());
    else all(std::integral_constant<int, 1>());
  };
  int64_t tr, tc, tr_n = 0, tc_n = 0;
  if (blockIdx.x < n_tiles) place(blockIdx.x, tr_n, tc_n);
  if constexpr (COL) {
    if (blockIdx.x < n_tiles) load(tr_n, tc_n);
  }
  for (int64_t i = blockIdx.x; i < n_tiles; i += gridDim.x) {
    tr = tr_n;
    tc = tc_n;
    const bool more = i + gridDim.x < n_tiles;
    if (more) place(i + gridDim.x, tr_n, tc_n);
    if constexpr (!COL) load(tr, tc);
    const int64_t r0 = tr * kFTile, c0 = tc * kFTile;
    const int rows = c0 + blk * kFBlock < a.C ? (int)min((int64_t)kFTile, a.R - r0) : 0;
    uint8_t* const to = ROW ? a.q + (r0 + row0) * (a.C / 2) + (c0 + blk * kFBlock) / 2 : nullptr;
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int row = 32 * j + row0;
      const bool in = row < rows;
      if constexpr (COL) {
#pragma unroll
        for (int e = 0; e < Run16<DT>::kWords; ++e)
          tile[row * kPitch + blk * Run16<DT>::kWords + e] = v[j].w[e];
      }
      if constexpr (ROW) {
        uint32_t m = v[j].amax();
        if constexpr (FMT == GS_MXFP4) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        float r;
        bool ok;
        const uint32_t s = block_scale4<FMT>(__uint_as_float(m), ts, r, ok);
        // past the edges: zeros in the padding of the scale tiles
        const int k = FMT == GS_NVFP4 ? blk : blk >> 1;
        if (FMT == GS_NVFP4 || (blk & 1) == 0)
          sc[(k >> 2) * 512 + (row0 << 4) + (j << 2) + (k & 3)] = (uint8_t)(in ? s : 0u);
        if (in) *reinterpret_cast<uint2*>(to + 32 * j * (a.C / 2)) = v[j].codes(r, ok);
      }
    }
    if constexpr (COL) {
      if (more) load(tr_n, tc_n);  // while this tile's columns are taken
      __syncthreads();
      // a word's columns (two of 16 bits, one of 32), the rows of a block
      constexpr int kSide = DT == GS_F32 ? kFTile : kFTile / 2;
      constexpr int kStep = kFThreads / kSide;
#pragma unroll
      for (int k = tid / kSide; k < kFScales<FMT>; k += kStep) {
        const int word = tid % kSide;
        uint32_t w[kBlk];
#pragma unroll
        for (int e = 0; e < kBlk; ++e) w[e] = tile[(k * kBlk + e) * kPitch + word];
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int e = 0; e < kBlk; ++e) m0 = max_mag<DT>(m0, w[e]);
        if constexpr (DT != GS_F32) {
          m1 = __float_as_uint(mag16<DT>(m0 >> 16 & 0x7FFFu));
          m0 = __float_as_uint(mag16<DT>(m0 & 0x7FFFu));
        }
#pragma unroll
        for (int side = 0; side < (DT == GS_F32 ? 1 : 2); ++side) {
          const int col = DT == GS_F32 ? word : 2 * word + side;
          const bool inside = c0 + col < a.C && r0 + k * kBlk < a.R;
          float r;
          bool ok;
          const uint32_t s = block_scale4<FMT>(__uint_as_float(side ? m1 : m0), ts, r, ok);
          sct[(k >> 2) * 512 + scale_place(col, k)] = (uint8_t)(inside ? s : 0u);
          uint32_t c[kBlk / 8];
#pragma unroll
          for (int g = 0; g < kBlk / 8; ++g) {
            uint64_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x0 = w[8 * g + 2 * e], x1 = w[8 * g + 2 * e + 1];
              if constexpr (DT == GS_F32) p[e] = pair(__uint_as_float(x0), __uint_as_float(x1));
              else p[e] = side ? pair(Half<DT>::hi(x0), Half<DT>::hi(x1))
                               : pair(Half<DT>::lo(x0), Half<DT>::lo(x1));
            }
            c[g] = codes8(p, pair(r, r)) & (ok ? 0xFFFFFFFFu : 0u);
          }
#pragma unroll
          for (int g = 0; g < kBlk / 8; g += 2)
            *reinterpret_cast<uint2*>(out_t + col * kOutPitch + k * (kBlk / 2) + 4 * g) =
                make_uint2(c[g], c[g + 1]);
        }
      }
      __syncthreads();
      // 64 bytes of codes per column, eight lanes to a column
#pragma unroll
      for (int j = 0; j < kFTile * 8 / kFThreads; ++j) {
        const int col = j * (kFThreads / 8) + tid / 8, part = tid % 8;
        if (c0 + col < a.C && r0 + 16 * part < a.R)
          *reinterpret_cast<uint2*>(a.qt + (c0 + col) * (a.R / 2) + r0 / 2 + 8 * part) =
              *reinterpret_cast<const uint2*>(out_t + col * kOutPitch + 8 * part);
      }
    } else {
      __syncthreads();
    }
    if constexpr (ROW) put_scales<FMT>(sc, a.scales, tr, tc, k_tiles);
    if constexpr (COL) put_scales<FMT>(sct, a.scales_t, tc, tr, kt_tiles);
    __syncthreads();
  }
}

// ---- the tensor scale -----------------------------------------------------------
// The largest magnitude of R rows of C (a multiple of 16) elements: one partial
// per CTA.  A tensor without gaps comes as one row.
template <int DT>
__global__ void __launch_bounds__(kFThreads)
    amax_rows_kernel(const void* __restrict__ x, int64_t ldx, int64_t R, int64_t C, int align,
                     uint32_t* __restrict__ partials) {
  __shared__ uint32_t red[kFThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  uint32_t m = 0;
  const int64_t per_row = C / kFBlock, n = R * per_row, step = (int64_t)gridDim.x * kFThreads;
  int64_t i = (int64_t)blockIdx.x * kFThreads + threadIdx.x;
  int64_t r = i / per_row, c = i % per_row;
  const int64_t dr = step / per_row, dc = step % per_row;
  const auto next = [&] {
    i += step;
    r += dr;
    c += dc;
    if (c >= per_row) c -= per_row, ++r;
  };
  constexpr int kAhead = DT == GS_F32 ? 2 : 4;
  while (i < n) {
    Run16<DT> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      v[u].zero();
      if (i < n) v[u].load(x, r * ldx + c * kFBlock, align);
      next();
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u].fold(m);
  }
  m = block_max(mag_of<DT>(m), red);
  if (threadIdx.x == 0) partials[blockIdx.x] = m;
}

// Sets the tensor scale of an empty tensor.
__global__ void empty_scale_kernel(float* ts) { *ts = scale_of_amax(0); }

template <int DT, int FMT, bool ROW, bool COL, bool ONE>
static cudaError_t quant4_t(const Quant4Args& a, cudaStream_t st) {
  auto k = quant4_kernel<DT, FMT, ROW, COL, ONE>;
  constexpr int kPitch = DT == GS_F32 ? kFTile + 1 : kFTile / 2 + 1;
  constexpr int smem = COL ? kFTile * kPitch * 4 + kFTile * 72 : 0;
  int occ = 0;
  const cudaError_t e = kernel_blocks_per_sm((const void*)k, kFThreads, smem, &occ);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  const int64_t tiles = a.tiles_r * a.tiles_c;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  if (ONE) {
    unsigned ctas = 1;
    while (ctas < kFOneCtas && ctas < tiles) ctas *= 2;
    cfg.gridDim = dim3(ctas);
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
  } else {
    // tiles loaded ahead: one wave; else several, which even out the SMs' progress
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, (int64_t)sm_count() * (COL ? occ : 64)));
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = ONE || a.partials ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, a);
}
template <int DT, int FMT, bool ROW, bool COL>
static cudaError_t quant4_v(const Quant4Args& a, bool one, cudaStream_t st) {
  if constexpr (FMT == GS_NVFP4) {
    if (one) return quant4_t<DT, FMT, ROW, COL, true>(a, st);
  }
  return quant4_t<DT, FMT, ROW, COL, false>(a, st);
}
template <int DT, int FMT>
static cudaError_t quant4_d(const Quant4Args& a, bool one, cudaStream_t st) {
  if (!a.qt) return quant4_v<DT, FMT, true, false>(a, one, st);
  if (!a.q) return quant4_v<DT, FMT, false, true>(a, one, st);
  return quant4_v<DT, FMT, true, true>(a, one, st);
}

// Bytes (32, 16 or 1) that every run of 16 elements begins at a multiple of.
template <int DT>
static int run_align(const void* p, int64_t ld) {
  const uintptr_t b = (uintptr_t)p | (uintptr_t)(ld * (int64_t)sizeof(typename Elem<DT>::type));
  return b % 32 == 0 ? 32 : b % 16 == 0 ? 16 : 1;
}

template <int DT>
static cudaError_t quant4_dt(Quant4Args a, int fmt, uint32_t* partials, cudaStream_t st) {
  if (a.R == 0 || a.C == 0) {
    if (partials) empty_scale_kernel<<<1, 1, 0, st>>>(a.ts);
    return cudaGetLastError();
  }
  a.align = run_align<DT>(a.x, a.ldx);
  const bool one = partials && a.R * a.C <= kFOneElems;
  if (partials && !one) {
    const bool gaps = a.ldx != a.C;
    const int64_t rows = gaps ? a.R : 1, cols = gaps ? a.C : a.R * a.C, n = rows * (cols / kFBlock);
    const unsigned grid = (unsigned)std::min<int64_t>({(n + kFThreads - 1) / kFThreads, (int64_t)kMaxAmaxBlocks,
                                                       (int64_t)sm_count() * 8});
    amax_rows_kernel<DT><<<grid, kFThreads, 0, st>>>(a.x, a.ldx, rows, cols, a.align, partials);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    a.partials = partials;
    a.n_partials = (int)grid;
  }
  return fmt == GS_MXFP4 ? quant4_d<DT, GS_MXFP4>(a, false, st) : quant4_d<DT, GS_NVFP4>(a, one, st);
}

cudaError_t launch_quant4(const void* x, int64_t ldx, int dtype, int64_t R, int64_t C, int fmt,
                          uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t, float* ts,
                          uint32_t* partials, cudaStream_t st) {
  const Quant4Args a = {x, R == 1 ? C : ldx, R, C, q, scales, qt, scales_t, ts, nullptr, 0, 1,
                        (R + kFTile - 1) / kFTile, (C + kFTile - 1) / kFTile};
  if (dtype == GS_F32) return quant4_dt<GS_F32>(a, fmt, partials, st);
  if (dtype == GS_F16) return quant4_dt<GS_F16>(a, fmt, partials, st);
  return quant4_dt<GS_BF16>(a, fmt, partials, st);
}

// ---- dequantisation ---------------------------------------------------------------
// y = fp32(v s) t: the first product is exact (2 bits of e2m1 times 4 of e4m3,
// or a power of two), the second rounds; then to the output's type.  A CTA takes
// 128 rows x 256 columns, whose scale tiles it stages; sixteen lanes to a row.
constexpr int kDCols = 256;

// ROWS: of a CTA, 128 or, for tensors that would leave SMs without any, 16 (see
// dequant4_t).
template <int DT, int FMT, int ROWS>
__global__ void __launch_bounds__(kFThreads)
    dequant4_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                    const float* __restrict__ tsp, int64_t R, int64_t C, void* __restrict__ y,
                    int64_t ldy, int align, int64_t tiles_c) {
  constexpr int kBlk = kFBlk<FMT>, kPer = kDCols / (4 * kBlk);  // scale tiles side by side
  __shared__ __align__(16) uint8_t sc[kPer * 512];
  const float t = FMT == GS_NVFP4 ? *tsp : 1.0f;
  const int tid = threadIdx.x;
  const int64_t k_tiles = (C + 4 * kBlk - 1) / (4 * kBlk);
  const int64_t row0 = blockIdx.x / tiles_c * ROWS, tc = blockIdx.x % tiles_c;
  const int64_t c = tc * kDCols + tid % 16 * kFBlock;
  constexpr int kRows = ROWS * 16 / kFThreads;
  uint2 codes[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = row0 + tid / 16 + j * (kFThreads / 16);
    codes[j] = make_uint2(0, 0);
    if (r < R && c < C) codes[j] = __ldcs(reinterpret_cast<const uint2*>(q + r * (C / 2) + c / 2));
  }
  for (int i = tid; i < kPer * 128; i += kFThreads)
    if (tc * kPer + i / 128 < k_tiles)
      reinterpret_cast<uint32_t*>(sc)[i] =
          __ldg(reinterpret_cast<const uint32_t*>(scales) + (row0 / kFTile * k_tiles + tc * kPer) * 128 + i);
  __syncthreads();
  if (c >= C) return;
  const int k = tid % 16 * kFBlock / kBlk;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t r = row0 + tid / 16 + j * (kFThreads / 16);
    if (r >= R) break;
    const uint32_t sb = sc[(k >> 2) * 512 + scale_place((int)(r & 127), k)];
    float s;
    if constexpr (FMT == GS_NVFP4) s = lo_f16(cvt_fp8x2_f16x2<GS_E4M3>((uint16_t)sb));
    else s = sb == 0 ? 0x1p-127f : __uint_as_float(sb == 255u ? 0x7FC00000u : sb << 23);
    float v[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = cvt_e2m1x2_f16x2((e < 4 ? codes[j].x : codes[j].y) >> (8 * (e & 3)) & 0xFFu);
      v[2 * e] = __fmul_rn(lo_f16(h), s);
      v[2 * e + 1] = __fmul_rn(hi_f16(h), s);
      if constexpr (FMT == GS_NVFP4) {
        v[2 * e] = __fmul_rn(v[2 * e], t);
        v[2 * e + 1] = __fmul_rn(v[2 * e + 1], t);
      }
    }
    typename Elem<DT>::type* const to = static_cast<typename Elem<DT>::type*>(y) + r * ldy + c;
    if (align == 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e) to[e] = Elem<DT>::put(v[e]);
      continue;
    }
    constexpr int kWords = DT == GS_F32 ? 16 : 8;
    uint32_t w[kWords];
#pragma unroll
    for (int e = 0; e < kWords; ++e) {
      if constexpr (DT == GS_F32) w[e] = __float_as_uint(v[e]);
      else if constexpr (DT == GS_BF16) w[e] = cvt_f32x2_bf16x2(v[2 * e + 1], v[2 * e]);
      else w[e] = (uint32_t)Elem<DT>::put(v[2 * e]) | (uint32_t)Elem<DT>::put(v[2 * e + 1]) << 16;
    }
    if (align == 32) {
#pragma unroll
      for (int e = 0; e < kWords; e += 8) {
        V8 a;
#pragma unroll
        for (int i = 0; i < 8; ++i) a.w[i] = w[e + i];
        st_stream8(reinterpret_cast<uint32_t*>(to) + e, a);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kWords; e += 4)
        st_stream(reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(to) + e),
                  make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]));
    }
  }
}

template <int DT, int FMT>
static cudaError_t dequant4_t(const uint8_t* q, const uint8_t* scales, const float* ts, int64_t R,
                              int64_t C, void* y, int64_t ldy, cudaStream_t st) {
  const int64_t tiles_c = div_up(C, kDCols);
  const int align = run_align<DT>(y, R == 1 ? C : ldy);
  const int64_t large = div_up(R, kFTile) * tiles_c;
  // from two thirds of the SMs on.  128 and 16 rows, NVFP4 to bf16 on the device:
  // 512 x 4096 (64 CTAs of 128) 3.2 and 2.8 us, 1024 x 4096 (128) 3.2 and 3.7,
  // 640 x 8192 (160) 4.4 and 4.2, 2048 x 8192 (512) 7.1 and 8.9, 28672 x 8192 98 and
  // 130; 333 x 992 to fp32 4.1 and 2.0
  if (3 * large >= 2 * sm_count())
    dequant4_kernel<DT, FMT, kFTile>
        <<<(unsigned)large, kFThreads, 0, st>>>(q, scales, ts, R, C, y, ldy, align, tiles_c);
  else
    dequant4_kernel<DT, FMT, 16><<<(unsigned)(div_up(R, 16) * tiles_c), kFThreads, 0, st>>>(
        q, scales, ts, R, C, y, ldy, align, tiles_c);
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

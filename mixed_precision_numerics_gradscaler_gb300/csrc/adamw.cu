// adamw.cu -- the AdamW step over a list of parameters, moments in fp32 or in
// E4M3 with one scale per 128 elements ("Numerical Precision, Mixed Precision,
// and Loss Scaling", six-step training step, step 5: clip and update -- write
// into FP32 master state, and skip invalid steps).
//
//   m = b1 m + (1 - b1) g,  v = b2 v + ((1 - b2) g) g,  r = sqrt(v)
//   w = w (1 - lr wd) - (lr / (1 - b1^t)) m / (r / sqrt(1 - b2^t) + eps)
// The moments' operations are rounded one by one, so that a state is a pure
// function of the inputs that the oracle restates bit for bit; the weight's
// last division is an approximate one (2 ulp of the update, far below an ulp
// of the weight).
//
// 8-bit moments.  A block's scale is a / 448 with a its largest magnitude;
// x * (448 / a) is rounded to E4M3 at random: 16 random bits are added below
// the three kept significand bits and the carry decides.  Nearest rounding
// would lose the second moment: with b2 = 0.999 a step moves it by a
// thousandth of its distance, E4M3's steps are 1/16 to 1/8 apart.  The root
// of v is stored, not v: E4M3 spans 2^18 between its largest and smallest
// values, which is 2^36 in v.  A positive root is kept at the smallest code
// at least: a zero would turn the next update into a division by eps.
// The rounded root has the root's mean, so its square, the next step's v, gains
// the rounding's variance: under Gaussian gradients v settles above the fp32 one,
// by 2 % with b2 = 0.95, 4 % with 0.99, 5 % with 0.999, and updates are half as
// much smaller.
//
// fp32 moments: HBM-bound, 567 M parameters with fp32 gradients and a bf16 copy in
// 2485 us, 6.85 TB/s of their 30 bytes each.  8-bit moments: some 80 instructions
// per element beside 18 bytes, both near their limits: 1595 us, 6.45 TB/s.  Short
// lists (1 M parameters: 5.9 and 7.6 us from a graph) are the launch and one pass's latency.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gs_elem.cuh"
#include "gs_internal.h"
#include "gs_quant.cuh"

namespace gs {

constexpr int kAdamThreads = 256;

// The smallest magnitude a block's scale is formed from: 448 / a stays
// finite.
constexpr float kMomentFloor = 1e-30f;

// 32 well-mixed bits of x: two rounds of xor-shift and multiply (multipliers
// from C. Wellons' 2018 search for low-bias mixers).
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// The E4M3 code (without sign) of t >= 0 rounded up or down, up with
// probability equal to the fraction of the way (r16: 16 random bits): they are
// added below the three kept significand bits and the rest cut off.  Below
// 2^-6 E4M3's step stays 2^-9; adding 2^-6 moves the value into the binade
// with that step.  Codes count steps, so they are the fp32 word's upper twelve
// bits less the exponents' difference; 126 is 448.
__device__ __forceinline__ uint32_t round_e4m3_random(float t, uint32_t r16) {
  const bool low = t < 0.015625f;
  const uint32_t b = __float_as_uint(low ? t + 0.015625f : t) + (r16 << 4);
  const int c = (int)(b >> 20) - (low ? 968 : 960);
  return (uint32_t)(c < 126 ? c : 126);
}

__device__ __forceinline__ float decode_e4m3(uint8_t q) {
  return lo_f16(cvt_fp8x2_f16x2<GS_E4M3>(q));
}

struct AdamWStep {
  // gradient factor; lr / (1 - b1^t) and 1 / sqrt(1 - b2^t), both times eps_shift
  float coef, c1, c2;
  uint32_t key;        // of the random bits, without the place's high word
  bool skip;           // the step is not taken: nothing is written
};

// The step's factors, by the CTA's first thread for all of them (the
// exponentials are a few hundred instructions).  1 - b^t = -expm1(t log b);
// b = 0 gives 1.
__device__ __forceinline__ AdamWStep step_of(const AdamWArgs& a) {
  __shared__ AdamWStep shared;
  if (threadIdx.x == 0) {
    AdamWStep s;
    const int64_t t = *a.step + 1;
    const float nrm = a.max_norm > 0.0f ? *a.grad_norm : 0.0f;
    s.skip = *a.found_inf != 0;
    s.coef = a.max_norm > 0.0f && nrm > a.max_norm ? __fdiv_rn(a.max_norm, nrm) : 1.0f;
    s.c1 = a.eps_shift * __fdiv_rn(a.lr, -expm1f((float)t * a.log_beta1));
    s.c2 = a.eps_shift * __fdiv_rn(1.0f, __fsqrt_rn(-expm1f((float)t * a.log_beta2)));
    s.key = a.seed + 0x9E3779B9u * (uint32_t)t;
    shared = s;
  }
  __syncthreads();
  return shared;
}

// The last CTA to have read the step's number counts it.  Each arrives, its read
// released, after the barrier behind the read, and asks which it was only at its
// end, so that no chunk waits for the answer (a microsecond of a short list's 8).
__device__ __forceinline__ uint32_t arrive(const AdamWArgs& a) {
  uint32_t before = 0;
  if (threadIdx.x == 0)
    asm volatile("atom.release.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(a.arrived)
                 : "memory");
  return before;
}
__device__ __forceinline__ void count_step(const AdamWArgs& a, uint32_t before) {
  if (threadIdx.x == 0 && before == gridDim.x - 1) {
    __threadfence();  // every CTA's read comes before the write
    *a.arrived = 0;
    *a.step += 1;
  }
}

// n / d, off by 2 ulp at most, where d and 1 / d are normal numbers (or d is 0:
// NaN or Inf).  Here d = r c2 + eps: a root is 0 or at least 2^-75, and r c2 at
// most 2^76 (both times eps_shift); eps by itself is brought into range by the
// factor eps_shift of numerator and divisor.
__device__ __forceinline__ float quotient(float n, float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return n * r;
}

// sqrt(v) rounded to nearest for v in [2^-96, 2^96], two at once: s = v y and
// h = y / 2 with y near 1 / sqrt(v), then s + h (v - s^2), the residual exact by
// a fused multiply-add (Markstein, "IA-64 and Elementary Functions", 2000,
// chapter 9: one such step from an estimate within an ulp rounds correctly
// but where y is too coarse; a test compares it with the IEEE root at every
// significand of two binades, at the middle and at both ends of the range).
__device__ __forceinline__ uint64_t sqrt_f32x2(uint64_t v) {
  float v0, v1, y0, y1;
  upk_f32x2(v, v0, v1);
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(v0));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(v1));
  const uint64_t y = pk_f32x2(y0, y1), s = mul_f32x2(v, y);
  const uint64_t e = fma_f32x2(s ^ 0x8000000080000000ull, s, v);
  return fma_f32x2(e, mul_f32x2(y, pk_f32x2(0.5f, 0.5f)), s);
}
// The roots of any two, rounded to nearest.
__device__ __forceinline__ void roots2(uint64_t v, float* r) {
  float v0, v1;
  upk_f32x2(v, v0, v1);
  if (fminf(v0, v1) >= 0x1p-96f && fmaxf(v0, v1) <= 0x1p96f) {
    upk_f32x2(sqrt_f32x2(v), r[0], r[1]);
  } else {
    r[0] = __fsqrt_rn(v0);
    r[1] = __fsqrt_rn(v1);
  }
}

// One element's new moments and weight.
struct Adam1 {
  float m, v, r, w;
};
__device__ __forceinline__ Adam1 adam1(const AdamWArgs& a, const AdamWStep& s, float keep, float w,
                                       float g, float m, float v) {
  g = __fmul_rn(g, s.coef);
  Adam1 o;
  o.m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_beta1));
  o.v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, a.one_beta2), g));
  o.r = __fsqrt_rn(o.v);
  o.w = __fsub_rn(__fmul_rn(w, keep),
                  quotient(__fmul_rn(o.m, s.c1), __fmaf_rn(o.r, s.c2, a.eps)));
  return o;
}

// Eight gradients, 16 bytes at a time.
template <int GT>
__device__ __forceinline__ void load_grads8(const void* g, int64_t i, float* f) {
  if constexpr (GT == GS_F32) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const uint4 w = ld_stream(reinterpret_cast<const uint4*>(static_cast<const float*>(g) + i + j));
      f[j] = __uint_as_float(w.x);
      f[j + 1] = __uint_as_float(w.y);
      f[j + 2] = __uint_as_float(w.z);
      f[j + 3] = __uint_as_float(w.w);
    }
  } else {
    using Tag = std::conditional_t<GT == GS_BF16, BF16Tag, F16Tag>;
    const uint4 w = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + i));
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = lo16<Tag>(q[j]);
      f[2 * j + 1] = hi16<Tag>(q[j]);
    }
  }
}
// State arrays are read and written in place: not through the read-only path.
__device__ __forceinline__ V8 ld_state8(const float* p) {
  V8 a;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.w[0]), "=r"(a.w[1]), "=r"(a.w[2]), "=r"(a.w[3]), "=r"(a.w[4]),
                 "=r"(a.w[5]), "=r"(a.w[6]), "=r"(a.w[7])
               : "l"(p));
  return a;
}
__device__ __forceinline__ float4 ld_state4(const float* p) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ bool aligned_to(const void* p, uint32_t n) {
  return ((uint32_t)(uintptr_t)p & (n - 1)) == 0;
}

// fp32 moments: 4 x 4 bytes read, 3 x 4 and the copy's 2 written per
// parameter; 32-byte accesses where the chunk's arrays allow them.
template <int GT>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_f32_kernel(const AChunk* __restrict__ chunks, int64_t n_chunks, const AdamWArgs a) {
  AChunk ch{};
  if (blockIdx.x < n_chunks) ch = chunks[blockIdx.x];  // on its way while the factors are formed
  const AdamWStep s = step_of(a);
  if (s.skip) return;
  const uint32_t before = arrive(a);
  for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    if (c != blockIdx.x) ch = chunks[c];
    const float keep = __fsub_rn(1.0f, __fmul_rn(a.lr, __fmul_rn(a.weight_decay, ch.decay)));
    float* m = static_cast<float*>(ch.m);
    float* v = static_cast<float*>(ch.v);
    const bool vec = aligned_to(ch.w, 32) && aligned_to(m, 32) && aligned_to(v, 32) &&
                     aligned_to(ch.g, 16) && aligned_to(ch.w_bf16, 16);
    const int n8 = vec ? (int)(ch.n >> 3) : 0;
    for (int i = threadIdx.x; i < n8; i += kAdamThreads) {
      V8 w8 = ld_state8(ch.w + 8 * i), m8 = ld_state8(m + 8 * i), v8 = ld_state8(v + 8 * i);
      float g[8];
      load_grads8<GT>(ch.g, 8 * i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Adam1 o = adam1(a, s, keep, __uint_as_float(w8.w[j]), g[j], __uint_as_float(m8.w[j]),
                              __uint_as_float(v8.w[j]));
        w8.w[j] = __float_as_uint(o.w);
        m8.w[j] = __float_as_uint(o.m);
        v8.w[j] = __float_as_uint(o.v);
      }
      st_stream8(ch.w + 8 * i, w8);
      st_stream8(m + 8 * i, m8);
      st_stream8(v + 8 * i, v8);
      if (ch.w_bf16) {
        const float* f = reinterpret_cast<const float*>(w8.w);
        st_stream(reinterpret_cast<uint4*>(ch.w_bf16 + 8 * i),
                  make_uint4(cvt_f32x2_bf16x2(f[1], f[0]), cvt_f32x2_bf16x2(f[3], f[2]),
                             cvt_f32x2_bf16x2(f[5], f[4]), cvt_f32x2_bf16x2(f[7], f[6])));
      }
    }
    for (int64_t i = n8 * 8 + threadIdx.x; i < ch.n; i += kAdamThreads) {
      const Adam1 o = adam1(a, s, keep, ch.w[i], load1<GT>(ch.g, i), m[i], v[i]);
      m[i] = o.m;
      v[i] = o.v;
      ch.w[i] = o.w;
      if (ch.w_bf16) ch.w_bf16[i] = Elem<GS_BF16>::put(o.w);
    }
  }
  count_step(a, before);
}

// Two elements' new moments and weights: adam1, both at once (f32x2
// operations round each half like the single ones).
__device__ __forceinline__ uint64_t pk1(float f) { return pk_f32x2(f, f); }
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// A product that is rounded by itself: the compiler fuses a packed product
// with the sum it goes into (whatever -fmad and .rn say), but not this one,
// whose addend, -0, changes nothing and is not known to it.
__device__ __forceinline__ uint64_t product_f32x2(const AdamWArgs& a, uint64_t x, uint64_t y) {
  return fma_f32x2(x, y, pk_f32x2(a.minus_zero, a.minus_zero));
}
struct Adam2 {
  float m[2], r[2], w[2];
};
__device__ __forceinline__ Adam2 adam2(const AdamWArgs& a, const AdamWStep& s, float keep,
                                       uint64_t w, uint64_t g, uint64_t m, uint64_t v) {
  g = mul_f32x2(g, pk1(s.coef));
  m = add_f32x2(product_f32x2(a, m, pk1(a.beta1)), product_f32x2(a, g, pk1(a.one_beta1)));
  v = add_f32x2(product_f32x2(a, v, pk1(a.beta2)),
                product_f32x2(a, mul_f32x2(g, pk1(a.one_beta2)), g));
  Adam2 o;
  upk_f32x2(m, o.m[0], o.m[1]);
  roots2(v, o.r);
  const uint64_t num = mul_f32x2(m, pk1(s.c1));
  const uint64_t den = fma_f32x2(pk_f32x2(o.r[0], o.r[1]), pk1(s.c2), pk1(a.eps));
  float n0, n1, d0, d1;
  upk_f32x2(num, n0, n1);
  upk_f32x2(den, d0, d1);
  const uint64_t upd = pk_f32x2(-quotient(n0, d0), -quotient(n1, d1));
  upk_f32x2(fma_f32x2(w, pk1(keep), upd), o.w[0], o.w[1]);
  return o;
}

// 8-bit moments.  A warp takes blocks of 128 two at a time, four consecutive
// elements per lane; the new moments stay in registers until the blocks'
// maxima are known (as integer maxima of the magnitudes' bits: a NaN is above
// everything and makes the scale NaN).
constexpr int kAdamBlocks = 2;

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Four gradients as they are in memory.
template <int GT>
__device__ __forceinline__ void load_raw(const void* g, int64_t i, uint32_t* w) {
  if constexpr (GT == GS_F32) {
    const uint4 v = ld_stream(reinterpret_cast<const uint4*>(static_cast<const float*>(g) + i));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(w[0]), "=r"(w[1])
                 : "l"(static_cast<const uint16_t*>(g) + i));
  }
}
template <int GT>
__device__ __forceinline__ void unpack_raw(const uint32_t* w, float* f) {
  if constexpr (GT == GS_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(w[j]);
  } else {
    using Tag = std::conditional_t<GT == GS_BF16, BF16Tag, F16Tag>;
    f[0] = lo16<Tag>(w[0]);
    f[1] = hi16<Tag>(w[0]);
    f[2] = lo16<Tag>(w[1]);
    f[3] = hi16<Tag>(w[1]);
  }
}
// A lane's part of a block as it is in memory.
template <int GT>
struct RawBlock {
  float4 w;
  uint32_t g[GT == GS_F32 ? 4 : 2];
  uint32_t m, v;
  float sm, sv;
};

// A moment's scale a / 448 and factor 448 / a of up to four maxima (two
// blocks' m and root), lane i of a group of eight dividing for one of the
// eight: four divisions of every lane's own cost more than all else here.
struct BlockScales {
  float scale;  // of this lane: its block's and moment's (lanes 0-3 of eight)
  float inv[2 * kAdamBlocks];
};
__device__ __forceinline__ BlockScales block_scales(const float* mx, int lane) {
  float a[2 * kAdamBlocks];
#pragma unroll
  for (int i = 0; i < 2 * kAdamBlocks; ++i) {
    const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mx[i]));
    const uint32_t least = __float_as_uint(kMomentFloor);
    a[i] = __uint_as_float(bits > least ? bits : least);
  }
  const float x = (lane & 2) ? ((lane & 1) ? a[3] : a[2]) : ((lane & 1) ? a[1] : a[0]);
  const bool inverse = lane & 4;
  BlockScales b;
  b.scale = __fdiv_rn(inverse ? 448.0f : x, inverse ? x : 448.0f);
#pragma unroll
  for (int i = 0; i < 2 * kAdamBlocks; ++i) b.inv[i] = __shfl_sync(0xFFFFFFFFu, b.scale, 4 + i);
  return b;
}

__device__ __forceinline__ uint32_t encode_m(float m, float inv, uint32_t h) {
  const float t = __fmul_rn(m, inv);
  return round_e4m3_random(fabsf(t), h & 0xFFFFu) | ((__float_as_uint(t) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t encode_r(float r, float inv, uint32_t h) {
  const uint32_t q = round_e4m3_random(__fmul_rn(r, inv), h >> 16);
  return q == 0 && r > 0.0f ? 1u : q;
}
__device__ __forceinline__ uint32_t pack4(const uint32_t* q) {
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

template <int GT>
__global__ void __launch_bounds__(kAdamThreads, 4)
    adamw_e4m3_kernel(const AChunk* __restrict__ chunks, int64_t n_chunks, const AdamWArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = kAdamThreads / 32, U = kAdamBlocks;
  AChunk ch{};
  if (blockIdx.x < n_chunks) ch = chunks[blockIdx.x];  // on its way while the factors are formed
  const AdamWStep s = step_of(a);
  if (s.skip) return;
  const uint32_t before = arrive(a);
  for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    if (c != blockIdx.x) ch = chunks[c];
    const float keep = __fsub_rn(1.0f, __fmul_rn(a.lr, __fmul_rn(a.weight_decay, ch.decay)));
    uint8_t* mq = static_cast<uint8_t*>(ch.m);
    uint8_t* vq = static_cast<uint8_t*>(ch.v);
    const bool vec = aligned_to(ch.w, 16) && aligned_to(ch.g, 16) && aligned_to(mq, 4) &&
                     aligned_to(vq, 4) && aligned_to(ch.w_bf16, 8);
    // blocks of the vector path, whole ones in pairs
    const int whole = vec ? (int)(ch.n / kMomentBlock) / U * U : 0;
    // The warp's next blocks are brought to the L2 cache while these are worked
    // on (567 M parameters: 1792 us without, 1590 with; two steps ahead the same,
    // four 1690): lanes 0-3 ask for one array each, where it allows the copy.
    const char* from = static_cast<const char*>(lane == 0   ? static_cast<const void*>(ch.w)
                                                : lane == 1 ? ch.g
                                                : lane == 2 ? ch.m
                                                            : ch.v);
    const uint32_t block_bytes = kMomentBlock * (lane == 0 ? 4 : lane == 1 ? (GT == GS_F32 ? 4 : 2) : 1);
    const bool asks = lane < 4 && aligned_to(from, 16);
    for (int b0 = warp * U; b0 < whole; b0 += kWarps * U) {
      const int b1 = b0 + kWarps * U;
      if (asks && b1 < whole)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                         from + (int64_t)b1 * block_bytes),
                     "r"(U * block_bytes)
                     : "memory");
      RawBlock<GT> now[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (b0 + u) * kMomentBlock + lane * 4;
        now[u].w = ld_state4(ch.w + i);
        load_raw<GT>(ch.g, i, now[u].g);
        now[u].m = *reinterpret_cast<const uint32_t*>(mq + i);
        now[u].v = *reinterpret_cast<const uint32_t*>(vq + i);
        now[u].sm = ch.m_scale[b0 + u];
        now[u].sv = ch.v_scale[b0 + u];
      }
      float m[U][4], r[U][4], mx[2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (b0 + u) * kMomentBlock + lane * 4;
        const float wf[4] = {now[u].w.x, now[u].w.y, now[u].w.z, now[u].w.w};
        float g[4];
        unpack_raw<GT>(now[u].g, g);
        float nw[4];
        mx[2 * u] = mx[2 * u + 1] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint32_t hm = cvt_fp8x2_f16x2<GS_E4M3>((uint16_t)(now[u].m >> (8 * j)));
          const uint32_t hv = cvt_fp8x2_f16x2<GS_E4M3>((uint16_t)(now[u].v >> (8 * j)));
          const uint64_t m2 = mul_f32x2(pk_f32x2(lo_f16(hm), hi_f16(hm)), pk1(now[u].sm));
          const uint64_t r2 = mul_f32x2(pk_f32x2(lo_f16(hv), hi_f16(hv)), pk1(now[u].sv));
          const Adam2 o = adam2(a, s, keep, pk_f32x2(wf[j], wf[j + 1]),
                                pk_f32x2(g[j], g[j + 1]), m2, mul_f32x2(r2, r2));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            nw[j + k] = o.w[k];
            m[u][j + k] = o.m[k];
            r[u][j + k] = o.r[k];
            mx[2 * u] = max_nan(mx[2 * u], fabsf(o.m[k]));
            mx[2 * u + 1] = max_nan(mx[2 * u + 1], o.r[k]);
          }
        }
        *reinterpret_cast<float4*>(ch.w + i) = make_float4(nw[0], nw[1], nw[2], nw[3]);
        if (ch.w_bf16)
          st_stream(reinterpret_cast<uint2*>(ch.w_bf16 + i),
                    make_uint2(cvt_f32x2_bf16x2(nw[1], nw[0]), cvt_f32x2_bf16x2(nw[3], nw[2])));
      }
      const BlockScales b = block_scales(mx, lane);
      if (lane < 2 * U)
        ((lane & 1) ? ch.v_scale : ch.m_scale)[b0 + (lane >> 1)] = b.scale;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (b0 + u) * kMomentBlock + lane * 4;
        const int64_t place = ch.place + (int64_t)(b0 + u) * kMomentBlock;  // one high word
        const uint32_t key = mix32(s.key + 0x85EBCA6Bu * (uint32_t)(place >> 32));
        uint32_t qm[4], qr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (place is a multiple of 128: the sum of place and j is their xor)
          const uint32_t h = mix32(((uint32_t)place + lane * 4) ^ key ^ (uint32_t)j);
          qm[j] = encode_m(m[u][j], b.inv[2 * u], h);
          qr[j] = encode_r(r[u][j], b.inv[2 * u + 1], h);
        }
        *reinterpret_cast<uint32_t*>(mq + i) = pack4(qm);
        *reinterpret_cast<uint32_t*>(vq + i) = pack4(qr);
      }
    }
    // a tensor's last blocks, and chunks off alignment: one block at a time
    for (int b0 = whole + warp; (int64_t)b0 * kMomentBlock < ch.n; b0 += kWarps) {
      const float sm = ch.m_scale[b0], sv = ch.v_scale[b0];
      const int64_t place = ch.place + (int64_t)b0 * kMomentBlock;
      const uint32_t key = mix32(s.key + 0x85EBCA6Bu * (uint32_t)(place >> 32));
      Adam1 o[4];
      float mx[2 * U] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = (int64_t)b0 * kMomentBlock + j * 32 + lane;
        if (i >= ch.n) continue;
        const float rv = __fmul_rn(decode_e4m3(vq[i]), sv);
        o[j] = adam1(a, s, keep, ch.w[i], load1<GT>(ch.g, i), __fmul_rn(decode_e4m3(mq[i]), sm),
                     __fmul_rn(rv, rv));
        ch.w[i] = o[j].w;
        if (ch.w_bf16) ch.w_bf16[i] = Elem<GS_BF16>::put(o[j].w);
        mx[0] = max_nan(mx[0], fabsf(o[j].m));
        mx[1] = max_nan(mx[1], o[j].r);
      }
      const BlockScales b = block_scales(mx, lane);
      if (lane < 2) ((lane & 1) ? ch.v_scale : ch.m_scale)[b0] = b.scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = (int64_t)b0 * kMomentBlock + j * 32 + lane;
        if (i >= ch.n) continue;
        const uint32_t h = mix32((uint32_t)(place + j * 32 + lane) ^ key);
        mq[i] = (uint8_t)encode_m(o[j].m, b.inv[0], h);
        vq[i] = (uint8_t)encode_r(o[j].r, b.inv[1], h);
      }
    }
  }
  count_step(a, before);
}

cudaError_t launch_master_update_adamw(const AChunk* d_chunks, int64_t n_chunks, int grad_dtype,
                                       int moments, const AdamWArgs& args, cudaStream_t stream) {
  int64_t grid = (int64_t)sm_count() * 64;
  if (grid > n_chunks) grid = n_chunks;
  if (grid < 1) grid = 1;
#define GS_F(K)                                                                             \
  if (grad_dtype == GS_F32)                                                                 \
    K<GS_F32><<<(unsigned)grid, kAdamThreads, 0, stream>>>(d_chunks, n_chunks, args);       \
  else if (grad_dtype == GS_F16)                                                            \
    K<GS_F16><<<(unsigned)grid, kAdamThreads, 0, stream>>>(d_chunks, n_chunks, args);       \
  else                                                                                      \
    K<GS_BF16><<<(unsigned)grid, kAdamThreads, 0, stream>>>(d_chunks, n_chunks, args);
  if (moments == GS_MOMENTS_F32) {
    GS_F(adamw_f32_kernel)
  } else {
    GS_F(adamw_e4m3_kernel)
  }
#undef GS_F
  return cudaGetLastError();
}

// The step's roots by themselves, for a test (n even).
__global__ void __launch_bounds__(kAdamThreads)
    adamw_root_kernel(const float* __restrict__ v, float* __restrict__ r, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * kAdamThreads * 2;
  for (int64_t i = ((int64_t)blockIdx.x * kAdamThreads + threadIdx.x) * 2; i < n; i += step)
    roots2(pk_f32x2(v[i], v[i + 1]), r + i);
}
cudaError_t launch_adamw_root(const float* v, float* r, int64_t n, cudaStream_t stream) {
  const int64_t ctas = (n / 2 + kAdamThreads - 1) / kAdamThreads, most = (int64_t)sm_count() * 8;
  adamw_root_kernel<<<(unsigned)(ctas < most ? ctas : most), kAdamThreads, 0, stream>>>(v, r, n);
  return cudaGetLastError();
}

}  // namespace gs

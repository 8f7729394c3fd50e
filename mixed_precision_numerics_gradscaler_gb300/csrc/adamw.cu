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
#include <cuda_runtime.h>
#include <stdint.h>

#include "gs_elem.cuh"
#include "gs_internal.h"

namespace gs {

constexpr int kAdamThreads = 256;

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

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

// |t| rounded up or down to a multiple of E4M3's step at |t|, up with
// probability equal to the fraction (r16: 16 random bits): the bits are
// added below the three kept significand bits and the rest cut off.  Below
// 2^-6 E4M3's step stays 2^-9; adding 2^-6 moves the value into the binade
// with that step.
__device__ __forceinline__ float round_e4m3_random(float t, uint32_t r16) {
  const float a = fabsf(t);
  const bool low = a < 0.015625f;
  const uint32_t b = __float_as_uint(low ? a + 0.015625f : a) + (r16 << 4);
  const float c = __uint_as_float(b & 0xFFF00000u);
  return copysignf(fminf(low ? c - 0.015625f : c, 448.0f), t);
}

__device__ __forceinline__ float decode_e4m3(uint8_t q) {
  return lo_f16(cvt_fp8x2_f16x2<GS_E4M3>(q));
}
__device__ __forceinline__ uint8_t encode_e4m3(float f) {
  return (uint8_t)cvt_f32x2_fp8x2<GS_E4M3>(0.0f, f);
}

struct AdamWStep {
  float coef, c1, c2;  // gradient factor; lr / (1 - b1^t); 1 / sqrt(1 - b2^t)
  uint32_t key;        // of the random bits, without the place's high word
};

// 1 - b^t = -expm1(t log b); b = 0 gives 1.
__device__ __forceinline__ AdamWStep step_of(const AdamWArgs& a) {
  AdamWStep s;
  s.coef = 1.0f;
  if (a.max_norm > 0.0f) {
    const float nrm = *a.grad_norm;
    if (nrm > a.max_norm) s.coef = __fdiv_rn(a.max_norm, nrm);
  }
  const int64_t t = *a.step + 1;
  s.c1 = __fdiv_rn(a.lr, -expm1f((float)t * a.log_beta1));
  s.c2 = __fdiv_rn(1.0f, __fsqrt_rn(-expm1f((float)t * a.log_beta2)));
  s.key = a.seed + 0x9E3779B9u * (uint32_t)t;
  return s;
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
                  __fdividef(__fmul_rn(o.m, s.c1), __fmaf_rn(o.r, s.c2, a.eps)));
  return o;
}

// The last CTA to arrive counts the step: every other one has read it.
__device__ __forceinline__ void count_step(const AdamWArgs& a) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.arrived, 1u) == gridDim.x - 1) {
      *a.arrived = 0;
      *a.step += 1;
    }
  }
}

template <int GT>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_f32_kernel(const AChunk* __restrict__ chunks, int64_t n_chunks, const AdamWArgs a) {
  if (*a.found_inf) return;  // skipped step: leave every state untouched
  const AdamWStep s = step_of(a);
  for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    const AChunk ch = chunks[c];
    const float keep = __fsub_rn(1.0f, __fmul_rn(a.lr, __fmul_rn(a.weight_decay, ch.decay)));
    float* m = static_cast<float*>(ch.m);
    float* v = static_cast<float*>(ch.v);
    for (int64_t i = threadIdx.x; i < ch.n; i += kAdamThreads) {
      const Adam1 o = adam1(a, s, keep, ch.w[i], load1<GT>(ch.g, i), m[i], v[i]);
      m[i] = o.m;
      v[i] = o.v;
      ch.w[i] = o.w;
      if (ch.w_bf16) ch.w_bf16[i] = Elem<GS_BF16>::put(o.w);
    }
  }
  count_step(a);
}

template <int GT>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_e4m3_kernel(const AChunk* __restrict__ chunks, int64_t n_chunks, const AdamWArgs a) {
  if (*a.found_inf) return;
  const AdamWStep s = step_of(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
    const AChunk ch = chunks[c];
    const float keep = __fsub_rn(1.0f, __fmul_rn(a.lr, __fmul_rn(a.weight_decay, ch.decay)));
    uint8_t* mq = static_cast<uint8_t*>(ch.m);
    uint8_t* vq = static_cast<uint8_t*>(ch.v);
    // one warp per block of 128, four elements per lane
    for (int64_t b = warp; b * kMomentBlock < ch.n; b += kAdamThreads / 32) {
      const float sm = ch.m_scale[b], sv = ch.v_scale[b];
      const int64_t place = ch.place + b * kMomentBlock;  // one high word per block
      const uint32_t key = mix32(s.key + 0x85EBCA6Bu * (uint32_t)(place >> 32));
      Adam1 o[4];
      float am = 0.0f, ar = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = b * kMomentBlock + j * 32 + lane;
        if (i >= ch.n) continue;
        const float rv = __fmul_rn(decode_e4m3(vq[i]), sv);
        o[j] = adam1(a, s, keep, ch.w[i], load1<GT>(ch.g, i), __fmul_rn(decode_e4m3(mq[i]), sm),
                     __fmul_rn(rv, rv));
        ch.w[i] = o[j].w;
        if (ch.w_bf16) ch.w_bf16[i] = Elem<GS_BF16>::put(o[j].w);
        am = max_nan(am, fabsf(o[j].m));
        ar = max_nan(ar, o[j].r);
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) {
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, k));
        ar = max_nan(ar, __shfl_xor_sync(0xFFFFFFFFu, ar, k));
      }
      am = am < kMomentFloor ? kMomentFloor : am;  // a NaN stays: it makes the scale NaN
      ar = ar < kMomentFloor ? kMomentFloor : ar;
      const float im = __fdiv_rn(448.0f, am), ir = __fdiv_rn(448.0f, ar);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = b * kMomentBlock + j * 32 + lane;
        if (i >= ch.n) continue;
        const uint32_t h = mix32((uint32_t)(ch.place + i) ^ key);
        mq[i] = encode_e4m3(round_e4m3_random(__fmul_rn(o[j].m, im), h & 0xFFFFu));
        uint8_t q = encode_e4m3(round_e4m3_random(__fmul_rn(o[j].r, ir), h >> 16));
        if (q == 0 && o[j].r > 0.0f) q = 1;
        vq[i] = q;
      }
      if (lane == 0) {
        ch.m_scale[b] = __fdiv_rn(am, 448.0f);
        ch.v_scale[b] = __fdiv_rn(ar, 448.0f);
      }
    }
  }
  count_step(a);
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

}  // namespace gs

// token_logprob.cu -- log probabilities of given tokens, entropy and the
// largest alternatives of each row of logits, and their gradient under the
// loss scale ("Loss scaling, FP8, and the failure that never crashes",
// section "Loss scaling, derived from the chain rule you already have": the
// scaled loss's gradient is where S enters the backward pass).
//
//   lse = m + log s,  m = max x,  s = sum e^(x - m)
//   entropy = log s - t / s,  t = sum e^(x - m) (x - m)
//   dlogits = S (dlogprob (1[target] - p) - dentropy p (x - lse + entropy))
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "gs_elem.cuh"
#include "gs_internal.h"

namespace gs {

constexpr int kLossThreads = 256;

// Beyond this |lse| its rounding to fp32 (2^-24 |lse|, the relative error it
// brings to every p) is no longer small beside the rest, and the gradient
// forms the row's sum anew.
constexpr float kLseExact = 256.0f;

// A logit and its index as one number whose unsigned order is the order of
// the alternatives: larger logits first (NaN above all, -0 equal to +0), and
// the lower index first among equals.  0 stands for no element.
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

template <int DT>
__global__ void __launch_bounds__(kLossThreads)
    token_logprob_kernel(const void* logits, int64_t ld, int64_t R, int64_t V,
                         const int64_t* targets, float* logprob, float* lse, float* entropy,
                         int top_k, int32_t* top_ids, float* top_logprob) {
  __shared__ float red[kLossThreads / 32];
  __shared__ unsigned long long best[kLossThreads / 32];
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t o = r * ld;
    float m = -CUDART_INF_F;
    bool nan = false;
    for (int64_t c = threadIdx.x; c < V; c += kLossThreads) {
      const float x = load1<DT>(logits, o + c);
      nan |= x != x;
      m = fmaxf(m, x);
    }
    nan = __syncthreads_or(nan);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < kLossThreads / 32; ++i) m = fmaxf(m, red[i]);
    __syncthreads();
    float s = 0.0f, t = 0.0f;
    if (m > -CUDART_INF_F) {
      for (int64_t c = threadIdx.x; c < V; c += kLossThreads) {
        const float d = load1<DT>(logits, o + c) - m, e = expf(d);
        s += e;
        if (e > 0.0f || d != d) t = __fmaf_rn(e, d, t);
      }
    }
    s = block_sum<kLossThreads>(s, red);
    t = block_sum<kLossThreads>(t, red);
    nan |= m == CUDART_INF_F;
    const bool none = !nan && m == -CUDART_INF_F;
    const float ls = logf(s);
    const float l = nan ? CUDART_NAN_F : none ? m : m + ls;
    if (threadIdx.x == 0) {
      if (lse) lse[r] = l;
      if (entropy) entropy[r] = nan ? CUDART_NAN_F : none ? 0.0f : ls - t / s;
      if (logprob) {
        const int64_t a = targets[r];
        float p = 0.0f;
        if (a >= V) p = CUDART_NAN_F;
        else if (a >= 0) p = nan ? CUDART_NAN_F : none ? m : (load1<DT>(logits, o + a) - m) - ls;
        logprob[r] = p;
      }
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < top_k; ++k) {  // the largest pair below the last one
      uint64_t b = 0;
      for (int64_t c = threadIdx.x; c < V; c += kLossThreads) {
        const uint64_t q = order_pair(load1<DT>(logits, o + c), (uint32_t)c);
        if (q < last && q > b) b = q;
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) {
        const uint64_t q = __shfl_xor_sync(0xFFFFFFFFu, b, i);
        b = q > b ? q : b;
      }
      if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = b;
      __syncthreads();
      for (int i = 0; i < kLossThreads / 32; ++i) b = best[i] > b ? best[i] : b;
      __syncthreads();
      last = b;
      if (threadIdx.x == 0) {
        const float x = key_value((uint32_t)(b >> 32));
        top_ids[r * top_k + k] = (int32_t)(0xFFFFFFFFu - (uint32_t)b);
        top_logprob[r * top_k + k] = nan ? CUDART_NAN_F : none ? m : (x - m) - ls;
      }
    }
  }
}

template <int DT, int OT>
__global__ void __launch_bounds__(kLossThreads)
    token_logprob_bwd_kernel(const void* logits, int64_t ld, int64_t V, const int64_t* targets,
                             const float* lse, const float* dlogprob, const float* entropy,
                             const float* dentropy, const float* loss_scale, void* dlogits,
                             int64_t ld_out) {
  __shared__ float red[kLossThreads / 32];
  const float S = loss_scale ? *loss_scale : 1.0f;
  const int64_t r = blockIdx.x;
  const float l = lse[r];
  const int64_t a = targets[r];
  const bool none = l == -CUDART_INF_F;
  float gl = a < 0 ? 0.0f : dlogprob[r];
  if (a >= V) gl = CUDART_NAN_F;
  float ls = 0.0f;  // log of the row's sum of exp(x - lse), where lse's rounding shows
  if (fabsf(l) > kLseExact && !none) {
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < V; c += kLossThreads)
      s += expf(load1<DT>(logits, r * ld + c) - l);
    ls = logf(block_sum<kLossThreads>(s, red));
  }
  const float ge = dentropy ? dentropy[r] : 0.0f, h = dentropy ? entropy[r] : 0.0f;
  for (int64_t c = threadIdx.x; c < V; c += kLossThreads) {
    float o = 0.0f;
    if (!none || a >= V) {
      const float d = (load1<DT>(logits, r * ld + c) - l) - ls, p = expf(d);
      o = gl * ((c == a ? 1.0f : 0.0f) - p);
      if (p > 0.0f) o -= ge * p * (d + h);
    }
    store1<OT>(dlogits, r * ld_out + c, S * o);
  }
}

cudaError_t launch_token_logprob(const void* logits, int64_t ld, int dtype, int64_t R, int64_t V,
                                 const int64_t* targets, float* logprob, float* lse,
                                 float* entropy, int top_k, int32_t* top_ids, float* top_logprob,
                                 cudaStream_t stream) {
  const int64_t most = (int64_t)sm_count() * 64;
  const unsigned grid = (unsigned)(R < most ? R : most);
#define GS_F(DT)                                                                              \
  token_logprob_kernel<DT><<<grid, kLossThreads, 0, stream>>>(                                \
      logits, ld, R, V, targets, logprob, lse, entropy, top_k, top_ids, top_logprob)
  if (dtype == GS_F32) GS_F(GS_F32);
  else if (dtype == GS_F16) GS_F(GS_F16);
  else GS_F(GS_BF16);
#undef GS_F
  return cudaGetLastError();
}

cudaError_t launch_token_logprob_bwd(const void* logits, int64_t ld, int dtype, int64_t R,
                                     int64_t V, const int64_t* targets, const float* lse,
                                     const float* dlogprob, const float* entropy,
                                     const float* dentropy, const float* loss_scale,
                                     void* dlogits, int64_t ld_out, int out_dtype,
                                     cudaStream_t stream) {
#define GS_F(DT, OT)                                                                      \
  token_logprob_bwd_kernel<DT, OT><<<(unsigned)R, kLossThreads, 0, stream>>>(             \
      logits, ld, V, targets, lse, dlogprob, entropy, dentropy, loss_scale, dlogits, ld_out)
#define GS_G(DT)                                   \
  if (out_dtype == GS_F32) GS_F(DT, GS_F32);       \
  else if (out_dtype == GS_F16) GS_F(DT, GS_F16);  \
  else GS_F(DT, GS_BF16)
  if (dtype == GS_F32) { GS_G(GS_F32); }
  else if (dtype == GS_F16) { GS_G(GS_F16); }
  else { GS_G(GS_BF16); }
#undef GS_G
#undef GS_F
  return cudaGetLastError();
}

}  // namespace gs

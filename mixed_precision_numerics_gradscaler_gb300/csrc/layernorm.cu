// layernorm.cu -- layer norm of rows and its backward pass, statistics and
// sums in fp32 ("Numerical Precision, Mixed Precision, and Loss Scaling",
// paragraph on autocast: normalisations run in fp32).
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y = (x - mean) rstd gamma + beta
//   d = dy gamma,  xhat = (x - mean) rstd
//   dx = rstd (d - sum d / C - xhat (sum d xhat) / C)
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
#include <cuda_runtime.h>
#include <stdint.h>

#include "gs_elem.cuh"
#include "gs_internal.h"

namespace gs {

constexpr int kNormThreads = 256;

template <int DT, int WT>
__global__ void __launch_bounds__(kNormThreads)
    layernorm_fwd_kernel(const void* x, int64_t ldx, int64_t R, int64_t C, const void* gamma,
                         const void* beta, float eps, void* y, int64_t ldy, float* mean,
                         float* rstd) {
  __shared__ float red[kNormThreads / 32];
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t xo = r * ldx, yo = r * ldy;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kNormThreads) s += load1<DT>(x, xo + c);
    const float mu = block_sum<kNormThreads>(s, red) / (float)C;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kNormThreads) {
      const float d = load1<DT>(x, xo + c) - mu;
      s = __fmaf_rn(d, d, s);
    }
    const float rs = 1.0f / sqrtf(block_sum<kNormThreads>(s, red) / (float)C + eps);
    for (int64_t c = threadIdx.x; c < C; c += kNormThreads) {
      const float h = (load1<DT>(x, xo + c) - mu) * rs;
      const float g = gamma ? load1<WT>(gamma, c) : 1.0f;
      const float b = beta ? load1<WT>(beta, c) : 0.0f;
      store1<DT>(y, yo + c, __fmaf_rn(h, g, b));
    }
    if (threadIdx.x == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

template <int DT, int WT>
__global__ void __launch_bounds__(kNormThreads)
    layernorm_dx_kernel(const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t R,
                        int64_t C, const void* gamma, const float* mean, const float* rstd,
                        void* dx, int64_t lddx) {
  __shared__ float red[kNormThreads / 32];
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < C; c += kNormThreads) {
      const float h = (load1<DT>(x, r * ldx + c) - mu) * rs;
      const float d = load1<DT>(dy, r * lddy + c) * (gamma ? load1<WT>(gamma, c) : 1.0f);
      s1 += d;
      s2 = __fmaf_rn(d, h, s2);
    }
    s1 = block_sum<kNormThreads>(s1, red) / (float)C;
    s2 = block_sum<kNormThreads>(s2, red) / (float)C;
    for (int64_t c = threadIdx.x; c < C; c += kNormThreads) {
      const float h = (load1<DT>(x, r * ldx + c) - mu) * rs;
      const float d = load1<DT>(dy, r * lddy + c) * (gamma ? load1<WT>(gamma, c) : 1.0f);
      store1<DT>(dx, r * lddx + c, rs * (d - s1 - h * s2));
    }
  }
}

// Partial sums of dgamma and dbeta: CTA (i, j) adds rows i, i + P, ... of
// columns [256 j, 256 j + 256) and writes row i of ws [2, P, C].
template <int DT>
__global__ void __launch_bounds__(kNormThreads)
    layernorm_dw_kernel(const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t R,
                        int64_t C, const float* mean, const float* rstd, float* ws, int64_t P) {
  const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x, i = blockIdx.y;
  if (c >= C) return;
  float sg = 0.0f, sb = 0.0f;
  for (int64_t r = i; r < R; r += P) {
    const float d = load1<DT>(dy, r * lddy + c);
    sg = __fmaf_rn(d, (load1<DT>(x, r * ldx + c) - mean[r]) * rstd[r], sg);
    sb += d;
  }
  ws[i * C + c] = sg;
  ws[(P + i) * C + c] = sb;
}

template <int OT>
__global__ void __launch_bounds__(kNormThreads)
    layernorm_dw_join_kernel(const float* ws, int64_t P, int64_t C, void* dgamma, void* dbeta) {
  const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= C) return;
  float sg = 0.0f, sb = 0.0f;
  for (int64_t i = 0; i < P; ++i) {
    sg += ws[i * C + c];
    sb += ws[(P + i) * C + c];
  }
  if (dgamma) store1<OT>(dgamma, c, sg);
  if (dbeta) store1<OT>(dbeta, c, sb);
}

int64_t layernorm_partials(int64_t R, int64_t) { return R < 128 ? R : 128; }

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
  const int64_t most = (int64_t)sm_count() * 64;
  const unsigned grid = (unsigned)(R < most ? R : most);
#define GS_F(DT, WT)                                                                           \
  layernorm_fwd_kernel<DT, WT><<<grid, kNormThreads, 0, stream>>>(x, ldx, R, C, gamma, beta,  \
                                                                  eps, y, ldy, mean, rstd);
  GS_NORM_TYPES(dtype, w_dtype, GS_F)
#undef GS_F
  return cudaGetLastError();
}

cudaError_t launch_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                 int dtype, int64_t R, int64_t C, const void* gamma, int w_dtype,
                                 const float* mean, const float* rstd, void* dx, int64_t lddx,
                                 void* dgamma, void* dbeta, int dw_dtype, float* ws,
                                 cudaStream_t stream) {
  const int64_t most = (int64_t)sm_count() * 64;
  if (R > 0) {
    const unsigned grid = (unsigned)(R < most ? R : most);
#define GS_F(DT, WT)                                                                        \
  layernorm_dx_kernel<DT, WT><<<grid, kNormThreads, 0, stream>>>(dy, lddy, x, ldx, R, C,    \
                                                                 gamma, mean, rstd, dx, lddx);
    GS_NORM_TYPES(dtype, w_dtype, GS_F)
#undef GS_F
  }
  if (!dgamma && !dbeta) return cudaGetLastError();
  const int64_t P = layernorm_partials(R, C);
  const unsigned cols = (unsigned)((C + kNormThreads - 1) / kNormThreads);
  if (P > 0) {
    const dim3 grid(cols, (unsigned)P);
    if (dtype == GS_F32)
      layernorm_dw_kernel<GS_F32><<<grid, kNormThreads, 0, stream>>>(dy, lddy, x, ldx, R, C, mean,
                                                                     rstd, ws, P);
    else if (dtype == GS_F16)
      layernorm_dw_kernel<GS_F16><<<grid, kNormThreads, 0, stream>>>(dy, lddy, x, ldx, R, C, mean,
                                                                     rstd, ws, P);
    else
      layernorm_dw_kernel<GS_BF16><<<grid, kNormThreads, 0, stream>>>(dy, lddy, x, ldx, R, C, mean,
                                                                      rstd, ws, P);
  }
  if (dw_dtype == GS_F32)
    layernorm_dw_join_kernel<GS_F32><<<cols, kNormThreads, 0, stream>>>(ws, P, C, dgamma, dbeta);
  else if (dw_dtype == GS_F16)
    layernorm_dw_join_kernel<GS_F16><<<cols, kNormThreads, 0, stream>>>(ws, P, C, dgamma, dbeta);
  else
    layernorm_dw_join_kernel<GS_BF16><<<cols, kNormThreads, 0, stream>>>(ws, P, C, dgamma, dbeta);
  return cudaGetLastError();
}

}  // namespace gs

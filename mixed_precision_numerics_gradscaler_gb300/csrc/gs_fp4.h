// gs_fp4.h -- launchers of the 4-bit tensors' kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gsfp8.h"

namespace gs {

// partials: kMaxAmaxBlocks words when the tensor scale is to be formed and
// written to ts, else null.
cudaError_t launch_quant4(const void* x, int64_t ldx, int dtype, int64_t R, int64_t C, int fmt,
                          uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t, float* ts,
                          uint32_t* partials, cudaStream_t st);
cudaError_t launch_dequant4(const uint8_t* q, const uint8_t* scales, const float* ts, int64_t R,
                            int64_t C, int fmt, int out_dtype, void* y, int64_t ldy,
                            cudaStream_t st);
// ta, tb: device scalars, null for MXFP4.  status: the device status word.
cudaError_t launch_gemm_fp4(const uint8_t* qa, const uint8_t* sa, const float* ta, const uint8_t* qb,
                            const uint8_t* sb, const float* tb, int64_t M, int64_t N, int64_t K,
                            int fmt, int out_dtype, void* d, int64_t ldd, int32_t* status,
                            cudaStream_t st);

}  // namespace gs

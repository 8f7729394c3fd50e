// gs_elem.cuh -- element access by type code for the operators that take
// fp16, bf16 or fp32 tensors, and block-wide reductions.
#pragma once

#include "gs_device.cuh"

namespace gs {

// The stored type of a gs_dtype.
template <int DT>
struct Elem;
template <>
struct Elem<GS_F16> {
  using type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t b) {
    return __half2float(__ushort_as_half(b));
  }
  static __device__ __forceinline__ uint16_t put(float f) {
    return __half_as_ushort(__float2half_rn(f));
  }
};
template <>
struct Elem<GS_BF16> {
  using type = uint16_t;
  static __device__ __forceinline__ float get(uint16_t b) {
    return __uint_as_float((uint32_t)b << 16);
  }
  static __device__ __forceinline__ uint16_t put(float f) {
    return (uint16_t)(cvt_f32x2_bf16x2(0.0f, f) & 0xFFFFu);
  }
};
template <>
struct Elem<GS_F32> {
  using type = float;
  static __device__ __forceinline__ float get(float f) { return f; }
  static __device__ __forceinline__ float put(float f) { return f; }
};

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return Elem<DT>::get(static_cast<const typename Elem<DT>::type*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float f) {
  static_cast<typename Elem<DT>::type*>(p)[i] = Elem<DT>::put(f);
}

// Sum over the block of NT threads, the same value in every thread; `red`
// holds NT / 32 floats of shared memory that no thread still reads.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) s += red[i];
  __syncthreads();
  return s;
}

}  // namespace gs

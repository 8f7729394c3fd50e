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

// ---- thread-block clusters ---------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// Shared memory of another CTA of the cluster, at the address of p in ours.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(d)
      : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ void store_remote_f32(float* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(p, rank)), "f"(v) : "memory");
}

}  // namespace gs

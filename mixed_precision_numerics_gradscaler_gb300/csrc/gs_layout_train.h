// gs_layout_train.h -- the chunk table and arguments of the AdamW step, kept
// apart from gs_layout.h: the recorded DRAM traffic of the unscale kernel holds
// for the sources that it is compiled from, byte for byte.
#pragma once

#include "gs_layout.h"

namespace gs {

// One contiguous run of a parameter tensor for the AdamW step: at most
// kAChunkMost elements, so that an index in it is an int; with 8-bit moments
// beginning at a multiple of kAChunkLeast elements of the tensor, a multiple of two
// blocks of 128 that share a moment's scale.
constexpr int64_t kAChunkLeast = kChunkElems / 4, kAChunkMost = 4 * kChunkElems;
struct AChunk {
  float* w;            // fp32 master weights (updated in place)
  uint16_t* w_bf16;    // bf16 copy, or nullptr
  const void* g;       // gradients
  void* m;             // first moment: fp32, or E4M3 codes
  void* v;             // second moment: fp32, or E4M3 codes of its root
  float* m_scale;      // one per 128 elements of this chunk (8-bit moments)
  float* v_scale;
  int64_t n;
  int64_t place;       // the list's elements before this chunk, every tensor
                       // counted up to a multiple of 128
  float decay;         // the tensor's factor of the weight decay
};
constexpr int kMomentBlock = 128;
static_assert(kAChunkMost <= INT32_MAX / 4 && kAChunkLeast % (2 * kMomentBlock) == 0,
              "the kernels index a chunk by int and take its blocks in pairs");

// Elements of a tensor with fp32 moments before the first one at which w, m
// and v are 32-byte aligned and the gradients (gsz bytes each) and the bf16
// copy 16-byte aligned, or 0 when there is no such element before the end (or
// the tensor starts aligned): a tensor at any place of flat buffers still gets
// full chunks the 32-byte path takes.
__host__ __device__ inline int64_t achunk_head(const float* w, const uint16_t* wb, const void* g,
                                               const void* m, const void* v, int64_t gsz,
                                               int64_t n) {
  const int64_t h = (int64_t)(((32u - ((uint32_t)(uintptr_t)w & 31u)) & 31u) >> 2);
  if (h == 0 || h >= n) return 0;
  const bool ok = (((uintptr_t)m + 4 * h) & 31u) == 0 && (((uintptr_t)v + 4 * h) & 31u) == 0 &&
                  (((uintptr_t)g + gsz * h) & 15u) == 0 &&
                  (!wb || (((uintptr_t)(wb + h)) & 15u) == 0);
  return ok ? h : 0;
}

struct AdamWArgs {
  float lr, beta1, beta2, weight_decay, max_norm;
  float eps;                    // times eps_shift
  float eps_shift;              // power of two, 1 for an eps in [2^-126, 2^126]
  float one_beta1, one_beta2;   // fp32(1 - beta), from double
  float log_beta1, log_beta2;   // fp32(log beta), from double (-Inf for 0)
  const float* grad_norm;
  const int32_t* found_inf;
  int64_t* step;
  uint32_t seed;
  float minus_zero;             // -0, where the compiler must not know it
  unsigned int* arrived;        // the list's arrival count, 0 between calls
};

}  // namespace gs

// gs_api_train.cu -- the C entry points of the training step around the cast
// path (include/gsfp8.h): layer norm, token log probabilities and the AdamW
// step.  Argument validation on the host; nothing is launched unless every
// check passes.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "gs_args.h"
#include "gs_internal.h"
#include "gsfp8.h"
#include "gsfp8_test.h"

struct gs_adamw_list {
  int device;
  int grad_dtype;
  int moments;
  gs::AChunk* d_chunks;
  int64_t n_chunks;
  unsigned int* d_arrived;
};

namespace gs {

static int cuda_fail(cudaError_t e) {
  record_cuda_error(e);
  return GS_ERR_CUDA;
}

// Rows of a matrix in memory: R rows of `row` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t R, row, ld;
  uintptr_t lo() const { return (uintptr_t)p; }
  uintptr_t hi() const { return lo() + (uintptr_t)((R - 1) * ld + row); }
};

// True when two row sets share a byte.  Exact for two sets with the same
// distance of rows (columns side by side in one wider buffer do not
// overlap); otherwise the ranges from first to last byte are compared.
static bool rows_overlap(const Rows& a, const Rows& b) {
  if (a.row == 0 || b.row == 0) return false;
  if (!(a.lo() < b.hi() && b.lo() < a.hi())) return false;
  if (a.ld != b.ld || a.R == 1 || b.R == 1) return true;
  const uintptr_t ld = (uintptr_t)a.ld;
  const uintptr_t off = a.lo() >= b.lo() ? (a.lo() - b.lo()) % ld
                                         : (ld - (b.lo() - a.lo()) % ld) % ld;  // a after b
  return off < (uintptr_t)b.row || off + (uintptr_t)a.row > ld;
}

// R rows of C elements of `esz` bytes, ld apart: every address computable.
static bool rows_ok(int64_t R, int64_t C, int64_t ld, size_t esz) {
  return ld >= C && mul_ok(R, ld) && mul_ok(R * ld, (int64_t)esz);
}

}  // namespace gs

using namespace gs;

extern "C" {

int gs_layernorm_fwd(const void* x, int64_t ldx, int dtype, int64_t R, int64_t C,
                     const void* gamma, const void* beta, int w_dtype, float eps, void* y,
                     int64_t ldy, float* mean, float* rstd, void* stream) {
  if (!valid_dtype(dtype) || !(w_dtype == GS_F32 || w_dtype == dtype)) return GS_ERR_DTYPE;
  const size_t esz = dtype_size(dtype), wsz = dtype_size(w_dtype);
  if (R < 0 || C < 0 || !rows_ok(R, C, ldx, esz) || !rows_ok(R, C, ldy, esz)) return GS_ERR_SHAPE;
  if (!std::isfinite(eps) || eps < 0.0f) return GS_ERR_ARG;
  if (R == 0 || C == 0) return GS_OK;
  if (!x || !y) return GS_ERR_NULL;
  if (!aligned(x, esz) || !aligned(y, esz) || !aligned(gamma, wsz) || !aligned(beta, wsz) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return GS_ERR_ARG;
  for (const void* p : {x, (const void*)y, gamma, beta, (const void*)mean, (const void*)rstd})
    if (p && !device_reachable(p)) return GS_ERR_ARG;
  const int64_t row = C * (int64_t)esz;
  const Rows in[] = {{x, R, row, ldx * (int64_t)esz},
                     {gamma, 1, gamma ? C * (int64_t)wsz : 0, 0},
                     {beta, 1, beta ? C * (int64_t)wsz : 0, 0}};
  const Rows out[] = {{y, R, row, ldy * (int64_t)esz},
                      {mean, 1, mean ? R * 4 : 0, 0},
                      {rstd, 1, rstd ? R * 4 : 0, 0}};
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (rows_overlap(out[i], r)) return GS_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j])) return GS_ERR_ARG;
  }
  const cudaError_t e = launch_layernorm_fwd(x, ldx, dtype, R, C, gamma, beta, w_dtype, eps, y,
                                             ldy, mean, rstd, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

size_t gs_layernorm_ws_bytes(int64_t R, int64_t C) {
  if (R < 0 || C < 0 || !mul_ok(R, C) || !mul_ok(R * C, 4)) return 0;
  return (size_t)(2 * layernorm_partials(R, C) * C) * sizeof(float);
}

int gs_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, int dtype,
                     int64_t R, int64_t C, const void* gamma, int w_dtype, const float* mean,
                     const float* rstd, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                     int dw_dtype, void* ws, void* stream) {
  if (!valid_dtype(dtype) || !(w_dtype == GS_F32 || w_dtype == dtype) || !valid_dtype(dw_dtype))
    return GS_ERR_DTYPE;
  const size_t esz = dtype_size(dtype), wsz = dtype_size(w_dtype), dsz = dtype_size(dw_dtype);
  if (R < 0 || C < 0 || !mul_ok(R, C) || !mul_ok(R * C, 4) || !rows_ok(R, C, lddy, esz) ||
      !rows_ok(R, C, ldx, esz) || !rows_ok(R, C, lddx, esz))
    return GS_ERR_SHAPE;
  if (C == 0) return GS_OK;
  const bool sums = dgamma || dbeta;
  const size_t wsb = gs_layernorm_ws_bytes(R, C);
  if (R > 0 && (!dy || !x || !mean || !rstd || !dx || (sums && !ws))) return GS_ERR_NULL;
  if (!sums) ws = nullptr;
  if (!aligned(dy, esz) || !aligned(x, esz) || !aligned(dx, esz) || !aligned(gamma, wsz) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, dsz) || !aligned(dbeta, dsz) ||
      !aligned(ws, 16))
    return GS_ERR_ARG;
  const bool rows = R > 0;  // without rows only dgamma and dbeta are touched
  for (const void* p : {rows ? dy : nullptr, rows ? x : nullptr, rows ? gamma : nullptr,
                        rows ? (const void*)mean : nullptr, rows ? (const void*)rstd : nullptr,
                        rows ? (const void*)dx : nullptr, (const void*)dgamma,
                        (const void*)dbeta, rows ? (const void*)ws : nullptr})
    if (p && !device_reachable(p)) return GS_ERR_ARG;
  const int64_t row = C * (int64_t)esz, w = C * (int64_t)dsz;
  const int64_t e8 = (int64_t)esz;
  const Rows out[] = {{dgamma, 1, dgamma ? w : 0, 0},
                      {dbeta, 1, dbeta ? w : 0, 0},
                      {dx, rows ? R : 1, rows ? row : 0, lddx * e8},
                      {ws, 1, rows && ws ? (int64_t)wsb : 0, 0}};
  const Rows in[] = {{dy, rows ? R : 1, rows ? row : 0, lddy * e8},
                     {x, rows ? R : 1, rows ? row : 0, ldx * e8},
                     {gamma, 1, rows && gamma ? C * (int64_t)wsz : 0, 0},
                     {mean, 1, rows ? R * 4 : 0, 0},
                     {rstd, 1, rows ? R * 4 : 0, 0}};
  for (int i = 0; i < 4; ++i) {
    for (const Rows& r : in)
      if (rows_overlap(out[i], r)) return GS_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j])) return GS_ERR_ARG;
  }
  const cudaError_t e = launch_layernorm_bwd(dy, lddy, x, ldx, dtype, R, C, gamma, w_dtype, mean,
                                             rstd, dx, lddx, dgamma, dbeta, dw_dtype,
                                             static_cast<float*>(ws),
                                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_token_logprob(const void* logits, int64_t ld, int dtype, int64_t R, int64_t V,
                     const int64_t* targets, float* logprob, float* lse, float* entropy,
                     int32_t top_k, int32_t* top_ids, float* top_logprob, void* stream) {
  if (!valid_dtype(dtype)) return GS_ERR_DTYPE;
  const size_t esz = dtype_size(dtype);
  if (R < 0 || V < 1 || V > INT32_MAX || !rows_ok(R, V, ld, esz)) return GS_ERR_SHAPE;
  if (top_k < 0 || top_k > GS_MAX_TOP || top_k > V || !mul_ok(R, 4 * GS_MAX_TOP))
    return GS_ERR_SHAPE;
  if (R == 0) return GS_OK;
  if (!logits || !targets != !logprob) return GS_ERR_NULL;
  if (top_k > 0 && (!top_ids || !top_logprob)) return GS_ERR_NULL;
  if (top_k == 0) top_ids = nullptr, top_logprob = nullptr;
  if (!aligned(logits, esz) || !aligned(targets, 8) || !aligned(logprob, 4) || !aligned(lse, 4) ||
      !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprob, 4))
    return GS_ERR_ARG;
  for (const void* p : {logits, (const void*)targets, (const void*)logprob, (const void*)lse,
                        (const void*)entropy, (const void*)top_ids, (const void*)top_logprob})
    if (p && !device_reachable(p)) return GS_ERR_ARG;
  const Rows in[] = {{logits, R, V * (int64_t)esz, ld * (int64_t)esz},
                     {targets, 1, targets ? R * 8 : 0, 0}};
  const Rows out[] = {{logprob, 1, logprob ? R * 4 : 0, 0},
                      {lse, 1, lse ? R * 4 : 0, 0},
                      {entropy, 1, entropy ? R * 4 : 0, 0},
                      {top_ids, 1, R * top_k * 4, 0},
                      {top_logprob, 1, R * top_k * 4, 0}};
  for (int i = 0; i < 5; ++i) {
    for (const Rows& r : in)
      if (rows_overlap(out[i], r)) return GS_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j])) return GS_ERR_ARG;
  }
  const cudaError_t e = launch_token_logprob(logits, ld, dtype, R, V, targets, logprob, lse,
                                             entropy, top_k, top_ids, top_logprob,
                                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_token_logprob_bwd(const void* logits, int64_t ld, int dtype, int64_t R, int64_t V,
                         const int64_t* targets, const float* lse, const float* dlogprob,
                         const float* entropy, const float* dentropy, const float* loss_scale,
                         void* dlogits, int64_t ld_out, int out_dtype, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return GS_ERR_DTYPE;
  const size_t esz = dtype_size(dtype), osz = dtype_size(out_dtype);
  if (R < 0 || V < 1 || V > INT32_MAX || !rows_ok(R, V, ld, esz) || !rows_ok(R, V, ld_out, osz))
    return GS_ERR_SHAPE;
  if (R == 0) return GS_OK;
  if (!logits || !targets || !lse || !dlogprob || !dlogits || !entropy != !dentropy)
    return GS_ERR_NULL;
  if (!aligned(logits, esz) || !aligned(targets, 8) || !aligned(lse, 4) ||
      !aligned(dlogprob, 4) || !aligned(entropy, 4) || !aligned(dentropy, 4) ||
      !aligned(loss_scale, 4) || !aligned(dlogits, osz))
    return GS_ERR_ARG;
  for (const void* p : {logits, (const void*)targets, (const void*)lse, (const void*)dlogprob,
                        (const void*)entropy, (const void*)dentropy, (const void*)loss_scale,
                        (const void*)dlogits})
    if (p && !device_reachable(p)) return GS_ERR_ARG;
  const Rows out = {dlogits, R, V * (int64_t)osz, ld_out * (int64_t)osz};
  const bool in_place = dlogits == logits && dtype == out_dtype && ld == ld_out;
  const Rows in[] = {{logits, R, V * (int64_t)esz, ld * (int64_t)esz},
                     {targets, 1, R * 8, 0},
                     {lse, 1, R * 4, 0},
                     {dlogprob, 1, R * 4, 0},
                     {entropy, 1, entropy ? R * 4 : 0, 0},
                     {dentropy, 1, dentropy ? R * 4 : 0, 0},
                     {loss_scale, 1, loss_scale ? 4 : 0, 0}};
  for (const Rows& r : in)
    if (!(in_place && r.p == logits) && rows_overlap(out, r)) return GS_ERR_ARG;
  const cudaError_t e = launch_token_logprob_bwd(logits, ld, dtype, R, V, targets, lse, dlogprob,
                                                 entropy, dentropy, loss_scale, dlogits, ld_out,
                                                 out_dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_adamw_list_create(float* const* master, uint16_t* const* master_bf16,
                         const void* const* grads, int grad_dtype, int moments, void* const* m,
                         void* const* v, float* const* m_scale, float* const* v_scale,
                         const float* decay, const int64_t* numels, int32_t n_tensors,
                         gs_adamw_list** out) {
  if (!out) return GS_ERR_NULL;
  *out = nullptr;
  if (!valid_dtype(grad_dtype) || !(moments == GS_MOMENTS_F32 || moments == GS_MOMENTS_E4M3))
    return GS_ERR_DTYPE;
  const bool e4m3 = moments == GS_MOMENTS_E4M3;
  if (n_tensors < 0) return GS_ERR_SHAPE;
  if (n_tensors > 0 && (!master || !grads || !m || !v || !numels)) return GS_ERR_NULL;
  if (n_tensors > 0 && e4m3 && (!m_scale || !v_scale)) return GS_ERR_NULL;
  if (!e4m3 && (m_scale || v_scale)) return GS_ERR_ARG;
  const int64_t gsz = (int64_t)dtype_size(grad_dtype), msz = e4m3 ? 1 : 4;
  std::vector<AChunk> chunks;
  try {  // nothing may throw across the C ABI (a vector that cannot grow)
    std::vector<Span> written, read;
    const auto range = [](std::vector<Span>& to, const void* p, int64_t bytes) {
      to.push_back(Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes});
    };
    int64_t place = 0, total = 0;
    for (int32_t i = 0; i < n_tensors; ++i)
      if (numels[i] > 0 && numels[i] <= (INT64_MAX >> 4) && total <= (INT64_MAX >> 1))
        total += numels[i];
    // Chunks as large as leave every SM its four CTAs of one, and four times that in
    // large lists, whose CTAs then begin less often (8-bit moments; the quarter,
    // the half and the whole: 1 M parameters 7.5, 8.0 and 10.1 us, 4 M 18.6, 16.6 and
    // 18.3; the whole and fourfold: 350 M 1048 and 1005).
    const int64_t wave = (int64_t)sm_count() * 4;
    const int64_t chunk = total <= wave * kAChunkLeast       ? kAChunkLeast
                          : total <= wave * kChunkElems      ? kChunkElems / 2
                          : total < wave * 16 * kChunkElems ? kChunkElems
                                                            : kAChunkMost;
    for (int32_t i = 0; i < n_tensors; ++i) {
      const int64_t n = numels[i];
      if (n < 0 || n > (INT64_MAX >> 4) || place > (INT64_MAX >> 1) - n) return GS_ERR_SHAPE;
      if (n == 0) continue;
      uint16_t* wb = master_bf16 ? master_bf16[i] : nullptr;
      const float dk = decay ? decay[i] : 1.0f;
      if (!std::isfinite(dk) || dk < 0.0f) return GS_ERR_ARG;
      if (!master[i] || !grads[i] || !m[i] || !v[i]) return GS_ERR_NULL;
      if (e4m3 && (!m_scale[i] || !v_scale[i])) return GS_ERR_NULL;
      if (!aligned(master[i], 4) || !aligned(grads[i], (size_t)gsz) ||
          !aligned(m[i], (size_t)msz) || !aligned(v[i], (size_t)msz) || !aligned(wb, 2))
        return GS_ERR_ARG;
      for (const void* p : {(const void*)master[i], grads[i], (const void*)m[i],
                            (const void*)v[i], (const void*)wb})
        if (p && !device_reachable(p)) return GS_ERR_ARG;
      const int64_t blocks = (n + kMomentBlock - 1) / kMomentBlock;
      if (e4m3) {
        if (!aligned(m_scale[i], 4) || !aligned(v_scale[i], 4)) return GS_ERR_ARG;
        if (!device_reachable(m_scale[i]) || !device_reachable(v_scale[i])) return GS_ERR_ARG;
        range(written, m_scale[i], blocks * 4);
        range(written, v_scale[i], blocks * 4);
      }
      range(written, master[i], n * 4);
      if (wb) range(written, wb, n * 2);
      range(written, m[i], n * msz);
      range(written, v[i], n * msz);
      range(read, grads[i], n * gsz);
      // fp32 moments: a short first chunk up to where the vector path's
      // alignments hold (E4M3 blocks begin with the tensor)
      const int64_t head = e4m3 ? 0 : achunk_head(master[i], wb, grads[i], m[i], v[i], gsz, n);
      for (int64_t off = 0; off < n;) {
        const int64_t b = off / kMomentBlock;
        const int64_t len = off == 0 && head > 0 ? head : std::min(n - off, chunk);
        chunks.push_back(AChunk{master[i] + off, wb ? wb + off : nullptr,
                                static_cast<const char*>(grads[i]) + off * gsz,
                                static_cast<char*>(m[i]) + off * msz,
                                static_cast<char*>(v[i]) + off * msz,
                                e4m3 ? m_scale[i] + b : nullptr, e4m3 ? v_scale[i] + b : nullptr,
                                len, place + off, dk});
        off += len;
      }
      place += blocks * kMomentBlock;
    }
    // everything but the gradients is written: no two ranges may meet
    if (spans_conflict(written.data(), written.size(), read.data(), read.size()))
      return GS_ERR_ARG;
  } catch (...) {
    return GS_ERR_ARG;
  }
  gs_adamw_list* l = new (std::nothrow)
      gs_adamw_list{current_device(), grad_dtype, moments, nullptr, (int64_t)chunks.size(), nullptr};
  if (!l) return GS_ERR_ARG;
  // one allocation: the arrival count (256 bytes), then the chunk table
  const size_t head = 256, bytes = head + chunks.size() * sizeof(AChunk);
  char* d = nullptr;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&d), bytes);
  if (e == cudaSuccess) e = cudaMemsetAsync(d, 0, head, cudaStreamLegacy);
  if (e == cudaSuccess && !chunks.empty())
    e = cudaMemcpyAsync(d + head, chunks.data(), chunks.size() * sizeof(AChunk),
                        cudaMemcpyHostToDevice, cudaStreamLegacy);
  // on the device before the call returns: the step may follow on any stream
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
  if (e != cudaSuccess) {
    if (d) cudaFree(d);
    delete l;
    return cuda_fail(e);
  }
  l->d_arrived = reinterpret_cast<unsigned int*>(d);
  l->d_chunks = reinterpret_cast<AChunk*>(d + head);
  *out = l;
  return GS_OK;
}

int gs_adamw_list_destroy(gs_adamw_list* list) {
  if (!list) return GS_OK;
  const int prev = current_device();
  cudaSetDevice(list->device);
  const cudaError_t e = cudaDeviceSynchronize();
  cudaFree(list->d_arrived);
  cudaSetDevice(prev);
  delete list;
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_master_update_adamw(const gs_adamw_list* list, float lr, float beta1, float beta2,
                           float eps, float weight_decay, float max_norm,
                           const float* grad_norm, const int32_t* found_inf, int64_t* step,
                           uint32_t seed, void* stream) {
  if (!list || !found_inf || !step || (max_norm > 0.0f && !grad_norm)) return GS_ERR_NULL;
  for (const float x : {lr, eps, weight_decay})
    if (!std::isfinite(x) || x < 0.0f) return GS_ERR_ARG;
  for (const float b : {beta1, beta2})
    if (!(b >= 0.0f && b < 1.0f)) return GS_ERR_ARG;
  if (std::isnan(max_norm)) return GS_ERR_ARG;
  if (!aligned(found_inf, 4) || !aligned(step, 8) || !aligned(grad_norm, 4)) return GS_ERR_ARG;
  if (list->device != current_device()) return GS_ERR_ARG;
  for (const void* p : {(const void*)found_inf, (const void*)step,
                        max_norm > 0.0f ? (const void*)grad_norm : nullptr})
    if (p && !device_reachable(p)) return GS_ERR_ARG;
  AdamWArgs a;
  a.lr = lr;
  a.beta1 = beta1;
  a.beta2 = beta2;
  // An eps with no normal reciprocal is brought to one that has: 2^23 times the
  // smallest subnormal is 2^-126, a quarter of the largest number below 2^126.
  a.eps_shift = eps > 0.0f && eps < 0x1p-126f ? 0x1p23f : eps > 0x1p126f ? 0.25f : 1.0f;
  a.eps = eps * a.eps_shift;
  a.weight_decay = weight_decay;
  a.max_norm = max_norm;
  a.one_beta1 = (float)(1.0 - (double)beta1);
  a.one_beta2 = (float)(1.0 - (double)beta2);
  a.log_beta1 = (float)std::log((double)beta1);
  a.log_beta2 = (float)std::log((double)beta2);
  a.grad_norm = grad_norm;
  a.found_inf = found_inf;
  a.step = step;
  a.seed = seed;
  a.minus_zero = -0.0f;
  a.arrived = list->d_arrived;
  const cudaError_t e = launch_master_update_adamw(list->d_chunks, list->n_chunks,
                                                   list->grad_dtype, list->moments, a,
                                                   static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_test_adamw_root(const float* v, float* r, int64_t n, void* stream) {
  if (n < 0 || n % 2 || !mul_ok(n, 4)) return GS_ERR_SHAPE;
  if (n == 0) return GS_OK;
  if (!v || !r) return GS_ERR_NULL;
  if (!aligned(v, 4) || !aligned(r, 4) || !device_reachable(v) || !device_reachable(r) ||
      overlaps(v, (size_t)n * 4, r, (size_t)n * 4))
    return GS_ERR_ARG;
  const cudaError_t e = launch_adamw_root(v, r, n, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

}  // extern "C"

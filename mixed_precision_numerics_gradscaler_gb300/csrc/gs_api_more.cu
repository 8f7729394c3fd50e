// gs_api_more.cu -- the C entry points of the 4-bit tensors, the policy loss and
// the update by orthogonalised momentum (include/gsfp8.h).  Argument validation on the host; nothing is launched
// unless every check passes.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "gs_args.h"
#include "gs_fp4.h"
#include "gs_internal.h"
#include "gs_muon.h"
#include "gs_policy.h"
#include "gsfp8.h"

struct gs_muon_list {
  int device;
  int grad_dtype;
  char* d_memory;   // tables, tensor maps, sums and the products' operands
  gs::MuonTable table;
};

namespace gs {

static int cuda_fail(cudaError_t e) {
  record_cuda_error(e);
  return GS_ERR_CUDA;
}

// The tensor cores add 16 products at a time to an fp32 sum and cut off what it
// does not hold: a sum of n positive products ends up to n / 16 2^-24 below
// itself, half of that in the mean.  The momentum's sides are held to where that
// is two of fp16's roundings (2^24 elements gave a polynomial 8 % off); the 4-bit
// product's to where the bound it states still says something.
constexpr int64_t kMostSum = 1LL << 24, kMostSide = 1LL << 18;

static bool valid_fmt4(int f) { return f == GS_MXFP4 || f == GS_NVFP4; }

// Reachable or absent.
static bool reach(const void* p) { return !p || device_reachable(p); }

// The bytes [p, p + n) as a range; empty for a null p.
static Span span(const void* p, int64_t n) {
  return Span{(uintptr_t)p, (uintptr_t)p + (p ? (uintptr_t)n : 0)};
}

// R rows of C elements of `esz` bytes, ld apart: every address computable.
static bool rows_ok(int64_t R, int64_t C, int64_t ld, size_t esz) {
  return ld >= C && mul_ok(R, ld) && mul_ok(R * ld, (int64_t)esz);
}
static int64_t rows_bytes(int64_t R, int64_t C, int64_t ld, size_t esz) {
  return R == 0 || C == 0 ? 0 : ((R - 1) * ld + C) * (int64_t)esz;
}

// log(v) for v = 1 + x as two fp32 numbers (from fp64: 2^-48 of it).
static Border border(double log_v) {
  Border b;
  b.hi = (float)log_v;
  b.lo = std::isfinite(log_v) ? (float)(log_v - (double)b.hi) : 0.0f;
  return b;
}

}  // namespace gs

using namespace gs;

extern "C" {

size_t fp4_scale_bytes(int64_t R, int64_t C, int fmt) {
  if (!valid_fmt4(fmt) || R < 0 || C < 0) return 0;
  const int64_t a = div_up(R, 128), b = div_up(C, fmt == GS_NVFP4 ? 64 : 128);
  if (!mul_ok(a, b) || !mul_ok(a * b, 512)) return 0;
  return (size_t)(a * b) * 512;
}

int fp4_quant(const void* x, int64_t ldx, int in_dtype, int64_t R, int64_t C, int fmt, uint8_t* q,
              uint8_t* scales, uint8_t* qt, uint8_t* scales_t, float* tensor_scale, void* ws,
              void* stream) {
  if (!valid_dtype(in_dtype) || !valid_fmt4(fmt)) return GS_ERR_DTYPE;
  const size_t esz = dtype_size(in_dtype);
  if (R < 0 || C < 0 || !rows_ok(R, C, ldx, esz) || C % 32 || (qt && R % 32)) return GS_ERR_SHAPE;
  const bool nv = fmt == GS_NVFP4, empty = R == 0 || C == 0;
  if (!empty && !x) return GS_ERR_NULL;
  if (nv && !tensor_scale) return GS_ERR_NULL;
  if (!empty && ((!q && !qt) || !q != !scales || !qt != !scales_t)) return GS_ERR_NULL;
  if (!nv && (tensor_scale || ws)) return GS_ERR_ARG;
  if (!aligned(x, esz) || !aligned(q, 16) || !aligned(scales, 16) || !aligned(qt, 16) ||
      !aligned(scales_t, 16) || !aligned(tensor_scale, 4) || !aligned(ws, 4))
    return GS_ERR_ARG;
  if (!(empty || reach(x)) || !(empty || (reach(q) && reach(scales) && reach(qt) && reach(scales_t))) ||
      !reach(tensor_scale) || !reach(ws))
    return GS_ERR_ARG;
  const int64_t codes = R * C / 2;
  const Span in[] = {span(x, rows_bytes(R, C, ldx, esz)), span(ws ? nullptr : tensor_scale, 4)};
  Span out[] = {span(q, codes),
                span(scales, (int64_t)fp4_scale_bytes(R, C, fmt)),
                span(qt, codes),
                span(scales_t, (int64_t)fp4_scale_bytes(C, R, fmt)),
                span(ws ? tensor_scale : nullptr, 4),
                span(ws, (int64_t)gs_ws_bytes())};
  if (spans_conflict(out, 6, in, 2)) return GS_ERR_ARG;
  const cudaError_t e =
      launch_quant4(x, ldx, in_dtype, R, C, fmt, q, scales, qt, scales_t, tensor_scale,
                    static_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int fp4_dequant(const uint8_t* q, const uint8_t* scales, const float* tensor_scale, int64_t R,
                int64_t C, int fmt, int out_dtype, void* y, int64_t ldy, void* stream) {
  if (!valid_dtype(out_dtype) || !valid_fmt4(fmt)) return GS_ERR_DTYPE;
  const size_t esz = dtype_size(out_dtype);
  if (R < 0 || C < 0 || !rows_ok(R, C, ldy, esz) || C % 32) return GS_ERR_SHAPE;
  if (R == 0 || C == 0) return GS_OK;
  if (!q || !scales || !y || (fmt == GS_NVFP4 && !tensor_scale)) return GS_ERR_NULL;
  if (fmt != GS_NVFP4 && tensor_scale) return GS_ERR_ARG;
  if (!aligned(q, 16) || !aligned(scales, 16) || !aligned(tensor_scale, 4) || !aligned(y, esz))
    return GS_ERR_ARG;
  if (!reach(q) || !reach(scales) || !reach(tensor_scale) || !reach(y)) return GS_ERR_ARG;
  const Span in[] = {span(q, R * C / 2), span(scales, (int64_t)fp4_scale_bytes(R, C, fmt)),
                     span(tensor_scale, 4)};
  Span out[] = {span(y, rows_bytes(R, C, ldy, esz))};
  if (spans_conflict(out, 1, in, 3)) return GS_ERR_ARG;
  const cudaError_t e = launch_dequant4(q, scales, tensor_scale, R, C, fmt, out_dtype, y, ldy,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int fp4_gemm_block_scaled(const uint8_t* qa, const uint8_t* sa, const float* ta, const uint8_t* qb,
                          const uint8_t* sb, const float* tb, int64_t M, int64_t N, int64_t K,
                          int fmt, int out_dtype, void* d, int64_t ldd, void* stream) {
  if (!valid_fmt4(fmt) || !(out_dtype == GS_F32 || out_dtype == GS_BF16)) return GS_ERR_DTYPE;
  const size_t esz = dtype_size(out_dtype);
  if (M < 0 || N < 0 || K < 0 || K % 32 || M >= (1LL << 31) || N >= (1LL << 31) || K > kMostSum ||
      ldd >= (1LL << 36) || !rows_ok(M, N, ldd, esz) || !mul_ok(M, K) || !mul_ok(N, K))
    return GS_ERR_SHAPE;
  if (div_up(M, 128) * div_up(N, 128) >= (1LL << 30)) return GS_ERR_SHAPE;
  if (M == 0 || N == 0) return GS_OK;
  const bool nv = fmt == GS_NVFP4;
  if (!d || (K > 0 && (!qa || !sa || !qb || !sb))) return GS_ERR_NULL;
  if (nv && (!ta || !tb)) return GS_ERR_NULL;
  if (!nv && (ta || tb)) return GS_ERR_ARG;
  if (!aligned(d, esz) || !aligned(qa, 16) || !aligned(sa, 16) || !aligned(qb, 16) || !aligned(sb, 16) ||
      !aligned(ta, 4) || !aligned(tb, 4))
    return GS_ERR_ARG;
  if (!reach(d) || !reach(ta) || !reach(tb)) return GS_ERR_ARG;
  if (K > 0 && (!reach(qa) || !reach(sa) || !reach(qb) || !reach(sb))) return GS_ERR_ARG;
  const Span in[] = {span(qa, M * K / 2), span(sa, (int64_t)fp4_scale_bytes(M, K, fmt)),
                     span(qb, N * K / 2), span(sb, (int64_t)fp4_scale_bytes(N, K, fmt)),
                     span(ta, 4),         span(tb, 4)};
  Span out[] = {span(d, rows_bytes(M, N, ldd, esz))};
  if (spans_conflict(out, 1, in, 6)) return GS_ERR_ARG;
  int32_t* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e == cudaSuccess)
    e = launch_gemm_fp4(qa, sa, ta, qb, sb, tb, M, N, K, fmt, out_dtype, d, ldd, status,
                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

size_t gs_policy_loss_ws_bytes(int64_t T, int64_t S) {
  if (T < 0 || S < 0 || T > (int64_t)1 << 40 || S > (int64_t)1 << 40) return 0;
  return sizeof(PolicyHead) + (size_t)S * 8 + kPolicyCtas * sizeof(PolicyPart) +
         (size_t)policy_mask_words(T) * 4;
}

int gs_policy_loss(const float* logprob, const float* old_logprob, const float* ref_logprob,
                   const float* advantages, int64_t n_advantages, const int64_t* targets, int64_t T,
                   const int64_t* seq_offsets, int64_t S, float clip_low, float clip_high,
                   float dual_clip, float kl_coef, int reduction, const float* dloss, float* loss,
                   float* stats, float* dlogprob, void* ws, void* stream) {
  const size_t wsb = gs_policy_loss_ws_bytes(T, S);
  if (!wsb || S < 1 || (!seq_offsets && S != 1)) return GS_ERR_SHAPE;
  if (n_advantages != T && n_advantages != S && n_advantages != -S) return GS_ERR_SHAPE;
  const bool adv_per_seq = n_advantages != T;
  if (n_advantages < 0) n_advantages = -n_advantages;
  if (reduction != GS_LOSS_TOKEN_MEAN && reduction != GS_LOSS_SEQUENCE_MEAN && reduction != GS_LOSS_SUM)
    return GS_ERR_ARG;
  if (!(clip_low >= 0.0f) || !(clip_high >= 0.0f) || !std::isfinite(kl_coef)) return GS_ERR_ARG;
  if (!(dual_clip == 0.0f || dual_clip >= 1.0f)) return GS_ERR_ARG;
  if (!loss || !ws || (T > 0 && (!logprob || !old_logprob || !advantages))) return GS_ERR_NULL;
  if (T > 0 && kl_coef != 0.0f && !ref_logprob) return GS_ERR_NULL;
  for (const void* p : {(const void*)logprob, (const void*)old_logprob, (const void*)ref_logprob,
                        (const void*)advantages, (const void*)dloss, (const void*)loss,
                        (const void*)stats, (const void*)dlogprob})
    if (!aligned(p, 4)) return GS_ERR_ARG;
  if (!aligned(targets, 8) || !aligned(seq_offsets, 8) || !aligned(ws, 16)) return GS_ERR_ARG;
  if (T > 0 && (!reach(logprob) || !reach(old_logprob) || !reach(ref_logprob) || !reach(advantages) ||
                !reach(targets) || !reach(dlogprob)))
    return GS_ERR_ARG;
  if (!reach(seq_offsets) || !reach(dloss) || !reach(loss) || !reach(stats) || !reach(ws))
    return GS_ERR_ARG;
  const Span in[] = {span(logprob, T * 4),           span(old_logprob, T * 4), span(ref_logprob, T * 4),
                     span(advantages, n_advantages * 4), span(targets, T * 8),
                     span(seq_offsets, (S + 1) * 8), span(dloss, 4)};
  Span out[] = {span(loss, 4), span(stats, 16), span(dlogprob, T * 4), span(ws, (int64_t)wsb)};
  if (spans_conflict(out, 4, in, 7)) return GS_ERR_ARG;
  PolicyArgs a = {};
  a.logprob = logprob;
  a.old = old_logprob;
  a.ref = ref_logprob;
  a.adv = advantages;
  a.targets = targets;
  a.offsets = seq_offsets;
  a.dloss = dloss;
  a.loss = loss;
  a.stats = stats;
  a.grad = dlogprob;
  a.T = T;
  a.S = S;
  a.reduction = reduction;
  a.adv_per_seq = adv_per_seq;
  const double low = 1.0 - (double)clip_low, high = 1.0 + (double)clip_high;
  a.low = border(low > 0.0 ? std::log(low) : -HUGE_VAL);
  a.high = border(std::log(high));
  a.dual = border(dual_clip ? std::log((double)dual_clip) : HUGE_VAL);
  a.factor_low = (float)low;
  a.factor_high = (float)high;
  a.factor_dual = dual_clip;
  a.kl = kl_coef;
  char* p = static_cast<char*>(ws);
  a.head = reinterpret_cast<PolicyHead*>(p);
  a.n = reinterpret_cast<unsigned long long*>(p + sizeof(PolicyHead));
  a.part = reinterpret_cast<PolicyPart*>(p + sizeof(PolicyHead) + S * 8);
  a.mask = reinterpret_cast<unsigned*>(a.part + kPolicyCtas);
  const cudaError_t e = launch_policy_loss(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_muon_list_create(float* const* master, uint16_t* const* master_bf16, const void* const* grads,
                        int grad_dtype, float* const* momentum, const int64_t* rows,
                        const int64_t* cols, int32_t n, gs_muon_list** out) {
  if (!out) return GS_ERR_NULL;
  *out = nullptr;
  if (n < 0) return GS_ERR_SHAPE;
  if (!valid_dtype(grad_dtype)) return GS_ERR_DTYPE;
  if (n > 0 && (!master || !grads || !momentum || !rows || !cols)) return GS_ERR_NULL;
  const size_t gsz = dtype_size(grad_dtype);
  std::vector<MuonMat> mats;
  std::vector<CUtensorMap> maps;
  std::vector<Span> written, read;
  MuonTable t = {};
  size_t bytes = 0;
  const auto take = [&](size_t b) {  // room in the list's memory, 256-byte aligned
    const size_t at = bytes;
    bytes += (b + 255) / 256 * 256;
    return at;
  };
  size_t at_mats, at_maps, at_partials, at_arrived, at_done, at_factor;
  std::vector<size_t> at_x;
  try {
    for (int32_t i = 0; i < n; ++i) {
      const int64_t R = rows[i], C = cols[i];
      if (R < 0 || C < 0 || R > kMostSide || C > kMostSide || R * C >= (1LL << 31)) return GS_ERR_SHAPE;
      if (R == 0 || C == 0) continue;
      uint16_t* wb = master_bf16 ? master_bf16[i] : nullptr;
      if (!master[i] || !grads[i] || !momentum[i]) return GS_ERR_NULL;
      if (!aligned(master[i], 4) || !aligned(wb, 2) || !aligned(grads[i], gsz) || !aligned(momentum[i], 4))
        return GS_ERR_ARG;
      if (!reach(master[i]) || !reach(wb) || !reach(grads[i]) || !reach(momentum[i])) return GS_ERR_ARG;
      written.push_back(span(master[i], R * C * 4));
      written.push_back(span(wb, R * C * 2));
      written.push_back(span(momentum[i], R * C * 4));
      read.push_back(span(grads[i], R * C * (int64_t)gsz));
      MuonMat m = {};
      m.w = master[i];
      m.wb = wb;
      m.g = grads[i];
      m.m = momentum[i];
      m.rows = (int)R;
      m.cols = (int)C;
      m.s = (int)std::min(R, C);
      m.ldx = (int)((C + 7) / 8 * 8);
      m.lds = (m.s + 7) / 8 * 8;
      m.tall = R > C;
      // x begins with elements of 1 / sqrt(R C) and ends with 1 / sqrt(l) in the
      // mean and 1.21 at most; gram begins with a diagonal of 1 / s and ends near 1
      m.sx = std::ldexp(1.0f, (int)std::min<long>(14, std::lround(std::log2(std::sqrt((double)R * C)))));
      m.sa = std::ldexp(1.0f, (int)std::min<long>(14, std::lround(std::log2((double)m.s))));
      mats.push_back(m);
    }
    if (spans_conflict(written.data(), written.size(), read.data(), read.size())) return GS_ERR_ARG;
    // the longest sums first, so that a launch's last tiles are short ones
    std::stable_sort(mats.begin(), mats.end(), [](const MuonMat& x, const MuonMat& y) {
      return std::max(x.rows, x.cols) > std::max(y.rows, y.cols);
    });
    // tiles of 256 x 256, or of 256 x 128 where so few leave pairs of CTAs without
    // any: rounds of tiles times a tile's stages or its store, whichever is longer,
    // and a last store, in units of a stage of the wide ones (a narrow one takes
    // 0.62, for its loads).  Measured, wide and narrow: one matrix of 4096 x 2048
    // 634 and 607 us, one of 2048 x 2048 492 and 413, twelve of 256 x 768 185 and 164,
    // 32 of 512 x 512 377 and 405, two of 14336 x 4096 8020 and 9660.
    double cost[2];
    int64_t tiles[2][2];  // of either width: products of squares, of X
    for (int k = 0; k < 2; ++k) {
      const int64_t w = kMuonTile >> k, pairs = std::max(1, sm_count() / 2);
      double sums[3] = {0, 0, 0};  // stages of G, P and X over all tiles
      tiles[k][0] = tiles[k][1] = 0;
      for (const MuonMat& m : mats) {
        const int64_t ts = div_up(m.s, kMuonTile), syms = (ts * (ts + 1) / 2) << k;
        const int64_t apps = div_up(m.rows, kMuonTile) * div_up(m.cols, w);
        tiles[k][0] += syms;
        tiles[k][1] += apps;
        sums[0] += (double)syms * (double)div_up(std::max(m.rows, m.cols), 64);
        sums[1] += (double)syms * (double)div_up(m.s, 64);
        sums[2] += (double)apps * (double)div_up(m.s, 64) * 1.8;  // twice but in the last of five steps
      }
      cost[k] = 0;
      for (int j = 0; j < 3 && !mats.empty(); ++j) {
        const int64_t n = tiles[k][j == 2];
        const double sum = sums[j] / (double)n * (k ? 0.62 : 1.0), store = k ? 10 : 13;
        cost[k] += (double)div_up(n, pairs) * std::max(sum, store) + store;
      }
    }
    const int half = cost[1] < cost[0];
    t.tile_n = kMuonTile >> half;
    if (2 * tiles[half][0] + tiles[half][1] >= (1LL << 25)) return GS_ERR_SHAPE;  // of 20 steps: an int
    int sym = 0, app = 0;
    for (MuonMat& m : mats) {
      m.first_chunk = t.chunks;
      m.first_sym = sym;
      m.first_app = app;
      t.chunks += div_up((int64_t)m.rows * m.cols, kMuonChunk);
      const int64_t ts = div_up(m.s, kMuonTile);
      m.syms = (int)(ts * (ts + 1) / 2) << half;
      m.apps = (int)(div_up(m.rows, kMuonTile) * div_up(m.cols, t.tile_n));
      sym += m.syms;
      app += m.apps;
    }
    t.n = (int)mats.size();
    t.sym_tiles = sym;
    t.app_tiles = app;
    at_mats = take(mats.size() * sizeof(MuonMat));
    at_maps = take(mats.size() * 2 * kMuonMaps * sizeof(CUtensorMap));
    at_partials = take((size_t)t.chunks * sizeof(double));
    at_arrived = take(mats.size() * sizeof(unsigned));
    at_done = take(mats.size() * sizeof(unsigned));
    at_factor = take(mats.size() * sizeof(float));
    for (const MuonMat& m : mats) {
      const size_t x = (size_t)m.rows * m.ldx * 2, g = (size_t)m.s * m.lds * 2;
      for (const size_t b : {x, x, g, g, x, x}) at_x.push_back(take(b));
    }
    maps.resize(mats.size() * 2 * kMuonMaps);
  } catch (...) {
    return GS_ERR_ARG;
  }
  gs_muon_list* l = new (std::nothrow) gs_muon_list{current_device(), grad_dtype, nullptr, t};
  if (!l) return GS_ERR_ARG;
  if (mats.empty()) {
    *out = l;
    return GS_OK;
  }
  char* d = nullptr;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&d), bytes);
  if (e == cudaSuccess) {
    for (size_t i = 0; i < mats.size() && e == cudaSuccess; ++i) {
      MuonMat& m = mats[i];
      uint16_t* p[kMuonMaps];
      for (int j = 0; j < kMuonMaps; ++j) p[j] = reinterpret_cast<uint16_t*>(d + at_x[kMuonMaps * i + j]);
      m.x[0] = p[0];
      m.x[1] = p[1];
      m.gram = p[2];
      m.poly = p[3];
      m.x_lo[0] = p[4];
      m.x_lo[1] = p[5];
      for (int j = 0; j < 2 * kMuonMaps; ++j) {
        const int k = j % kMuonMaps;
        const bool square = k == 2 || k == 3;
        if (!muon_encode(&maps[2 * kMuonMaps * i + j], p[k], square ? m.s : m.rows, square ? m.s : m.cols,
                         square ? m.lds : m.ldx, j < kMuonMaps ? 64 : 32))
          e = cudaErrorNotSupported;
      }
    }
    MuonTable& lt = l->table;
    lt.mats = reinterpret_cast<const MuonMat*>(d + at_mats);
    lt.maps = reinterpret_cast<const CUtensorMap*>(d + at_maps);
    lt.partials = reinterpret_cast<double*>(d + at_partials);
    lt.arrived = reinterpret_cast<unsigned*>(d + at_arrived);
    lt.done = reinterpret_cast<unsigned*>(d + at_done);
    lt.factor = reinterpret_cast<float*>(d + at_factor);
    // counts start at 0, and so do the paddings of operands' rows, which TMA takes
    // in pieces of 16 bytes (it stores zeros there)
    if (e == cudaSuccess) e = cudaMemsetAsync(d, 0, bytes, cudaStreamLegacy);
    if (e == cudaSuccess)
      e = cudaMemcpyAsync(d + at_mats, mats.data(), mats.size() * sizeof(MuonMat), cudaMemcpyHostToDevice,
                          cudaStreamLegacy);
    if (e == cudaSuccess)
      e = cudaMemcpyAsync(d + at_maps, maps.data(), maps.size() * sizeof(CUtensorMap),
                          cudaMemcpyHostToDevice, cudaStreamLegacy);
    // on the device before the call returns: the step may follow on any stream
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
  }
  if (e != cudaSuccess) {
    if (d) cudaFree(d);
    delete l;
    return cuda_fail(e);
  }
  l->d_memory = d;
  *out = l;
  return GS_OK;
}

int gs_muon_list_destroy(gs_muon_list* list) {
  if (!list) return GS_OK;
  const int prev = current_device();
  cudaSetDevice(list->device);
  const cudaError_t e = cudaDeviceSynchronize();
  if (list->d_memory) cudaFree(list->d_memory);
  cudaSetDevice(prev);
  delete list;
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

int gs_master_update_muon(const gs_muon_list* list, float lr, float mu, float weight_decay,
                          int nesterov, int32_t ns_steps, int scale, float max_norm,
                          const float* grad_norm, const int32_t* found_inf, void* stream) {
  if (!list || !found_inf || (max_norm > 0.0f && !grad_norm)) return GS_ERR_NULL;
  for (const float x : {lr, weight_decay})
    if (!std::isfinite(x) || x < 0.0f) return GS_ERR_ARG;
  if (!(mu >= 0.0f && mu < 1.0f) || std::isnan(max_norm) || ns_steps < 1 || ns_steps > 20)
    return GS_ERR_ARG;
  if (scale != GS_MUON_SCALE_RMS && scale != GS_MUON_SCALE_ASPECT) return GS_ERR_ARG;
  if (!aligned(found_inf, 4) || !aligned(grad_norm, 4)) return GS_ERR_ARG;
  if (list->device != current_device()) return GS_ERR_ARG;
  if (!reach(found_inf) || (max_norm > 0.0f && !reach(grad_norm))) return GS_ERR_ARG;
  int32_t* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return cuda_fail(e);
  const MuonArgs a = {lr,       mu,    weight_decay,     max_norm,  nesterov ? 1 : 0, ns_steps,
                      scale,    list->grad_dtype, grad_norm, found_inf, status,
                      test_stall()};
  e = launch_master_update_muon(list->table, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GS_OK : cuda_fail(e);
}

}  // extern "C"

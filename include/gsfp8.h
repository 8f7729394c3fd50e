/*
 * gsfp8.h -- C ABI of the GB300 (sm_103a) mixed-precision cast-and-scale
 * library: dynamic loss scaling of FP16 gradient lists, FP8 quantisation with
 * fine-grained (1x128 / 128x128 / per-tensor) scaling, 4-bit tensors, and the
 * operators of training steps around them.
 *
 * Sources of the definitions (web pages, cited by title and section):
 *   [P1] "Loss scaling, FP8, and the failure that never crashes"
 *   [P3] "Numerical Precision, Mixed Precision, and Loss Scaling"
 *   [P4] "Why FP8 training is stable"
 *   [P5] "Mixed precision and FP8 training"
 *
 * Conventions shared by every entry point:
 *   - Return value: a gs_status code.  Argument errors are found on the
 *     host before anything is launched; nothing is enqueued when a call
 *     returns anything but GS_OK.  GS_ERR_CUDA means a CUDA call made by the
 *     library failed (see gs_last_cuda_error).  Nothing throws or aborts.
 *   - Streams: `stream` is a cudaStream_t passed as void*; NULL is the
 *     legacy default stream.  Every compute call is asynchronous on that
 *     stream and never synchronises the host.  The handle is passed to CUDA
 *     as given: it must be a live stream of the current context (CUDA has
 *     no safe check for an arbitrary handle; a launch CUDA refuses returns
 *     GS_ERR_CUDA).
 *   - Memory: every data pointer is device memory of the current device
 *     (or managed memory, or mapped host memory whose device address equals
 *     its host address); pointers the device cannot use as given are
 *     rejected with GS_ERR_ARG.  The caller owns all
 *     data buffers.  The library allocates only inside
 *     gs_tensor_list_create, gs_param_list_create, gs_adamw_list_create and
 *     gs_muon_list_create; no compute call allocates.
 *   - Layout: row-major and contiguous; element [r, c] of an R x C array is
 *     at offset r * C + c.  Outputs must not overlap inputs.  Any element-
 *     aligned address is accepted; 16-byte-aligned buffers take the
 *     vectorised paths.
 *   - Device-side waits are bounded: a kernel that gives up on a wait
 *     records GS_ERR_TIMEOUT in a device status word (gs_device_status)
 *     and returns; it never traps.
 */
#ifndef GSFP8_H
#define GSFP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gs_status {
  GS_OK = 0,
  GS_ERR_NULL = 1,    /* a required pointer is NULL                          */
  GS_ERR_SHAPE = 2,   /* sizes negative, not divisible by the block, too big */
  GS_ERR_DTYPE = 3,   /* unsupported element type or FP8 format              */
  GS_ERR_ARG = 4,     /* other invalid argument (pointer not reachable, ...) */
  GS_ERR_CUDA = 5,    /* a CUDA runtime call failed                          */
  GS_ERR_TIMEOUT = 6  /* a bounded device-side wait expired                  */
} gs_status;

typedef enum gs_dtype { GS_F16 = 0, GS_BF16 = 1, GS_F32 = 2 } gs_dtype;

/* OCP FP8 encodings ([P3] paragraph on the FP8 specification; [P4]
 * "Failure 2"): E4M3 -- bias 7, max 448 (S.1111.110), no infinities, one
 * NaN pattern; E5M2 -- bias 15, max 57344 (S.11110.11), IEEE-style Inf/NaN.
 * Casts are round-to-nearest-even and saturating (|v| beyond max and +-Inf
 * give +-max); every NaN is written as 0x7F. */
typedef enum gs_fp8 { GS_E4M3 = 0, GS_E5M2 = 1 } gs_fp8;

/* Human-readable name of a status code (static string, never NULL). */
const char* gs_status_str(int status);

/* The cudaError_t of the most recent GS_ERR_CUDA on the calling thread. */
int gs_last_cuda_error(void);

/* Library version string. */
const char* gs_version(void);

/* ------------------------------------------------------------------------
 * Dynamic loss scaling ([P1] "Loss scaling, derived from the chain rule you
 * already have" and its SimpleGradScaler listing; [P3] GradScaler defaults
 * paragraph and its six-step training step, step 4 "unscale and inspect"
 * and step 6 "adjust the dynamic loss scale").
 * --------------------------------------------------------------------- */

/* Opaque description of one gradient list: for each tensor, its scaled
 * FP16 gradient (input), its FP32 unscaled output and its element count.
 * The handle owns a device-resident table that cuts each tensor into chunks
 * of 8192 elements (after a short head chunk up to its first element where
 * input and output are both 32-byte aligned), built once so that each step
 * walks the whole list in a single grid, plus a device workspace: 256 bytes
 * for the step's epilogue words and one fp64 slot per CTA of the unscale
 * grid for the norm form. */
typedef struct gs_tensor_list gs_tensor_list;

/* Build a list on the current device.
 *   grads[i]  -- device pointer to numels[i] FP16 values (scaled gradients)
 *   outs[i]   -- device pointer to numels[i] FP32 values (written by
 *                gs_unscale_check_update)
 *   numels[i] -- >= 0; n_tensors >= 0 (0 gives an empty list)
 * Allocates device memory, uploads the chunk table and clears the
 * workspace, and returns once both are on the device (it synchronises the
 * legacy default stream), so the first step may follow on any stream.  The
 * pointers are captured: the list stays valid while those buffers live.  On
 * error *out is NULL. */
int gs_tensor_list_create(const void* const* grads, void* const* outs, const int64_t* numels,
                          int32_t n_tensors, gs_tensor_list** out);

/* Free a list (NULL is accepted).  Synchronises the device first, so it
 * must not be called while the list is in use by a capture. */
int gs_tensor_list_destroy(gs_tensor_list* list);

/* Total element count and chunk count of a list (host values). */
int gs_tensor_list_info(const gs_tensor_list* list, int64_t* total_elems, int64_t* n_chunks);

/* One GradScaler step over the whole list, in one kernel launch:
 *   out_i = fp32(g_i) * fp32(1 / S)   for every element of every tensor,
 *           where S is *scale as it was before this call; written on
 *           skipped steps too (the caller skips the optimizer);
 *   found_inf = 1 if any g_i is Inf or NaN (exponent field all ones, tested
 *           on the scaled FP16 input), else 0;
 *   then, on the device, after every element has been checked:
 *     found_inf: S *= backoff_factor, growth_tracker = 0, *skipped += 1;
 *     otherwise: growth_tracker += 1 and, if growth_tracker >=
 *                growth_interval, S *= growth_factor, growth_tracker = 0.
 * scale, growth_tracker, found_inf: device scalars (fp32, int32, int32);
 * skipped: device int64 or NULL.  The host never reads any of them.
 * growth_interval >= 1; factors finite and > 0.  (PyTorch-style defaults:
 * S0 = 65536, growth 2.0, backoff 0.5, interval 2000; a static scale is
 * growth_factor = backoff_factor = 1.)  Calls that use the same list must
 * be ordered on one stream (the list's workspace is reused each call). */
int gs_unscale_check_update(const gs_tensor_list* list, float* scale, int32_t* growth_tracker,
                            int32_t* found_inf, int64_t* skipped, float growth_factor,
                            float backoff_factor, int32_t growth_interval, void* stream);

/* The same step, also returning the global L2 norm of the unscaled
 * gradients (step 5 of [P3]'s training step clips by it):
 *   *grad_norm = sqrt(sum over every element of out_i^2)  (device fp32)
 * computed in the same pass (no extra traffic): fp32 fused multiply-adds
 * within a chunk of at most 32 terms per thread, compensated fp32 sums
 * across chunks, fp64 beyond; the sum of squares has a relative error below
 * 35 * 2^-24 and is bitwise reproducible on one device.  A step with
 * Inf/NaN gives an Inf/NaN norm. */
int gs_unscale_check_update_norm(const gs_tensor_list* list, float* scale, int32_t* growth_tracker,
                                 int32_t* found_inf, int64_t* skipped, float growth_factor,
                                 float backoff_factor, int32_t growth_interval, float* grad_norm,
                                 void* stream);

/* The same step under a loss-scale policy with hysteresis ([P3] DeepSpeed
 * paragraph: loss_scale_window 1000, hysteresis 2, consecutive_hysteresis
 * false, min_loss_scale 1 -- the pages name the settings; this reading is
 * the library's): on an overflow the step is skipped, the window restarts
 * (growth_tracker = 0) and, while *hysteresis_state > 1, one unit of it is
 * spent and S kept; with one unit left, S = max(S * backoff_factor,
 * min_scale).  A clean step advances the window; a full window
 * (growth_tracker reaching `window`) multiplies S by growth_factor and
 * restores *hysteresis_state to `hysteresis`; with consecutive_hysteresis
 * != 0 it is restored after every clean step instead.  hysteresis_state is
 * a device int32 the caller initialises to `hysteresis`.  hysteresis = 1
 * and min_scale = 0 give exactly gs_unscale_check_update. */
int gs_unscale_check_update_hysteresis(const gs_tensor_list* list, float* scale,
                                       int32_t* growth_tracker, int32_t* hysteresis_state,
                                       int32_t* found_inf, int64_t* skipped, float growth_factor,
                                       float backoff_factor, int32_t window, int32_t hysteresis,
                                       int32_t consecutive_hysteresis, float min_scale,
                                       void* stream);

/* ------------------------------------------------------------------------
 * The consumer of the step ([P3] six-step training step, step 5: clip and
 * update -- apply guardrails, write into FP32 master state, and skip
 * invalid steps; [P5] "Range and precision": FP32 master weights converted
 * to bf16 each step for the forward pass).
 * --------------------------------------------------------------------- */

/* Opaque list of parameters: per tensor, its fp32 master weights (updated
 * in place), an optional bf16 copy (master_bf16 NULL or master_bf16[i]
 * NULL: none) and its fp32 gradients (typically the outs of a
 * gs_tensor_list).  Allocates a device chunk table and returns once it is
 * on the device (it synchronises the legacy default stream). */
typedef struct gs_param_list gs_param_list;
int gs_param_list_create(float* const* master, uint16_t* const* master_bf16,
                         const float* const* grads, const int64_t* numels, int32_t n_tensors,
                         gs_param_list** out);
int gs_param_list_destroy(gs_param_list* list);

/* SGD step on every parameter of the list, one launch:
 *   if *found_inf != 0 (device): nothing is written (the skipped step);
 *   coef = max_norm / *grad_norm if max_norm > 0 and *grad_norm > max_norm,
 *          else 1 (fp32 division);
 *   w = w - lr * (coef * g), each product and the difference rounded to
 *       fp32 separately; bf16 copy = w rounded to nearest even.
 * grad_norm: device fp32 (from gs_unscale_check_update_norm); may be NULL
 * when max_norm <= 0 (no clipping).  Stream-ordered after the step that
 * produced found_inf / grad_norm; nothing is read on the host. */
int gs_master_update_sgd(const gs_param_list* list, float lr, float max_norm,
                         const float* grad_norm, const int32_t* found_inf, void* stream);

/* The AdamW form of the consumer step, with the moments in 32 or in 8 bits.
 *
 * Opaque list of parameters for it: per tensor, its fp32 master weights
 * (updated in place), an optional bf16 copy (master_bf16 NULL or
 * master_bf16[i] NULL: none), its gradients (grad_dtype GS_F32, GS_BF16 or
 * GS_F16, unscaled) and its two moments (updated in place; zeros before the
 * first step):
 *   GS_MOMENTS_F32   -- m[i] and v[i] hold numels[i] fp32 values each, the
 *       running means of g and of g^2; the scale arrays are NULL;
 *   GS_MOMENTS_E4M3  -- m[i] and v[i] hold numels[i] E4M3 codes each, with
 *       one fp32 scale per 128 consecutive elements of the tensor
 *       (m_scale[i], v_scale[i]: ceil(numels[i] / 128) values): m = code *
 *       scale, and v holds the square ROOT of the second moment, whose range
 *       in powers of two is half the moment's.  fp8_dequant reads either.
 * decay (n_tensors host floats, or NULL for all 1) multiplies the step's
 * weight decay per tensor (0: a norm or a bias).  Allocates a device chunk
 * table and returns once it is on the device (it synchronises the legacy
 * default stream).  The pointers are captured. */
typedef enum gs_moments { GS_MOMENTS_F32 = 0, GS_MOMENTS_E4M3 = 1 } gs_moments;
typedef struct gs_adamw_list gs_adamw_list;
int gs_adamw_list_create(float* const* master, uint16_t* const* master_bf16,
                         const void* const* grads, int grad_dtype, int moments, void* const* m,
                         void* const* v, float* const* m_scale, float* const* v_scale,
                         const float* decay, const int64_t* numels, int32_t n_tensors,
                         gs_adamw_list** out);
int gs_adamw_list_destroy(gs_adamw_list* list);

/* One AdamW step on every parameter of the list, one launch:
 *   if *found_inf != 0 (device): nothing is written (the skipped step, which
 *   does not count as one);
 *   t = *step + 1 (device int64; written back at the end);
 *   g = coef * g, coef as in gs_master_update_sgd (max_norm, grad_norm);
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + ((1 - beta2) g) g,
 *   r = sqrt(v)        (each product, sum and root rounded to fp32; 1 - beta
 *                       formed in double and rounded once);
 *   w = w (1 - lr weight_decay decay[i])
 *       - lr / (1 - beta1^t) m / (r / sqrt(1 - beta2^t) + eps);
 *   bf16 copy = w rounded to nearest even.
 * With GS_MOMENTS_E4M3 the update uses the new moments before they are
 * rounded; then, for each block of 128, a = max(max |x|, 1e-30), scale =
 * a / 448, and x * (448 / a) is rounded to E4M3 up or down at random in
 * proportion to the distance (so that the mean of many steps keeps what
 * rounding to nearest would always drop: beta2 near 1 moves v by less than
 * half a step of the format); a positive r is never stored as zero.  The mean
 * kept is the root's: its square, the next step's v, is larger by the
 * rounding's variance, which adds up to 2 % (beta2 0.95) to 5 % (0.999) of v.  The
 * random bits are a function of (seed, t, the element's place in the list):
 * the same inputs give the same bits.  Non-finite gradients are for the
 * check before this step to find; here they give non-finite states.
 * beta1, beta2 in [0, 1); lr, weight_decay, eps finite and >= 0.  grad_norm
 * may be NULL when max_norm <= 0.  Calls on one list must be ordered on one
 * stream.  *step counts the calls of one list: a model whose parameters are in
 * several lists (gradients or moments of two types) keeps a counter for each,
 * since one that they shared would advance once per list. */
int gs_master_update_adamw(const gs_adamw_list* list, float lr, float beta1, float beta2,
                           float eps, float weight_decay, float max_norm,
                           const float* grad_norm, const int32_t* found_inf, int64_t* step,
                           uint32_t seed, void* stream);

/* Checkpoint support: the scaler's whole state is {S, growth_tracker}.
 * get: copies the two device scalars to host variables and waits for the
 *      copy on `stream` (this call synchronises that stream).
 * set: writes host values into the device scalars, stream-ordered
 *      (asynchronous; the values are passed by value, no host buffer is
 *      kept). */
int gs_scaler_state_get(const float* scale, const int32_t* growth_tracker, float* h_scale,
                        int32_t* h_growth_tracker, void* stream);
int gs_scaler_state_set(float* scale, int32_t* growth_tracker, float h_scale,
                        int32_t h_growth_tracker, void* stream);

/* Allocation-free form of gs_unscale_check_update.  The pages have no
 * counterpart: this entry point exists for callers that cannot allocate
 * device memory (code running inside an allocator's own callbacks, or in a
 * process whose device memory another runtime has reserved up front), and so
 * cannot call gs_tensor_list_create.
 *   grads / outs / numels / n_tensors -- as for gs_tensor_list_create, given
 *       on every call (nothing is captured); the remaining arguments and the
 *       results are exactly those of gs_unscale_check_update.
 * The chunk table and the epilogue words live in one fixed device array of
 * this library (768 KiB + 256 B per GPU that loads the library, held until
 * the process exits).  Limits: at most 960 tensors and 32768 chunks of 8192
 * elements (268,435,456 elements in total); larger lists return
 * GS_ERR_SHAPE before anything is launched (see gs_noalloc_limits).
 * The call makes no cudaMalloc / cudaFree and allocates nothing; it uses
 * about 62 KB of the calling thread's stack for the tensor table it passes to
 * the GPU.  Its first call in a CUDA context looks up the array's device
 * address there (cudaGetSymbolAddress) and caches it under the context's ID:
 * each device's primary context, the new primary context that follows a
 * cudaDeviceReset, and any context the caller creates has its own copy of the
 * array and makes its own first call.  Make that first call before any
 * stream capture.  Every call in a context shares that context's array, and
 * its contents persist between calls; the call clears what must start at
 * zero itself.  Calls that overlap on the GPU (on different streams, or from
 * different host threads without ordering) race on the array: order them on
 * one stream. */
int gs_unscale_check_update_noalloc(const void* const* grads, void* const* outs,
                                    const int64_t* numels, int32_t n_tensors, float* scale,
                                    int32_t* growth_tracker, int32_t* found_inf, int64_t* skipped,
                                    float growth_factor, float backoff_factor,
                                    int32_t growth_interval, void* stream);

/* The limits of gs_unscale_check_update_noalloc (host values; any pointer
 * may be NULL). */
int gs_noalloc_limits(int32_t* max_tensors, int64_t* max_chunks, int64_t* chunk_elems);

/* ------------------------------------------------------------------------
 * FP8 quantisation with fine-grained scaling ([P5] "FP8 training", the
 * fp8_scaling.py listing: per-block amax, clamp at 1e-12, divide by MAX;
 * quantise x / s with clamp to +-MAX and cast; dequantise by multiplying
 * by s.  [P1] "FP8 needs a finer-grained fix than a single scale factor"
 * and [P4] "The seam": 1x128 tiles for activations, 128x128 blocks for
 * weights.  [P4] "Failure 1": per-tensor current scaling.)
 *
 * For each block B:   amax_B = max |x| over B (a NaN in B makes it NaN)
 *                     s_B    = max(amax_B, 1e-12f) / MAX      (fp32)
 *                     q      = fp8(clamp(x / s_B, -MAX, MAX)) (fp32 x/s,
 *                              round to nearest even)
 * MAX = 448 (E4M3) or 57344 (E5M2).
 * --------------------------------------------------------------------- */

/* Block-scaled quantisation of a row-major [R, C] tensor.
 *   x        -- R*C elements of in_dtype (GS_BF16, GS_F16 or GS_F32)
 *   (block_r, block_c) -- (1, 128): 1x128 tiles along the contiguous
 *               dimension; or (128, 128): square blocks.  R % block_r == 0
 *               and C % block_c == 0, else GS_ERR_SHAPE.
 *   q        -- R*C bytes of FP8 codes (fmt)
 *   scales   -- fp32 [R / block_r, C / block_c], row-major
 * R == 0 or C == 0 is a valid no-op. */
int fp8_quant_block(const void* x, int in_dtype, int64_t R, int64_t C, int32_t block_r,
                    int32_t block_c, int fmt, uint8_t* q, float* scales, void* stream);

/* Bytes of device workspace fp8_quant_tensor needs (independent of n). */
size_t gs_ws_bytes(void);

/* Per-tensor (current) scaling of n elements: one scale for the whole
 * tensor, computed in a first pass over x and used by a second pass, both
 * on the device (the host never reads amax).
 *   scale -- device fp32 [1], written;  ws -- device workspace of at least
 *   gs_ws_bytes() bytes, 4-byte aligned, any contents (fully overwritten).
 * Calls sharing one ws must be ordered on one stream. */
int fp8_quant_tensor(const void* x, int in_dtype, int64_t n, int fmt, uint8_t* q, float* scale,
                     void* ws, void* stream);

/* Per-tensor quantisation with delayed scaling ([P4] "Failure 1": keep a
 * short history of recent max-abs values and derive s from it; [P5] "FP8
 * training" figure: per tensor, delayed, from recent amax).  One pass over
 * x: the scale applied is s = max(max|amax_history|, 1e-12) / MAX (written
 * to *scale_used); q = fp8(clamp(x / s)); then amax(x) is written at
 * amax_history[*history_pos] and *history_pos advances modulo
 * history_len (1..65536).  amax_history (fp32), history_pos (int32) and
 * scale_used are device memory the caller owns and initialises (a zero
 * history gives the floor scale: everything non-tiny saturates on the
 * first step).  ws: >= gs_ws_bytes() bytes of device scratch.  A NaN in the
 * history makes the scale NaN (every code 0x7F) until it leaves the
 * window.  Calls sharing a history or ws must be ordered on one stream. */
int fp8_quant_tensor_delayed(const void* x, int in_dtype, int64_t n, int fmt, uint8_t* q,
                             float* amax_history, int32_t history_len, int32_t* history_pos,
                             float* scale_used, void* ws, void* stream);

/* Dequantise: y = decode(q) * s (fp32 product), stored as fp32 or rounded
 * to nearest-even bfloat16 (out_dtype GS_F32 or GS_BF16).
 * Block shapes: (1, 128) and (128, 128) with scales laid out as written by
 * fp8_quant_block, or (R, C) -- one scale for the whole [R, C] tensor, as
 * written by fp8_quant_tensor (use R = 1, C = n for a flat tensor). */
int fp8_dequant(const uint8_t* q, const float* scales, int64_t R, int64_t C, int32_t block_r,
                int32_t block_c, int fmt, int out_dtype, void* y, void* stream);

/* ------------------------------------------------------------------------
 * MXFP8: one power-of-two scale per 32 consecutive elements ([P5] "FP8
 * training": Blackwell's MX formats keep one scaling factor per 32 elements
 * in hardware).  The pages give only the block size; the scale rule is the
 * OCP Microscaling convention: an E8M0 byte c means 2^(c - 127) (255 is
 * NaN); for each 1x32 block, e = floor(log2(amax)) - emax_elem (8 for E4M3,
 * 15 for E5M2), clamped to [-127, 127], e = -127 for an all-zero block;
 * q = fp8(x * 2^-e), round to nearest even, saturating at +-MAX; a block
 * holding Inf or NaN gets scale 255 and codes 0x7F.
 * --------------------------------------------------------------------- */

/* x: row-major [R, C] of in_dtype (GS_BF16 / GS_F16 / GS_F32), C % 32 == 0
 * (else GS_ERR_SHAPE); q: R*C FP8 codes; scales: R*C/32 E8M0 bytes,
 * row-major [R, C/32].  Buffers 32-byte aligned with 16-bit input take the
 * vectorised path; any element-aligned buffers are accepted. */
int fp8_quant_mx(const void* x, int in_dtype, int64_t R, int64_t C, int fmt, uint8_t* q,
                 uint8_t* scales, void* stream);

/* y = decode(q) * 2^(scale - 127) in fp32, stored as fp32 or rounded to
 * nearest-even bfloat16 (out_dtype GS_F32 / GS_BF16). */
int fp8_dequant_mx(const uint8_t* q, const uint8_t* scales, int64_t R, int64_t C, int fmt,
                   int out_dtype, void* y, void* stream);

/* ------------------------------------------------------------------------
 * The consumer of the block-scaled tiles: an FP8 GEMM whose partial sums are
 * promoted to FP32 every 128 elements of K ([P1] "FP8 needs a
 * finer-grained fix than a single scale factor": the tensor cores'
 * accumulator keeps too few bits, so partial sums move to FP32 registers at
 * intervals; [P5] "FP8 training": promotion every 128 elements, 1x128
 * scales for activations, 128x128 for weights).
 * --------------------------------------------------------------------- */

/* D = A B^T with A = decode(qa) scaled per 1x128 block and B = decode(qb)
 * scaled per 128x128 block:
 *   D[m][n] = sum over kb of sa[m][kb] * sb[n / 128][kb] * P[m][n][kb],
 *   P[m][n][kb] = sum over k in [128 kb, 128 kb + 128) of
 *                 decode(qa[m][k]) * decode(qb[n][k]).
 * P is formed by the tensor cores (fp32 accumulator, order inside a block
 * not specified); the promotion is one fp32 fused multiply-add per block,
 * acc = fma(P, fp32(sa * sb), acc), in increasing kb.
 *   qa: row-major [M, K] codes, sa: row-major [M, K / 128] fp32 (as
 *       fp8_quant_block writes for block (1, 128));
 *   qb: row-major [N, K] codes (the weight stored [out, in]), sb:
 *       row-major [ceil(N / 128), K / 128] fp32 (block (128, 128));
 *   fmt_a, fmt_b: GS_E4M3 or GS_E5M2, the formats of A and of B; they may
 *      differ ([P5] "FP8 training": E4M3 for forward tensors, E5M2 for
 *      gradients, so a backward GEMM multiplies E5M2 by E4M3);
 *   d: row-major [M, N], out_dtype GS_F32 or GS_BF16 (rounded to nearest
 *      even from the fp32 sum).
 * K % 128 == 0, M, N, K < 2^31 and fewer than 2^30 tiles of 128 x 256
 * (else GS_ERR_SHAPE); M and N need not be multiples of 128; K == 0 writes
 * zeros.  qa and qb must be 16-byte
 * aligned (they are read by TMA; else GS_ERR_ARG).  Accuracy against the
 * exact sum: |error| <= (2^-24 * (nkb + 3) + e_blk) * sum over kb of
 * |sa sb| sum over k |a b|, e_blk being the tensor cores' relative
 * accumulation error within one block.  A wait that runs out records
 * GS_ERR_TIMEOUT (gs_device_status) and leaves d unspecified. */
int fp8_gemm_block_scaled(const uint8_t* qa, const float* sa, const uint8_t* qb, const float* sb,
                          int64_t M, int64_t N, int64_t K, int fmt_a, int fmt_b, int out_dtype,
                          void* d, void* stream);

/* ------------------------------------------------------------------------
 * The steps that mixed precision keeps in fp32 around the cast path ([P3]
 * paragraph on autocast: normalisations, softmax and losses run in fp32
 * whatever the tensors' type): layer norm, and the loss from which the
 * scaled gradients start.  16-bit or fp32 tensors in and out, every sum and
 * statistic in fp32.
 * Rows may lie further apart than their length: ld* is the distance of two
 * rows in elements (>= the row's length).  The elements between are not
 * written and change nothing; a load of 16 bytes that begins in one of them
 * and ends in a row may span a few.
 * --------------------------------------------------------------------- */

/* Layer norm of each row of x [R, C]:
 *   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),
 *   y = (x - mean) rstd gamma + beta.
 * dtype: of x and y; w_dtype: of gamma and beta, GS_F32 or dtype (any may be
 * NULL: 1 and 0).  mean, rstd: fp32 [R] for the backward pass, or NULL.
 * R == 0 or C == 0 is a valid no-op. */
int gs_layernorm_fwd(const void* x, int64_t ldx, int dtype, int64_t R, int64_t C,
                     const void* gamma, const void* beta, int w_dtype, float eps, void* y,
                     int64_t ldy, float* mean, float* rstd, void* stream);

/* Bytes of device workspace gs_layernorm_bwd needs for R x C (0 for sizes it
 * refuses). */
size_t gs_layernorm_ws_bytes(int64_t R, int64_t C);

/* Its backward pass, with xhat = (x - mean) rstd and d = dy gamma:
 *   dx = rstd (d - mean over the row of d - xhat * (mean over the row of
 *        d xhat)),   dgamma = sum over rows of dy xhat,
 *   dbeta = sum over rows of dy.
 * dtype: of dy, x and dx; dw_dtype (any of the three): of dgamma and dbeta,
 * which may be NULL (not computed; with both NULL ws may be NULL too).  GS_F16
 * gradients of gamma and beta go into a gs_tensor_list like any other.  The
 * sums over rows are formed in fp32 in an order that depends on the sizes and
 * the device alone.  R == 0 writes zeros to dgamma and dbeta.
 * ws: device workspace of gs_layernorm_ws_bytes(R, C) bytes, 16-byte
 * aligned, any contents; calls sharing one must be ordered on one stream. */
int gs_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, int dtype,
                     int64_t R, int64_t C, const void* gamma, int w_dtype, const float* mean,
                     const float* rstd, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                     int dw_dtype, void* ws, void* stream);

/* Log probabilities of given tokens under the softmax of each row of logits
 * [R, V] (dtype, row distance ld), with lse = log sum exp x:
 *   logprob[r] = x[r, targets[r]] - lse[r]       (fp32 [R]; formed as
 *       (x - max x) - log sum exp(x - max x), so that it keeps its digits
 *       where lse is large)
 *   lse[r]                                       (fp32 [R], or NULL)
 *   entropy[r] = -sum p log p                    (fp32 [R], or NULL)
 *   top_ids, top_logprob [R, top_k]: the top_k largest logits' indices
 *       (int32; equal logits in the order of their indices, lowest first)
 *       and their log probabilities.  top_k 0: none (both NULL);
 *       top_k <= min(V, GS_MAX_TOP).
 * targets: device int64 [R]; a negative target (no loss at this token) gives
 * logprob 0, one >= V gives NaN.  targets and logprob may both be NULL.
 * Logits of -Inf take no part (p = 0); a row of nothing else has lse -Inf,
 * entropy 0 and log probabilities -Inf.  A row with NaN or +Inf has NaN
 * statistics, and NaN counts as the largest logit in top_ids.
 * R == 0 is a valid no-op; V >= 1, V < 2^31. */
#define GS_MAX_TOP 32
int gs_token_logprob(const void* logits, int64_t ld, int dtype, int64_t R, int64_t V,
                     const int64_t* targets, float* logprob, float* lse, float* entropy,
                     int32_t top_k, int32_t* top_ids, float* top_logprob, void* stream);

/* The gradient of sum_r (dlogprob[r] logprob[r] + dentropy[r] entropy[r]),
 * times the loss scale, with respect to the logits:
 *   p = exp(x - lse),
 *   dlogits = S (dlogprob (1[j == target] - p) - dentropy p (x - lse +
 *             entropy)),
 * rounded to out_dtype (any of the three) to nearest even WITHOUT saturation:
 * a value beyond the type's range becomes Inf, which the loss scaler's check
 * then finds.  lse and entropy: as gs_token_logprob wrote them (where |lse| >
 * 256, so that its own rounding would show in p, the row's sum is formed
 * anew: a row whose every logit is the type's lowest value has p = 1 / V; at a
 * price, as each part of such a row reads all of it: 8192 rows of 128256 bf16
 * take 9 times the time of others, in place 1.9 times);
 * dlogprob, dentropy: fp32 [R]; entropy and dentropy may both be NULL; loss_scale:
 * device fp32 scalar S, or NULL for 1.  A negative target contributes no
 * logprob term, one >= V makes its row NaN; a row with lse -Inf has gradient
 * zero.  dlogits may be the logits themselves (same pointer, type and row
 * distance); otherwise they must not overlap. */
int gs_token_logprob_bwd(const void* logits, int64_t ld, int dtype, int64_t R, int64_t V,
                         const int64_t* targets, const float* lse, const float* dlogprob,
                         const float* entropy, const float* dentropy, const float* loss_scale,
                         void* dlogits, int64_t ld_out, int out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * Microscaled 4-bit tensors: e2m1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives), two to a byte (the even element in the low four bits),
 * with one scale per 32 (GS_MXFP4, E8M0) or 16 (GS_NVFP4, E4M3) consecutive
 * elements of a row, NVFP4 with an fp32 scale of the whole tensor besides.
 *   MXFP4: e = floor(log2(amax)) - 2, clamped to [-127, 127], -127 for a block
 *          of zeros; scale byte e + 127; q = e2m1(x * 2^-e).  (OCP
 *          Microscaling, as fp8_quant_mx.)
 *   NVFP4: t = max(amax of the tensor, 1e-12) / 2688;  s = e4m3(amax / (6 t));
 *          q = e2m1(x * (1 / (s t))), 0 where s is 0; every step in fp32.
 * Roundings to nearest even, saturating; a zero keeps its sign.  A block with
 * Inf or NaN gets a scale of NaN (255; 0x7F) and codes 0; Inf or NaN anywhere
 * makes a tensor scale formed here NaN, and with it every block's.
 *
 * Scales lie in tiles of 128 rows x 4 scales (512 bytes), as the tensor cores'
 * block-scaled products read them: the byte of row r and scale k (k = column /
 * block) of an R x C matrix is at
 *   ((r / 128) * K4 + k / 4) * 512 + (r % 32) * 16 + (r % 128 / 32) * 4 + k % 4,
 * K4 = ceil(C / (4 * block)).  Bytes past the edges are written as zeros and
 * have to be zeros where a product reads them.
 * --------------------------------------------------------------------- */
typedef enum gs_fp4 { GS_MXFP4 = 0, GS_NVFP4 = 1 } gs_fp4;

/* Bytes of the scales of an R x C matrix (0 for sizes it refuses). */
size_t fp4_scale_bytes(int64_t R, int64_t C, int fmt);

/* Quantises x [R, C] (in_dtype, row distance ldx in elements), C % 32 == 0:
 *   q [R, C / 2], scales (fp4_scale_bytes(R, C))       -- as x lies, and/or
 *   qt [C, R / 2], scales_t (fp4_scale_bytes(C, R))    -- its transpose, blocks
 *       along x's columns (R % 32 == 0): the operands of the two products of a
 *       backward pass, whose sums run over the other dimension.
 * Either pair may be NULL, not both.
 *   tensor_scale -- device fp32 scalar, GS_NVFP4 only (else NULL).  With ws
 *       (device, gs_ws_bytes() bytes, 4-byte aligned) it is formed from x in a
 *       pass of its own and written; with ws NULL it is read (a scale of the
 *       steps before, say): one outside [2^-100, 2^120] makes every block's
 *       scale NaN, elements beyond 6 * 448 times it saturate.
 * q, scales, qt, scales_t 16-byte aligned.  Calls sharing a ws must be ordered
 * on one stream.  R == 0 or C == 0 writes the tensor scale alone. */
int fp4_quant(const void* x, int64_t ldx, int in_dtype, int64_t R, int64_t C, int fmt, uint8_t* q,
              uint8_t* scales, uint8_t* qt, uint8_t* scales_t, float* tensor_scale, void* ws,
              void* stream);

/* y = decode(q) * scale [* tensor_scale] in fp32, rounded to out_dtype (any of
 * the three) to nearest even; y [R, C] with row distance ldy. */
int fp4_dequant(const uint8_t* q, const uint8_t* scales, const float* tensor_scale, int64_t R,
                int64_t C, int fmt, int out_dtype, void* y, int64_t ldy, void* stream);

/* D = A B^T with A [M, K] and B [N, K] (a weight stored [out, in]) 4-bit
 * tensors of one format, times the product of their tensor scales ta and tb
 * (device fp32 scalars, GS_NVFP4 only, else NULL):
 *   D[m][n] = ta tb sum over k of decode(qa[m][k]) sa[m][k / block]
 *                                 decode(qb[n][k]) sb[n][k / block].
 * The backward products of Y = X W^T are the same call on transposed operands:
 * dX = dY (W^T)^T and dW = dY^T (X^T)^T, from the qt of fp4_quant.
 *   d: [M, N] with row distance ldd, out_dtype GS_F32 or GS_BF16 (rounded to
 *      nearest even from the fp32 sum); what lies between rows is not written.
 * Products and scales are exact in the tensor cores, sums in fp32 in an order
 * that depends on the sizes and the device alone: |error| <= 2^-23 (K / 16 +
 * 8) sum of |terms| before the output's rounding (an addition's error for each
 * 16 products, however the tensor cores round it).  Where ta tb itself is beyond
 * fp32's range, or subnormal, the sum is multiplied by one after the other: 2^-24 more.
 * K % 32 == 0, K <= 2^24, M, N < 2^31 and fewer than 2^30 tiles of 128 x 128
 * (else GS_ERR_SHAPE); any M and N; K == 0 writes zeros.  Codes and scales 16-byte
 * aligned.  A wait that runs out records GS_ERR_TIMEOUT (gs_device_status) and
 * leaves d unspecified. */
int fp4_gemm_block_scaled(const uint8_t* qa, const uint8_t* sa, const float* ta, const uint8_t* qb,
                          const uint8_t* sb, const float* tb, int64_t M, int64_t N, int64_t K,
                          int fmt, int out_dtype, void* d, int64_t ldd, void* stream);

/* ------------------------------------------------------------------------
 * The clipped policy loss over packed sequences, and its gradient with respect
 * to the tokens' log probabilities (which gs_token_logprob forms and
 * gs_token_logprob_bwd takes on to the logits, with the loss scale).
 * For a token with log probability x, x' under the policy that sampled it, x''
 * under a reference, and advantage A:
 *   rho = exp(x - x'),
 *   obj = rho A, but (1 + clip_high) A where A > 0 and rho > 1 + clip_high,
 *         (1 - clip_low) A where A < 0 and rho < 1 - clip_low, and
 *         dual_clip A where A < 0 and rho > dual_clip (dual_clip 0: none),
 *   kl  = exp(x'' - x) - 1 - (x'' - x),
 *   l   = -obj + kl_coef kl,      loss = sum over tokens of w l.
 * reduction: w = 1 / (tokens that count) for GS_LOSS_TOKEN_MEAN; 1 / (S' n_s)
 * for GS_LOSS_SEQUENCE_MEAN (n_s tokens that count in the token's sequence, S'
 * sequences that have any); 1 for GS_LOSS_SUM.
 *   logprob, old_logprob, ref_logprob: fp32 [T]; ref_logprob may be NULL with
 *       kl_coef 0 (given with it, it changes the mean of kl alone);
 *   advantages: fp32; n_advantages = T: one per token; S or -S: one per sequence
 *       (-S says so where T == S, which S does not);
 *   targets: int64 [T] as gs_token_logprob takes them: a token with a negative
 *       one does not count, whatever the other arrays hold there; NULL: all do;
 *   seq_offsets: int64 [S + 1], not decreasing: sequence s is the tokens
 *       [seq_offsets[s], seq_offsets[s + 1]); empty ones are fine.  Tokens before the
 *       first and after the last are in none: they do not count and their
 *       dlogprob is left as it was.  NULL: one sequence of all T (S = 1);
 *   dloss: device fp32 scalar that the gradient is multiplied by, or NULL (1);
 *   loss: device fp32 scalar, written; stats: fp32 [4] or NULL, over the tokens
 *       that count: their number, and the means of rho, of "obj is held" (0 or
 *       1) and of kl;
 *   dlogprob: fp32 [T] or NULL: dloss w dl/dx, 0 for tokens that do not count.
 *   ws: device workspace of gs_policy_loss_ws_bytes(T, S) bytes, 16-byte
 *       aligned, any contents; calls sharing one must be ordered on one stream.
 * clip_low, clip_high >= 0 (1 or more, Inf: never held there); dual_clip 0 or
 * >= 1.  A ratio or a divergence beyond fp32's range counts as what it is: a result
 * that is inside is finite, one beyond its infinity.  A log probability that is NaN
 * shows in the loss and in its token's gradient, an advantage of 0 or not.  No token that counts: loss,
 * statistics and gradient 0.  T, S <= 2^40,
 * S >= 1.  The same inputs give the same bits.
 * Gradients and the loss are off by at most 2^-20 of the terms they are made of,
 * |w| ((2 + |x - x'|) rho |A| + kl_coef (2 + |x'' - x|) (exp(x'' - x) + 1)), and half
 * a step of themselves.  In batches of up to 5120 tokens in up to 2048 sequences the loss sums A
 * and A (rho - 1) apart, so that advantages that cancel leave an objective that is off
 * by 2^-20 of |w A (rho - 1)| and 2^-40 of its terms; longer ones hold to the first
 * bound alone. */
typedef enum gs_loss_reduction {
  GS_LOSS_TOKEN_MEAN = 0,
  GS_LOSS_SEQUENCE_MEAN = 1,
  GS_LOSS_SUM = 2
} gs_loss_reduction;
size_t gs_policy_loss_ws_bytes(int64_t T, int64_t S);
int gs_policy_loss(const float* logprob, const float* old_logprob, const float* ref_logprob,
                   const float* advantages, int64_t n_advantages, const int64_t* targets, int64_t T,
                   const int64_t* seq_offsets, int64_t S, float clip_low, float clip_high,
                   float dual_clip, float kl_coef, int reduction, const float* dloss, float* loss,
                   float* stats, float* dlogprob, void* ws, void* stream);

/* ------------------------------------------------------------------------
 * The update of weight matrices by their orthogonalised momentum (K. Jordan,
 * "Muon: an optimizer for hidden layers in neural networks", 2024), on the
 * fp32 masters and skipped on the device like the other updates.
 * --------------------------------------------------------------------- */

/* A list of matrices: master[i] fp32 [rows[i], cols[i]], its bf16 copy
 * (master_bf16 or an entry of it may be NULL), gradients of grad_dtype (any of
 * the three) and momentum[i] fp32, each contiguous, element-aligned, of the
 * current device; nothing that is written may overlap anything else.  Fewer
 * than 2^31 elements per matrix, sides of up to 2^18 (fp32 sums of more would
 * be further off than the operands' roundings); empty ones are left out.  Allocates the list's
 * workspace: 8 bytes per element (rows counted up to a multiple of 8 elements) and
 * 4 per element of a square of the smaller side. */
typedef struct gs_muon_list gs_muon_list;
int gs_muon_list_create(float* const* master, uint16_t* const* master_bf16, const void* const* grads,
                        int grad_dtype, float* const* momentum, const int64_t* rows,
                        const int64_t* cols, int32_t n, gs_muon_list** out);
/* Waits for the device and frees the list. */
int gs_muon_list_destroy(gs_muon_list* list);

typedef enum gs_muon_scale { GS_MUON_SCALE_RMS = 0, GS_MUON_SCALE_ASPECT = 1 } gs_muon_scale;

/* One step of every matrix of the list, unless *found_inf is set (then nothing
 * is written):
 *   g = gradient * (max_norm / *grad_norm if 0 < max_norm < *grad_norm, else 1),
 *   m = mu m + g,   u = g + mu m (nesterov) or m,   X = u / |u| (Frobenius; a
 *       u of zeros stays zero),
 *   ns_steps times, on the smaller side:  G = X X^T,
 *       X = 3.4445 X + (-4.7750 G + 2.0315 G G) X,
 *   w = w (1 - lr weight_decay) - lr scale X;   bf16 copy = w rounded to nearest
 *       even;  scale = 0.2 sqrt(max(rows, cols)) (GS_MUON_SCALE_RMS: an update of
 *       AdamW's size) or sqrt(max(1, rows / cols)) (GS_MUON_SCALE_ASPECT).
 * G, the polynomial and X are held in fp16, scaled by powers of two to their ranges,
 * X up to its last step with what fp16 leaves of it beside it (22 bits; G is formed
 * from the first 11), sums in fp32.  After five or six steps X is off the exact
 * polynomial by 4e-4 to 2.5e-3 of its norm, whatever the singular values (flat, or a
 * few up to 1e5 times the rest).  More steps move singular values about near 1 and
 * errors with them, by slopes of up to 3.9: twenty end 2e-3 to 2e-2 off.  Sums of squares are fp32 within a thread's elements and fp64
 * beyond: elements of u below 2^-75 count as zero there, and a thread's sum above
 * fp32's range makes the matrix NaN.  Non-finite gradients are for
 * the check before this step to find.
 * lr, weight_decay finite and >= 0, mu in [0, 1), ns_steps 1 to 20; grad_norm
 * may be NULL when max_norm <= 0.  Calls on one list must be ordered on one
 * stream.  A wait that runs out records GS_ERR_TIMEOUT (gs_device_status) and
 * leaves the weights unspecified. */
int gs_master_update_muon(const gs_muon_list* list, float lr, float mu, float weight_decay,
                          int nesterov, int32_t ns_steps, int scale, float max_norm,
                          const float* grad_norm, const int32_t* found_inf, void* stream);

/* ------------------------------------------------------------------------
 * Diagnostics.
 * --------------------------------------------------------------------- */

/* Reads and clears the device status word of the current device
 * (GS_OK or GS_ERR_TIMEOUT recorded by a kernel that gave up waiting).
 * Synchronises `stream`. */
int gs_device_status(int32_t* h_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GSFP8_H */

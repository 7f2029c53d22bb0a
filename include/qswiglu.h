/*
 * qswiglu.h -- C ABI of libqswiglu.so, the GB300 (sm_103a) fused
 * weight-quantised SwiGLU expansion
 *
 *     hidden = silu(x . Wg^T) * (x . Wu^T)
 *
 * Source of the operation: mlx-bun source-diff pages ("mlx-bun 0.0.7 -> 0.0.9,
 * page 42" and "mlx-bun 0.0.8 -> 0.0.10, page 41"), file
 * src/model/fused-swiglu-kernel.ts: the header comment (what is fused, the MATCH
 * and F32 precision variants, down_proj left as a separate quantised matmul),
 * fusedSwigluSupported() (accepted quantisation specs) and fusedSwiglu()
 * (shapes, "caller owns" the result).  The standalone quantised linear follows
 * src/model/steel-linear-kernel.ts, steelLinear(), on page 43 ("mlx-bun 0.0.7 ->
 * 0.0.9, page 43").
 *
 * Data layout (all row-major, contiguous, device memory unless stated):
 *   x        bf16  [M, H]                 activation
 *   w        uint32 [rows, H*bits/32]     packed codes; code k of a row sits at
 *                                         bits (k mod pf)*bits of word k/pf,
 *                                         pf = 32/bits (little-endian, LSB first)
 *   scales   bf16  [rows, H/gs]           one scale per group of gs consecutive k
 *   biases   bf16  [rows, H/gs]           affine offsets ("zero points")
 *   dequantised weight  w[r,k] = bf16_rne(scale[r,k/gs] * q[r,k] + bias[r,k/gs])
 *   hidden   bf16  [M, I]
 *
 * Ownership: the caller allocates and owns every buffer; the library keeps no
 * pointer after a call returns and allocates no device memory.
 *
 * Execution: every entry point that takes `stream` (a cudaStream_t passed as
 * void*, NULL = the legacy default stream) only enqueues work on that stream
 * and returns; results are ready when the stream is synchronised.  The calling
 * thread's current CUDA device must be the one that owns the buffers.
 *
 * Errors: argument errors are detected on the host before anything is launched
 * (QSW_ERR_INVALID_ARG / QSW_ERR_UNSUPPORTED, nothing enqueued).  A failed
 * launch returns QSW_ERR_CUDA.  Kernels never trap: a device-side wait that
 * runs past its limit sets a device error word and the kernel exits; the word
 * is read (and cleared) by qsw_check_device_errors().  Nothing is thrown across
 * the ABI.
 */
#ifndef QSWIGLU_H_
#define QSWIGLU_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define QSW_API __attribute__((visibility("default")))
#else
#define QSW_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QSW_OK = 0,
    QSW_ERR_INVALID_ARG = 1,   /* null pointer, negative size, shape inconsistency */
    QSW_ERR_UNSUPPORTED = 2,   /* valid but not handled: bits, gs, H, alignment, size */
    QSW_ERR_CUDA = 3,          /* a CUDA runtime/driver call or launch failed */
    QSW_ERR_TIMEOUT = 4,       /* a kernel gave up on a device-side wait */
    QSW_ERR_BOUNDS = 5         /* debug build only: a device-side address or copy check failed */
} qsw_status;

/* Rounding variants of the fused expansion (fused-swiglu-kernel.ts, header
 * comment "PRECISION"; debug variants mirror its SWIGLU_DEBUG_GATE switch). */
typedef enum {
    QSW_MATCH = 0,       /* gate,up -> bf16; sigma, silu, product each rounded to bf16 */
    QSW_F32 = 1,         /* gate, up, sigma, silu kept f32; one rounding at the store */
    QSW_DEBUG_GATE = 2,  /* hidden := bf16(x . Wg^T), the stored gate projection */
    QSW_DEBUG_UP = 3     /* hidden := bf16(x . Wu^T), the stored up projection */
} qsw_variant;

/* Activation dtype of the *_ex entry points: x, the scales and biases of
 * both operands, and the result (fusedSwigluSupported() accepts bf16 or f16
 * activations; the dequantised weights, the stored projections and every MATCH
 * rounding are in the same dtype).  The other entry points are bf16. */
typedef enum {
    QSW_ACT_BF16 = 0,
    QSW_ACT_F16 = 1
} qsw_act_dtype;

/* Indices into the dispatch counters (fused-swiglu-kernel.ts keeps a call
 * counter so a test can prove the kernel ran). */
enum {
    QSW_CNT_FUSED_TC = 0,     /* fused expansion, tensor-core (tcgen05) kernel */
    QSW_CNT_FUSED_GEMV = 1,   /* fused expansion, small-M kernel */
    QSW_CNT_QMM_TC = 2,       /* affine_qmm, tensor-core kernel */
    QSW_CNT_QMM_GEMV = 3,     /* affine_qmm, small-M kernel */
    QSW_CNT_SILU_MUL = 4,     /* elementwise silu*mul */
    QSW_CNT_GEMV_STREAM = 5,  /* small-M calls (fused or affine_qmm) served by the warp-streamed kernel */
    QSW_CNT_FP4_QUANTIZE = 6,
    QSW_CNT_FP4_DEQUANTIZE = 7,
    QSW_CNT_FP4_LINEAR = 8,   /* qsw_fp4_linear and qsw_fp4_grouped_linear */
    QSW_CNT_MOE_ROUTE = 9,
    QSW_CNT_FP4_MOE = 10,     /* qsw_fp4_moe_mlp */
    QSW_CNT_NORM = 11,        /* qsw_rms_norm and qsw_post_norm */
    QSW_CNT_ROPE = 12,
    QSW_CNT_KV_APPEND = 13,
    QSW_CNT_PAGED_PLAN = 14,
    QSW_CNT_PAGED_ATTENTION = 15,
    QSW_NUM_COUNTERS = 16
};

/*
 * Fused expansion hidden[M,I] = epilogue(x . Wg^T, x . Wu^T).
 * Gate and up carry their own (gs, bits): fusedSwigluSupported() allows mixed
 * specs.  Accepted: M >= 0 (M = 0 enqueues nothing), H >= 32, I >= 1,
 * bits in {2,4,8}, gs a multiple of 32 dividing H, H a multiple of 32 (of 64
 * for 2-bit codes), variant in qsw_variant.  Pointers x, wg, wu, out must be
 * 16-byte aligned; scales/biases 2-byte aligned.  x and out must not overlap.
 * Rows M <= the small-M limit (qsw_set_gemv_max_m) run the memory-bound
 * kernel, the rest the tcgen05 tensor-core kernel; both compute the same
 * function.
 */
QSW_API qsw_status qswiglu_forward(const void *x, int64_t M, int64_t H, int64_t I,
                           const uint32_t *wg, const void *sg, const void *bg,
                           int gs_g, int bits_g,
                           const uint32_t *wu, const void *su, const void *bu,
                           int gs_u, int bits_u,
                           int variant, void *out, void *stream);

/*
 * Quantised linear y[M,N] = bf16(x[M,K] . W^T), W packed [N, K*bits/32]
 * with scales/biases [N, K/gs] (steel-linear-kernel.ts, steelLinear(): float
 * accumulator cast to bf16 at the store).  Used for the unfused comparison
 * path and for down_proj.  Same accepted shapes and alignment as above with
 * (H, I) -> (K, N).
 */
QSW_API qsw_status affine_qmm(const void *x, int64_t M, int64_t K, int64_t N,
                      const uint32_t *w, const void *s, const void *b,
                      int gs, int bits, void *y, void *stream);

/* Stream-K scheduling of the tensor-core kernel (qsw_set_stream_k). */
typedef enum {
    QSW_STREAM_K_OFF = 0,     /* whole output tiles, round-robin over the SMs */
    QSW_STREAM_K_AUTO = 1,    /* split K ranges where whole tiles would leave SMs idle (default) */
    QSW_STREAM_K_ALWAYS = 2   /* split whenever the tile count is not a multiple of the SM count */
} qsw_stream_k_mode;

/*
 * Bytes of workspace the *_ws entry points need on the current device
 * (a 1 KB header plus a 128 KB f32 partial accumulator per SM; 0 when no
 * device is current).
 */
QSW_API size_t qsw_workspace_bytes(void);

/*
 * qswiglu_forward / affine_qmm with a caller-owned device workspace that lets
 * the tensor-core kernel split the K range of output tiles between SMs
 * (stream-K) when whole tiles would fill the SMs unevenly -- e.g. 256 tiles on
 * 152 SMs.  A split tile is finished by the CTA holding its first K steps,
 * which adds the f32 partial accumulators that the others publish in the
 * workspace before the epilogue; results are the same function as the plain
 * entry points (f32 sums in a different order).
 *   workspace        device pointer, 256-byte aligned, zero-filled before its
 *                    first use (e.g. cudaMemsetAsync); the library keeps a
 *                    launch counter in it, so reuse it as is afterwards.  It
 *                    may be shared by the calls of one stream, not by calls
 *                    that can run concurrently.  NULL: whole tiles only.
 *   workspace_bytes  its size; less than qsw_workspace_bytes() returns
 *                    QSW_ERR_INVALID_ARG.
 * The small-M kernel does not use the workspace.  Other arguments, return
 * values and error behaviour as for the plain entry points.
 */
QSW_API qsw_status qswiglu_forward_ws(const void *x, int64_t M, int64_t H, int64_t I,
                           const uint32_t *wg, const void *sg, const void *bg,
                           int gs_g, int bits_g,
                           const uint32_t *wu, const void *su, const void *bu,
                           int gs_u, int bits_u,
                           int variant, void *out, void *workspace, size_t workspace_bytes,
                           void *stream);
QSW_API qsw_status affine_qmm_ws(const void *x, int64_t M, int64_t K, int64_t N,
                      const uint32_t *w, const void *s, const void *b,
                      int gs, int bits, void *y, void *workspace, size_t workspace_bytes,
                      void *stream);

/*
 * qswiglu_forward with stream-K scheduling and no caller workspace: the
 * split-tile partials go to a static device array of the library (sized for up
 * to 192 SMs; more SMs run whole tiles only), so the call allocates nothing
 * and takes no workspace argument.  The array is one per device: calls through
 * this entry point must not run concurrently with each other (use one stream,
 * or the *_ws form with one workspace per stream).  The first call on a device
 * also resolves the array's address and enqueues a 4 KB memset of its header
 * on `stream`; made inside a CUDA-graph capture, that memset becomes part of
 * the graph (every replay re-zeroes the header, which is harmless: the header
 * only needs to start at zero).  Should that first set-up fail, the call
 * returns QSW_ERR_CUDA and the next call tries again.  Arguments, results and
 * errors as for qswiglu_forward.
 */
QSW_API qsw_status qswiglu_forward_noalloc(const void *x, int64_t M, int64_t H, int64_t I,
                           const uint32_t *wg, const void *sg, const void *bg,
                           int gs_g, int bits_g,
                           const uint32_t *wu, const void *su, const void *bu,
                           int gs_u, int bits_u,
                           int variant, void *out, void *stream);

/*
 * The general forms: qswiglu_forward_ws / affine_qmm_ws / qsw_silu_mul with an
 * activation dtype (qsw_act_dtype; anything else returns QSW_ERR_INVALID_ARG).
 * With QSW_ACT_F16, x, scales, biases and the result are IEEE binary16 bit
 * patterns (same layouts and alignment), the dequantised weights are
 * f16(s*q + b) and the tensor cores run on f16 operands; everything else
 * (arguments, workspace, results, errors) is as for the bf16 forms.
 * affine_qmm_ex also takes `residual`: NULL, or [M, N] in the activation dtype
 * (16-byte aligned) added to the f32 accumulator before the one rounding,
 * y = T(x . W^T + residual); it may be y itself (each element is read before
 * it is written, by the same thread).
 */
QSW_API qsw_status qswiglu_forward_ex(const void *x, int64_t M, int64_t H, int64_t I,
                           const uint32_t *wg, const void *sg, const void *bg,
                           int gs_g, int bits_g,
                           const uint32_t *wu, const void *su, const void *bu,
                           int gs_u, int bits_u,
                           int variant, int act_dtype, void *out,
                           void *workspace, size_t workspace_bytes, void *stream);
QSW_API qsw_status affine_qmm_ex(const void *x, int64_t M, int64_t K, int64_t N,
                      const uint32_t *w, const void *s, const void *b,
                      int gs, int bits, int act_dtype, const void *residual, void *y,
                      void *workspace, size_t workspace_bytes, void *stream);
QSW_API qsw_status qsw_silu_mul_ex(const void *g, const void *u, int64_t n, int variant,
                        int act_dtype, void *out, void *stream);

/*
 * The whole MLP block with its residual (fused-mlp-kernel.ts on the pages:
 * the output is h + mlp(x)):
 *     hidden[M, I] = the fused expansion of x (variant QSW_MATCH or QSW_F32),
 *     y[M, Ho]     = T( h + hidden . Wd^T ),
 * down weights Wd packed [Ho, I*bits_d/32] with scales/biases [Ho, I/gs_d].
 * Two launches on `stream`: the fused expansion writes `hidden` (caller-owned,
 * [M, I] in the activation dtype, 16-byte aligned), then the down projection
 * adds the residual `h` ([M, Ho], or NULL for none; it may be y) to its f32
 * accumulator before the one rounding: deterministic, no atomics.  I must meet
 * the K rules of affine_qmm for the down weights (multiple of 32 and of gs_d).
 * The workspace (optional, as for the *_ws forms) serves both launches.
 * Argument errors in either stage return before anything is launched.
 */
QSW_API qsw_status qsw_mlp_forward_ex(const void *x, const void *h, int64_t M, int64_t H,
                           int64_t I, int64_t Ho,
                           const uint32_t *wg, const void *sg, const void *bg, int gs_g, int bits_g,
                           const uint32_t *wu, const void *su, const void *bu, int gs_u, int bits_u,
                           const uint32_t *wd, const void *sd, const void *bd, int gs_d, int bits_d,
                           int variant, int act_dtype, void *hidden, void *y,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Stream-K mode of the *_ws, *_ex and _noalloc entry points (qsw_stream_k_mode, default
 * QSW_STREAM_K_AUTO; other values are ignored).  Process-wide. */
QSW_API void qsw_set_stream_k(int mode);
QSW_API int qsw_get_stream_k(void);

/*
 * Elementwise out[i] = silu(g[i]) * u[i] over n bf16 values, the last step of
 * the unfused path (qwen3.ts, Qwen3MLP.forward: sigmoid, mul, mul).
 * variant QSW_MATCH rounds sigma, silu and the product to bf16; QSW_F32 rounds
 * once.  n >= 0; g, u, out 16-byte aligned; out may alias g or u.
 */
QSW_API qsw_status qsw_silu_mul(const void *g, const void *u, int64_t n, int variant,
                        void *out, void *stream);

/* ------------------------------------------------------------------------
 * Operators around the MLP block: microscaled 4-bit floating point, products
 * grouped by expert, routing, norms.  Inference only, like the rest of the
 * library (the weights are codes).  Same ownership, execution and error rules
 * as above.  An output must not overlap an input or another output except where
 * it is said that it may.
 * ------------------------------------------------------------------------ */

/*
 * Microscaled 4-bit formats: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives; sign in bit 3), two per byte with the even element in the low
 * nibble, and one scale per block of consecutive elements of a row.
 *   QSW_FP4_MX  blocks of 32, scale 2^(floor(log2 amax) - 2) held as E8M0
 *   QSW_FP4_NV  blocks of 16, scale E4M3(amax / (6 g)) times g, one positive
 *               f32 g for the whole tensor (the `scale` arguments below; 1 / (6 g)
 *               must be within f32's range, and g 1 for QSW_FP4_MX)
 * A code is the e2m1 value nearest to x / scale, ties to even, saturating at 6.
 * A block that holds an infinity or a NaN gets the scale NaN.
 *
 * A [rows, K] matrix is `codes`, rows * K/2 bytes, and `scales`, blocks of 128
 * rows by 4 scales of 512 bytes, row blocks outermost: row r, scale j is byte
 *     512 * ((r / 128) * ceil(K / (4 * block)) + j / 4)
 *     + 16 * (r % 32) + 4 * ((r / 32) % 4) + j % 4.
 * Bytes of rows past the last are never read for their values; those of scales
 * past the last must be 0 (qsw_fp4_quantize writes them).  A stack of matrices
 * is their codes and their scale blocks one after the other.
 */
typedef enum {
    QSW_FP4_MX = 0,
    QSW_FP4_NV = 1
} qsw_fp4_format;

/* Bytes of the scale blocks of `groups` matrices [rows, K]; 0 for arguments
 * that no call accepts. */
QSW_API size_t qsw_fp4_scale_bytes(int64_t groups, int64_t rows, int64_t K, int fmt);

/* Quantise x [groups, rows, K] (act_dtype) to codes and scales, and back.
 * K a multiple of 32, at most 2^22; all pointers 16-byte aligned. */
QSW_API qsw_status qsw_fp4_quantize(const void *x, int64_t groups, int64_t rows, int64_t K, int fmt, float scale,
                           int act_dtype, uint8_t *codes, uint8_t *scales, void *stream);
QSW_API qsw_status qsw_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t groups, int64_t rows,
                           int64_t K, int fmt, float scale, int act_dtype, void *out, void *stream);

/*
 * y[M, N] = T( Q(x) . W^T ): x [M, K] is quantised to the weights' format (with
 * the tensor scale x_scale) into the workspace, then multiplied on the
 * block-scaled tensor core with f32 accumulation, in an order that depends on
 * the sizes alone.  W: codes [N, K/2] and scale blocks, w_scale a device pointer
 * to its f32 tensor scale (NULL: 1).  K a multiple of 32; x, w, w_scales 16-byte
 * aligned, workspace 256-byte aligned with at least qsw_fp4_workspace_bytes(M,
 * K, 1, fmt) bytes (0: no call accepts such arguments, as for all sizes of these
 * operators).  The workspace need not be cleared; calls that can run
 * concurrently must not share it.  y may lie over x.
 */
QSW_API size_t qsw_fp4_workspace_bytes(int64_t rows, int64_t K, int groups, int fmt);
QSW_API qsw_status qsw_fp4_linear(const void *x, int64_t M, int64_t K, int64_t N, int fmt, float x_scale,
                           const uint8_t *w, const uint8_t *w_scales, const float *w_scale, int act_dtype,
                           void *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same with the rows of x sorted by group and a matrix per group: rows
 * offsets[e] .. offsets[e+1] - 1 are multiplied with W[e] (codes [groups, N,
 * K/2], a stack's scale blocks, w_scale [groups] or NULL).  offsets is
 * [groups + 1] int32 on the device, not decreasing from 0 to rows; a group may
 * be empty.  Any other table is taken as the nearest such one from below: an
 * entry counts as no less than 0 or than any entry before it, and as no more
 * than rows (nothing is read or written out of range, and no row belongs to two
 * groups).  Rows that no group covers are left unwritten.  At most 1024 groups.
 */
QSW_API qsw_status qsw_fp4_grouped_linear(const void *x, int64_t rows, int64_t K, int64_t N, int groups,
                           const int *offsets, int fmt, float x_scale, const uint8_t *w,
                           const uint8_t *w_scales, const float *w_scale, int act_dtype, void *y,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Logits may also be f32. */
enum { QSW_LOGITS_F32 = 2 };
typedef enum {
    QSW_ROUTE_SOFTMAX = 0,   /* weights are a softmax over all logits */
    QSW_ROUTE_SIGMOID = 1    /* weights are 1 / (1 + e^-logit) */
} qsw_route_scoring;

/*
 * Routing: per token the k largest of E logits (the lowest index first among
 * equals; NaN counts as -infinity) and their weights, largest logit first.
 * renormalize: the chosen weights are divided by their sum; then all are
 * multiplied by `scale`.  A row without any logit above -infinity gets the
 * weights 0; the sigmoid of logits up to -700 counts as 0.
 *   ids      int32 [T, k]  experts        weights  f32 [T, k]
 *   offsets  int32 [E + 1] first row of each expert in the expert-sorted order
 *   slots    int32 [T, k]  row of (token, choice) in that order
 *   order    int32 [T * k] the pair token * k + choice of each row
 * Rows of one expert are in token order.  E <= 1024, k <= 32.  logit_dtype:
 * qsw_act_dtype or QSW_LOGITS_F32.
 */
QSW_API qsw_status qsw_moe_route(const void *logits, int64_t T, int E, int k, int logit_dtype, int scoring,
                           int renormalize, float scale, int *ids, float *weights, int *offsets, int *slots,
                           int *order, void *stream);

/*
 * The MLP of a mixture of experts, with the routing of qsw_moe_route:
 *     hidden = silu(Q(x) . Wg[e]^T) * (Q(x) . Wu[e]^T)          in f32
 *     y[t]   = T( residual[t] + sum_j weights[t, j] Q(hidden) . Wd[e]^T )
 * with x [T, H] quantised with the tensor scale x_scale and hidden with h_scale.
 * wgu is [E, 2 I, H/2] with gate and up rows in alternating runs of 16 (rows
 * 32 i .. 32 i + 15 are gate features 16 i .. 16 i + 15, the next 16 the same
 * features' up rows), wd [E, H, I/2]; gu_scale and d_scale [E] or NULL.  H and
 * I multiples of 32.  residual [T, H] or NULL; it may be y.  A token's experts
 * must be distinct, as qsw_moe_route's are; with a routing that is not one of
 * qsw_moe_route's the values are unspecified, but nothing is read or written out
 * of range.  The weighted sum is one f32 sum of f32 rows per token in the order
 * of its choices, rounded once: the same bits every time.  (Among how many
 * others a token stands matters to them only where H or I passes 5888: the
 * products of few tokens may then add up K in parts.)
 */
QSW_API size_t qsw_fp4_moe_workspace_bytes(int64_t T, int k, int64_t H, int64_t I, int E, int fmt);
QSW_API qsw_status qsw_fp4_moe_mlp(const void *x, int64_t T, int64_t H, int64_t I, int E, int k, int fmt,
                           float x_scale, float h_scale, const int *ids, const float *weights,
                           const int *offsets, const int *slots, const int *order, const uint8_t *wgu,
                           const uint8_t *wgu_scales, const float *gu_scale, const uint8_t *wd,
                           const uint8_t *wd_scales, const float *d_scale, const void *residual,
                           int act_dtype, void *y, void *workspace, size_t workspace_bytes, void *stream);

/* out = T( x * rsqrt(mean(x^2) + eps) * weight ), weight [H] or NULL (1).
 * Any H up to 32768; statistics in f32.  out may be x. */
QSW_API qsw_status qsw_rms_norm(const void *x, const void *weight, int64_t rows, int64_t H, float eps,
                           int act_dtype, void *out, void *stream);

/*
 * What stands between two blocks, in one pass over the rows:
 *     z     = y * rsqrt(mean(y^2) + eps) * w_post     (norm_y; else z = y)
 *     h'    = h + scale * gate * z                     h_out = T(h')
 *     n_out = T( h' * rsqrt(mean(h'^2) + eps) * w_next )
 * n_out is computed from h' before it is rounded.  w_post, w_next [H] or NULL
 * (1); n_out may be NULL.  gate: NULL, or [gate_rows, gate_cols] with gate_cols
 * H or 1 and gate_rows a divisor of rows: row r takes gate row
 * r / (rows / gate_rows).  h_out may be h, n_out may be y.
 */
QSW_API qsw_status qsw_post_norm(const void *h, const void *y, int norm_y, const void *w_post, const void *gate,
                           int64_t gate_rows, int64_t gate_cols, float scale, const void *w_next, int64_t rows,
                           int64_t H, float eps, int act_dtype, void *h_out, void *n_out, void *stream);

/* ------------------------------------------------------------------------
 * The attention half of a decoder block: rotary positions, a paged cache of
 * keys and values, attention of new tokens over it.  Inference only.  Same
 * ownership, execution and error rules as above.
 * ------------------------------------------------------------------------ */

/* Heads of tokens: [T, heads, D] in the activation dtype, elements of a head
 * contiguous; strides in elements. */
typedef struct {
    const void *data;
    int64_t token_stride, head_stride;
} qsw_heads;

/* A paged cache: k and v [pages, kv_heads, page_size, D] in the activation dtype,
 * elements of a row contiguous, strides (page, head, row) in elements.  Token p of a
 * sequence is row p % page_size of page page_table[sequence][p / page_size].
 * page_size a multiple of 8, D a multiple of 8 from 8 to 128; pages * page_size
 * below 2^31.  k, v and all strides are multiples of 16 bytes, the strides positive and below
 * 2^40 bytes. */
typedef struct {
    void *k, *v;
    int64_t pages, kv_heads, page_size;
    int64_t k_strides[3], v_strides[3];
} qsw_kv_cache;

/*
 * Rotary positions: out[t, h] = x[t, h] with the pairs of its first `rot` elements
 * turned by the angle positions[t] * f_i and multiplied by `scale`; the others are
 * copied.  Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) with `interleaved`.
 * table[i] (int64 [rot / 2] on the device) is f_i in turns per position times 2^64,
 * modulo 2^64: positions (int32, of either sign; NULL: all 0) of any size keep their
 * angle to 2^-23 rad.  rot is even, from 0 to D; D at most 1024, heads at most 4096.  Any
 * strides; 2-byte alignment (16-byte alignment of everything is faster).  out may be
 * x with the same strides; else its rows share no memory with x's, nor with each other
 * (refused, of rows at other strides than x's only the latter).
 */
QSW_API qsw_status qsw_rope(const qsw_heads *x, int64_t T, int64_t heads, int64_t D, const int *positions,
                           const int64_t *table, int64_t rot, int interleaved, float scale, int act_dtype,
                           void *out, int64_t out_token_stride, int64_t out_head_stride, void *stream);

/*
 * Appends keys and values [T, kv_heads, D] to the cache: token t goes to row
 * slots[t] % page_size of page slots[t] / page_size, k turned as in qsw_rope (rot 0:
 * as it is).  q [T, heads, D], if not NULL, is turned into q_out in the same launch.  A slot
 * below 0 or past the cache is not written; a token at a negative position is left
 * out altogether, its row of q_out included.  Slots of two tokens should differ (else
 * the row is of either, or of parts of both).  The cache's alignment as stated there;
 * q, k, v and q_out as in qsw_rope; q_out may be q with the same strides, and is refused where
 * qsw_rope refuses it.
 */
QSW_API qsw_status qsw_kv_append(const qsw_heads *q, const qsw_heads *k, const qsw_heads *v, int64_t T, int64_t heads,
                                int64_t D, const int *slots, const int *positions, const int64_t *table,
                                int64_t rot, int interleaved, float scale, int act_dtype,
                                const qsw_kv_cache *cache, void *q_out, int64_t q_out_token_stride,
                                int64_t q_out_head_stride, void *stream);

/*
 * The plan of a step, which every layer's append and attention of that step share: the
 * new tokens of sequence b are rows offsets[b] .. offsets[b + 1] - 1 (int32 [B + 1] on
 * the device, not decreasing, from 0 to at most T), its last ones; lengths[b] (int32)
 * counts all its tokens, the new ones among them; page_table is int32 [B, max_pages]
 * with rows table_stride apart.  Writes positions and slots int32 [T] (-1: no
 * sequence's row, a position before the first, a page outside the cache) and the plan,
 * qsw_paged_plan_bytes(B, T) bytes, 16-byte aligned.  `window`: 0, or a token at
 * position p sees the keys p - window + 1 .. p.  A length counts as no less than 0 and
 * no more than max_pages * page_size; with offsets that decrease or pass T the values are
 * unspecified, but nothing is read or written out of range.  The plan holds
 * for calls with the same B, T, heads, D, window, max_pages and cache geometry; it is only read by them, so that
 * calls on several streams may share it.  B at most 65536, T at most 2^22, heads at
 * most 1024 and a multiple of kv_heads, T * heads at most 2^30, max_pages * page_size
 * below 2^31 - 1024.
 */
QSW_API size_t qsw_paged_plan_bytes(int64_t B, int64_t T);
QSW_API qsw_status qsw_paged_plan(const int *offsets, const int *lengths, int64_t B, const int *page_table,
                                 int64_t table_stride, int64_t max_pages, int64_t T, int64_t heads, int64_t D,
                                 int64_t window, const qsw_kv_cache *cache, int *positions, int *slots, void *plan,
                                 void *stream);

/*
 * out[t, h] = sum_j softmax_j(scale q[t, h] . k_j) v_j over the keys j that token t
 * sees: those of its sequence up to its own position (and within the window), of kv
 * head h / (heads / kv_heads).  out is [T, heads, D], contiguous, and
 * shares no memory with q (refused) or the cache.  A token that sees no key gets 0; rows
 * of no sequence are left as they were.  A page that is not in the cache counts as
 * zeros; what a row does not see has no effect on any bit of it, infinities and NaN among it.
 * Statistics and sums in f32, the weights rounded to the activation dtype before they
 * meet v (half a step of each, in f16 and below that 2^-32 of the row's largest); long histories are split over CTAs and joined in f32 in a fixed order: the same bits
 * every time.  scale > 0.  workspace: qsw_paged_attention_workspace_bytes(...) bytes
 * (max_len = max_pages * page_size), 256-byte aligned (0 bytes: may be NULL); it need not be cleared, and calls that can
 * run concurrently must not share it.  q, out: 16-byte aligned, as are q's strides.
 */
QSW_API size_t qsw_paged_attention_workspace_bytes(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t D,
                                                   int64_t max_len);
QSW_API qsw_status qsw_paged_attention(const qsw_heads *q, const qsw_kv_cache *cache, const int *page_table,
                                      int64_t table_stride, int64_t max_pages, const void *plan, int64_t B,
                                      int64_t T, int64_t heads, int64_t D, int64_t window, float scale,
                                      int act_dtype, void *out, void *workspace, size_t workspace_bytes,
                                      void *stream);

/* Synchronise `stream`, then read and clear the device error word.
 * Returns QSW_ERR_BOUNDS if a debug-build check failed (libqswiglu_debug.so
 * only), else QSW_ERR_TIMEOUT if any kernel gave up on a wait since the last
 * call, QSW_ERR_CUDA if synchronisation failed, else QSW_OK. */
QSW_API qsw_status qsw_check_device_errors(void *stream);

/* 1 in the debug build (libqswiglu_debug.so, compiled with QSW_DEBUG_BOUNDS):
 * every kernel fills its shared-memory staging areas -- and the tensor-core
 * kernel its TMEM accumulators -- with NaN bit patterns at start, so a read of
 * staging data that was never written shows up as NaN in the results, and
 * checks TMA copy coordinates (16-byte innermost offsets), shared-memory
 * ranges and output indices, reporting a failure as QSW_ERR_BOUNDS through
 * qsw_check_device_errors() without trapping.  0 in the regular build. */
QSW_API int qsw_debug_build(void);

/* Largest M routed to the small-M kernels (default 32; 0 sends every M to the
 * tensor-core kernel).  Values above 32 are clamped to 32.  Process-wide. */
QSW_API void qsw_set_gemv_max_m(int m);
QSW_API int qsw_get_gemv_max_m(void);

/* Which small-M kernel serves a call routed to the small-M path. */
typedef enum {
    QSW_SMALL_M_AUTO = 0,   /* the warp-streamed kernel where it applies (H <= 16384 and its staging
                               fits in shared memory; M > 16 runs as launches over row chunks of 16,
                               each streaming the weights once), else the slot-ring kernel (default) */
    QSW_SMALL_M_RING = 1,   /* always the slot-ring kernel (bulk copies into shared-memory slots
                               shared by a CTA's warps) */
    QSW_SMALL_M_STREAM = 2  /* the warp-streamed kernel where it applies (each warp copies its own
                               blocks into a private ring), else the slot-ring one */
} qsw_small_m_kernel;

/* Selects the small-M kernel (qsw_small_m_kernel; other values are ignored).
 * Both compute the same function; the choice changes only which one runs and,
 * within the f32 accumulation bound, the order of the additions.
 * Process-wide. */
QSW_API void qsw_set_small_m_kernel(int kernel);
QSW_API int qsw_get_small_m_kernel(void);

/* Early weight stream (default off).  When on, the small-M kernels are
 * launched as programmatic dependents of the work before them on the stream:
 * a call may start while the previous kernel is still running and requests
 * the packed weights (and, on the slot-ring kernel, the scales and biases) of
 * its first units or K blocks into shared memory at once; it reads x and
 * writes its output only after all earlier work on the stream has completed
 * (griddepcontrol.wait).  Turn it on only when no earlier work on the stream
 * writes the weight, scale or bias arrays of the call -- the usual decode loop,
 * where weights are constant.  Process-wide. */
QSW_API void qsw_set_early_weight_stream(int on);
QSW_API int qsw_get_early_weight_stream(void);

/* Per-wait limit for device-side waits, in nanoseconds (default 4e9). */
QSW_API void qsw_set_wait_timeout_ns(uint64_t ns);

/* Test hook, not for production use: the next call served by the slot-ring
 * small-M kernel (the warp-streamed kernel has no spin waits) never requests the first unit of each of its CTAs, so every wait on
 * that unit's shared-memory slot runs out after the qsw_set_wait_timeout_ns
 * limit.  The kernel then lets its other copies land and returns without
 * writing its output, and the next qsw_check_device_errors() returns
 * QSW_ERR_TIMEOUT.  Later calls are unaffected.  Nothing traps and nothing
 * waits without a limit. */
QSW_API void qsw_debug_withhold_next_fill(void);

/* The same for the next 4-bit product (qsw_fp4_linear, qsw_fp4_grouped_linear or the
 * first of qsw_fp4_moe_mlp): it never requests its weights, so its waits run out. */
QSW_API void qsw_debug_withhold_next_product(void);

/* The same for the next qsw_paged_attention: it never requests its first keys. */
QSW_API void qsw_debug_withhold_next_attention(void);

/* Dispatch counters (process-wide, monotonically increasing). `out` receives
 * min(n, QSW_NUM_COUNTERS) values. */
QSW_API void qsw_get_counters(uint64_t *out, int n);
QSW_API void qsw_reset_counters(void);

/* Static string for a status code. */
QSW_API const char *qsw_status_string(qsw_status s);

/* Library ABI version (major*100 + minor). */
QSW_API int qsw_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QSWIGLU_H_ */

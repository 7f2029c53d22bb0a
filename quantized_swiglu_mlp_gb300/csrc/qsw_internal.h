// Host-side declarations shared by the qswiglu translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qswiglu.h"

namespace qsw {

// One affine-quantised operand: packed codes [rows, K*bits/32], bf16
// scales/biases [rows, K/gs].
struct QuantOperand {
  const uint32_t *w;
  const uint16_t *s;
  const uint16_t *b;
  int gs;
  int bits;
};

// `act` (every launcher): the activation dtype, QSW_ACT_BF16 or QSW_ACT_F16 --
// x, scales, biases and the result share it.  `residual` (single-operand form
// only, else ignored): null, or [M, N] of that dtype added to the f32
// accumulator before the one rounding; it may be the output buffer itself.
//
// Small-M kernel: rows of x up to 32.  `dual` selects the fused SwiGLU
// (gate + up, epilogue `variant`) or a single quantised linear (y = bf16(x.W^T)).
// `early_weights`: launch as a programmatic dependent and stream weights
// before waiting for the preceding work (the caller guarantees that no earlier
// work on the stream writes the weight arrays).
cudaError_t launch_gemv(const void *x, int64_t M, int64_t K, int64_t N, const QuantOperand &op0,
                        const QuantOperand *op1, int variant, int act, void *out, const void *residual,
                        cudaStream_t stream, uint64_t timeout_ns, int num_sms, bool early_weights);

// Test hook: the next small-M launch never fills its CTAs' first slot, so
// that the waits on it run out.
void gemv_withhold_next();

// Warp-streamed small-M kernel (M <= 16): same arguments and result as
// launch_gemv; it has no spin waits.
cudaError_t launch_gemv_stream(const void *x, int64_t M, int64_t K, int64_t N, const QuantOperand &op0,
                               const QuantOperand *op1, int variant, int act, void *out, const void *residual,
                               cudaStream_t stream, int num_sms, bool early_weights);

// Whether the warp-streamed kernel applies (M <= 16, K <= 16384, x, the
// partial sums and the warps' rings fit in shared memory).
bool gemv_stream_fits(int64_t M, int64_t K, int64_t N, const QuantOperand &op0, const QuantOperand *op1,
                      int num_sms);

// Whether the slot-ring small-M kernel can stage rows of length K (else the
// tensor-core kernel serves every M).
bool gemv_fits(int64_t M, int64_t K, int64_t N, const QuantOperand &op0, const QuantOperand *op1, int num_sms);

// Stream-K workspace of the tensor-core kernel: null ptr (or fewer than
// prefill_workspace_bytes() bytes) means whole tiles only.
struct SplitWorkspace {
  void *ptr;
  size_t bytes;
  int mode;   // qsw_stream_k_mode
};

size_t prefill_workspace_bytes(int num_sms);

// The library's static stream-K workspace on the current device (a device
// array of the library, not an allocation); *ptr stays null where it is too
// small for the SM count.  Its header is zeroed on `stream` at first use.
cudaError_t prefill_static_workspace(int num_sms, cudaStream_t stream, void **ptr, size_t *bytes);

// Tensor-core kernel (tcgen05 + TMA), any M.
cudaError_t launch_prefill(const void *x, int64_t M, int64_t K, int64_t N, const QuantOperand &op0,
                           const QuantOperand *op1, int variant, int act, void *out, const void *residual,
                           cudaStream_t stream, uint64_t timeout_ns, int num_sms, const SplitWorkspace &ws);

cudaError_t launch_silu_mul(const void *g, const void *u, int64_t n, int variant, int act, void *out,
                            cudaStream_t stream);

// ------------------------------------------------- block operators ---------
// Microscaled 4-bit products, routing and norms (qsw_fp4*.cu, qsw_moe.cu,
// qsw_norm.cu).  `dependent`: launched as a programmatic dependent of the kernel
// before it on the stream.

// Quantise `groups` stacked [rows, K] matrices.
cudaError_t launch_fp4_quantize(const void *x, int64_t groups, int64_t rows, int64_t K, int fmt, int act, float g,
                                uint8_t *codes, uint8_t *scales, int num_sms, cudaStream_t stream);

// Quantise rows sorted by group, each group's scale blocks starting a new row
// block.
cudaError_t launch_fp4_quantize_ragged(const void *x, int64_t rows, int64_t K, const int *offsets, int groups,
                                       int fmt, int act, float g, uint8_t *codes, uint8_t *scales, int num_sms,
                                       cudaStream_t stream);

// Quantise tokens x [T, K], each to the rows slots[t, 0 .. k-1] of its groups
// ids[t, 0 .. k-1] in the order sorted by group.
cudaError_t launch_fp4_quantize_fan(const void *x, int64_t T, int64_t K, int k, const int *ids, const int *slots,
                                    const int *offsets, int groups, int fmt, int act, float g, uint8_t *codes,
                                    uint8_t *scales, cudaStream_t stream);

cudaError_t launch_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t groups, int64_t rows,
                                  int64_t K, int fmt, int act, float g, void *out, int num_sms, cudaStream_t stream);

struct Fp4GemmArgs {
  // either x in 4 bits, [rows, K] sorted by group, ragged scale blocks
  const uint8_t *x_codes, *x_scales;
  // or (fp4_gemm_quantizes) x itself, [x_tokens, K]; sorted row r is its row
  // order[r] / fan (order null: row r)
  const void *x;
  int64_t x_tokens;
  const int *order;
  int fan;
  int64_t rows, max_group;             // no group has more than max_group rows
  const int *offsets;                  // [groups + 1] on the device; null: one group
  int groups;
  const uint8_t *w_codes, *w_scales;   // [groups, N, K]
  int64_t N, K;
  const float *w_scale;                // [groups] on the device; null: 1
  float x_scale;
  int fmt, act;
  bool swiglu;                         // N = 2 I interleaved gate and up rows, result held in 4 bits
  void *out;                           // linear: [rows, N] in the activation dtype, or
  bool out_f32;                        // f32 (then x comes in 4 bits)
  uint8_t *h_codes, *h_scales;         // swiglu: [rows, I], ragged scale blocks
  float h_scale;
};
bool fp4_gemm_quantizes(int64_t rows, int64_t K, int fmt);
cudaError_t launch_fp4_gemm(const Fp4GemmArgs &a, int num_sms, uint64_t timeout_ns, cudaStream_t stream,
                            bool dependent);
cudaError_t fp4_gemm_take_errors(unsigned int *out);
void fp4_gemm_withhold_next();   // test hook: the next product's waits run out

cudaError_t launch_moe_route(const void *logits, int logit_dtype, int64_t T, int E, int k, int scoring,
                             int renormalize, float scale, int *ids, float *weights, int *offsets, int *slots,
                             int *order, cudaStream_t stream);
cudaError_t launch_moe_combine(const float *rows, int64_t n_rows, const int *slots, const float *weights,
                               const void *residual, int64_t T, int k, int64_t H, int act, void *y,
                               cudaStream_t stream, bool dependent);

struct NormArgs {
  const void *h, *y, *w_post, *gate, *w_next;
  int64_t gate_rows, gate_cols;
  int64_t rows, H;
  int norm_y, act;
  float scale, eps;
  void *h_out, *n_out;
};
cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t stream);

// ------------------------------------------------- attention ---------------
// Rotary positions, the paged cache and attention over it (qsw_rope.cu,
// qsw_attention*.cu).

struct RopeArgs {
  qsw_heads q, k, v;             // q.data null: none; k and v only with `slots`
  int64_t T, heads, D, rot;
  const int *positions, *slots;  // slots null: no cache
  const int64_t *table;
  int interleaved, act;
  float scale;
  void *out;                     // of q
  int64_t out_token_stride, out_head_stride;
  qsw_kv_cache cache;
};
cudaError_t launch_rope(const RopeArgs &a, int num_sms, cudaStream_t stream);

struct PlanArgs {
  const int *offsets, *lengths, *page_table;
  int64_t B, T, table_stride, max_pages, heads, D, window;
  qsw_kv_cache cache;
  int *positions, *slots;
  void *plan;
};
int64_t paged_plan_bytes(int64_t B, int64_t T);
cudaError_t launch_paged_plan(const PlanArgs &a, int num_sms, cudaStream_t stream);

struct AttentionArgs {
  qsw_heads q;
  qsw_kv_cache cache;
  int64_t B, T, table_stride, max_pages, heads, D, window;
  const int *page_table;
  const void *plan;
  float scale;
  int act;
  void *out, *workspace;
};
// Bytes of split results (0: no history is split).
size_t attention_workspace_bytes(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D, int64_t max_len,
                                 int num_sms);
cudaError_t attention_take_errors(unsigned int *out);
void attention_withhold_next();   // test hook: the next attention's waits run out
cudaError_t launch_paged_attention(const AttentionArgs &a, int num_sms, uint64_t timeout_ns, cudaStream_t stream);

// Shared state of the C entry points (qsw_api.cu).
int device_sm_count();
uint64_t wait_timeout_ns();
void count_call(int counter);

// Largest M the small-M kernel accepts.
constexpr int64_t kGemvMaxM = 32;

}  // namespace qsw

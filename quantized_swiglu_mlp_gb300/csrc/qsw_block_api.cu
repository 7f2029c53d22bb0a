// C entry points of the operators around the MLP block: microscaled 4-bit
// quantisation and products, products grouped by expert, routing and norms
// (include/qswiglu.h).  Arguments are checked before anything is enqueued.
#include <cfloat>
#include <cmath>

#include "qsw_fp4.cuh"
#include "qsw_internal.h"
#include "qswiglu.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kMaxGroups = 1024;
constexpr int kMaxTopK = 32;
constexpr int64_t kMaxK = int64_t(1) << 22;      // elements of a row
constexpr int64_t kMaxNorm = 32768;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
qsw_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSW_OK : QSW_ERR_CUDA; }
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Whether [a, a + n) and [b, b + m) have a byte in common.
bool overlap(const void *a, int64_t n, const void *b, int64_t m) {
  const auto p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q + static_cast<uintptr_t>(m) && q < p + static_cast<uintptr_t>(n);
}

bool act_ok(int act) { return act == QSW_ACT_BF16 || act == QSW_ACT_F16; }

// Format and tensor scale: the E8M0 format has no tensor scale, the other's needs a
// reciprocal within f32 (make_fp4_scale; a block of zeros would become NaN).
qsw_status check_format(int fmt, float g) {
  if (fmt != QSW_FP4_MX && fmt != QSW_FP4_NV) return QSW_ERR_INVALID_ARG;
  if (!(g > 0.0f) || !std::isfinite(g)) return QSW_ERR_INVALID_ARG;
  if (1.0 / (6.0 * static_cast<double>(g)) > static_cast<double>(FLT_MAX)) return QSW_ERR_INVALID_ARG;
  if (fmt == QSW_FP4_MX && g != 1.0f) return QSW_ERR_INVALID_ARG;
  return QSW_OK;
}

// Rows of `K` elements: whole MX blocks, 16-byte code rows.
qsw_status check_k(int64_t K) {
  if (K <= 0) return QSW_ERR_INVALID_ARG;
  return K % 32 != 0 || K > kMaxK ? QSW_ERR_UNSUPPORTED : QSW_OK;
}

size_t scale_bytes(int64_t row_blocks, int64_t K, int fmt) {
  return static_cast<size_t>(row_blocks * qsw::fp4_k_blocks(K, fmt) * qsw::kSfBytes);
}
// Scale blocks of `rows` rows in `groups` ragged groups.
size_t ragged_scale_bytes(int64_t rows, int groups, int64_t K, int fmt) {
  return scale_bytes(qsw::ragged_row_block(rows, groups), K, fmt);
}

qsw_status check_weights(const void *codes, const void *scales, const void *w_scale, int64_t groups, int64_t N) {
  if (!codes || !scales) return QSW_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(w_scale, 4)) return QSW_ERR_UNSUPPORTED;
  return groups * N > kMaxRows ? QSW_ERR_UNSUPPORTED : QSW_OK;
}

qsw_status grouped_linear(const void *x, int64_t rows, int64_t K, int64_t N, int groups, const int *offsets, int fmt,
                          float x_scale, const uint8_t *w, const uint8_t *ws, const float *w_scale, int act, void *y,
                          void *workspace, size_t workspace_bytes, cudaStream_t s) {
  if (rows < 0 || N <= 0) return QSW_ERR_INVALID_ARG;
  qsw_status st = check_format(fmt, x_scale);
  if (st != QSW_OK || (st = check_k(K)) != QSW_OK) return st;
  if (!act_ok(act)) return QSW_ERR_INVALID_ARG;
  if (rows > kMaxRows || N > kMaxRows) return QSW_ERR_UNSUPPORTED;
  if ((st = check_weights(w, ws, w_scale, groups, N)) != QSW_OK) return st;
  if (rows == 0) return QSW_OK;
  if (!x || !y || !workspace) return QSW_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 2) || !aligned(workspace, 256)) return QSW_ERR_UNSUPPORTED;
  if (workspace_bytes < qsw_fp4_workspace_bytes(rows, K, groups, fmt)) return QSW_ERR_INVALID_ARG;
  const int sms = qsw::device_sm_count();
  qsw::Fp4GemmArgs a = {};
  // Every CTA of the form without a quantiser reads x for itself, while others may be
  // writing y already: not where y lies over x.
  const bool fuse = qsw::fp4_gemm_quantizes(rows, K, fmt) && !overlap(x, rows * K * 2, y, rows * N * 2);
  if (fuse) {
    a.x = x;
    a.x_tokens = rows;
  } else {
    auto *codes = static_cast<uint8_t *>(workspace);
    uint8_t *scales = codes + up256(static_cast<size_t>(rows * (K / 2)));
    const cudaError_t e =
        offsets ? qsw::launch_fp4_quantize_ragged(x, rows, K, offsets, groups, fmt, act, x_scale, codes, scales, sms, s)
                : qsw::launch_fp4_quantize(x, 1, rows, K, fmt, act, x_scale, codes, scales, sms, s);
    if (e != cudaSuccess) return QSW_ERR_CUDA;
    a.x_codes = codes;
    a.x_scales = scales;
  }
  a.rows = a.max_group = rows;
  a.offsets = offsets;
  a.groups = groups;
  a.w_codes = w;
  a.w_scales = ws;
  a.N = N;
  a.K = K;
  a.w_scale = w_scale;
  a.x_scale = x_scale;
  a.fmt = fmt;
  a.act = act;
  a.out = y;
  a.h_scale = 1.0f;
  st = from_cuda(qsw::launch_fp4_gemm(a, sms, qsw::wait_timeout_ns(), s, !fuse));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_FP4_LINEAR);
  return st;
}

// Byte offsets of the parts of the expert MLP's workspace.  The experts' rows are f32
// until the weighted sum, at every size: rounded to T they overflow in f16 where the
// sum does not, and a token's result depends on how many others are in the batch.
// (Rows of T would halve what the down projection writes and the sum reads: 4096 tokens
// through 8 of 64 experts, H = 2048, I = 1024, take 208 us, with T 174.)
struct MoeWorkspace {
  size_t x_codes, x_scales, h_codes, h_scales, rows, total;
  MoeWorkspace(int64_t R, int64_t H, int64_t I, int E, int fmt) {
    x_codes = 0;
    x_scales = x_codes + up256(static_cast<size_t>(R * (H / 2)));
    h_codes = x_scales + up256(ragged_scale_bytes(R, E, H, fmt));
    h_scales = h_codes + up256(static_cast<size_t>(R * (I / 2)));
    rows = h_scales + up256(ragged_scale_bytes(R, E, I, fmt));
    total = rows + up256(static_cast<size_t>(R * H * 4));
  }
};

}  // namespace

extern "C" {

size_t qsw_fp4_scale_bytes(int64_t groups, int64_t rows, int64_t K, int fmt) {
  if (groups < 0 || rows < 0 || check_format(fmt, 1.0f) != QSW_OK || check_k(K) != QSW_OK) return 0;
  if (groups == 0 || rows > kMaxRows || groups > kMaxRows / (rows > 0 ? rows : 1)) return 0;
  return scale_bytes(groups * ((rows + qsw::kSfRows - 1) / qsw::kSfRows), K, fmt);
}

qsw_status qsw_fp4_quantize(const void *x, int64_t groups, int64_t rows, int64_t K, int fmt, float scale,
                            int act_dtype, uint8_t *codes, uint8_t *scales, void *stream) {
  if (groups < 0 || rows < 0) return QSW_ERR_INVALID_ARG;
  qsw_status st = check_format(fmt, scale);
  if (st != QSW_OK || (st = check_k(K)) != QSW_OK) return st;
  if (!act_ok(act_dtype)) return QSW_ERR_INVALID_ARG;
  if (groups == 0 || rows == 0) return QSW_OK;
  if (rows > kMaxRows || groups > kMaxRows / rows) return QSW_ERR_UNSUPPORTED;
  if (!x || !codes || !scales) return QSW_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return QSW_ERR_UNSUPPORTED;
  st = from_cuda(qsw::launch_fp4_quantize(x, groups, rows, K, fmt, act_dtype, scale, codes, scales,
                                          qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_FP4_QUANTIZE);
  return st;
}

qsw_status qsw_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t groups, int64_t rows, int64_t K,
                              int fmt, float scale, int act_dtype, void *out, void *stream) {
  if (groups < 0 || rows < 0) return QSW_ERR_INVALID_ARG;
  qsw_status st = check_format(fmt, scale);
  if (st != QSW_OK || (st = check_k(K)) != QSW_OK) return st;
  if (!act_ok(act_dtype)) return QSW_ERR_INVALID_ARG;
  if (groups == 0 || rows == 0) return QSW_OK;
  if (rows > kMaxRows || groups > kMaxRows / rows) return QSW_ERR_UNSUPPORTED;
  if (!codes || !scales || !out) return QSW_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16)) return QSW_ERR_UNSUPPORTED;
  st = from_cuda(qsw::launch_fp4_dequantize(codes, scales, groups, rows, K, fmt, act_dtype, scale, out,
                                            qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_FP4_DEQUANTIZE);
  return st;
}

size_t qsw_fp4_workspace_bytes(int64_t rows, int64_t K, int groups, int fmt) {
  if (rows < 0 || groups <= 0 || check_format(fmt, 1.0f) != QSW_OK || check_k(K) != QSW_OK) return 0;
  if (rows > kMaxRows || groups > kMaxGroups) return 0;
  return up256(static_cast<size_t>(rows * (K / 2))) + up256(ragged_scale_bytes(rows, groups, K, fmt));
}

qsw_status qsw_fp4_linear(const void *x, int64_t M, int64_t K, int64_t N, int fmt, float x_scale, const uint8_t *w,
                          const uint8_t *w_scales, const float *w_scale, int act_dtype, void *y, void *workspace,
                          size_t workspace_bytes, void *stream) {
  return grouped_linear(x, M, K, N, 1, nullptr, fmt, x_scale, w, w_scales, w_scale, act_dtype, y, workspace,
                        workspace_bytes, static_cast<cudaStream_t>(stream));
}

qsw_status qsw_fp4_grouped_linear(const void *x, int64_t rows, int64_t K, int64_t N, int groups, const int *offsets,
                                  int fmt, float x_scale, const uint8_t *w, const uint8_t *w_scales,
                                  const float *w_scale, int act_dtype, void *y, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  if (groups <= 0 || !offsets) return QSW_ERR_INVALID_ARG;
  if (groups > kMaxGroups || !aligned(offsets, 4)) return QSW_ERR_UNSUPPORTED;
  return grouped_linear(x, rows, K, N, groups, offsets, fmt, x_scale, w, w_scales, w_scale, act_dtype, y, workspace,
                        workspace_bytes, static_cast<cudaStream_t>(stream));
}

qsw_status qsw_moe_route(const void *logits, int64_t T, int E, int k, int logit_dtype, int scoring, int renormalize,
                         float scale, int *ids, float *weights, int *offsets, int *slots, int *order, void *stream) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return QSW_ERR_INVALID_ARG;
  if (logit_dtype != QSW_LOGITS_F32 && !act_ok(logit_dtype)) return QSW_ERR_INVALID_ARG;
  if (scoring != QSW_ROUTE_SOFTMAX && scoring != QSW_ROUTE_SIGMOID) return QSW_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return QSW_ERR_INVALID_ARG;
  if (E > kMaxGroups || k > kMaxTopK || T > kMaxRows / k) return QSW_ERR_UNSUPPORTED;
  if (!offsets || (T > 0 && (!logits || !ids || !weights || !slots || !order))) return QSW_ERR_INVALID_ARG;
  if (!aligned(logits, logit_dtype == QSW_LOGITS_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(offsets, 4) || !aligned(slots, 4) || !aligned(order, 4))
    return QSW_ERR_UNSUPPORTED;
  const qsw_status st =
      from_cuda(qsw::launch_moe_route(logits, logit_dtype, T, E, k, scoring, renormalize != 0, scale, ids, weights,
                                      offsets, slots, order, static_cast<cudaStream_t>(stream)));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_MOE_ROUTE);
  return st;
}

size_t qsw_fp4_moe_workspace_bytes(int64_t T, int k, int64_t H, int64_t I, int E, int fmt) {
  if (T < 0 || k <= 0 || E <= 0 || check_format(fmt, 1.0f) != QSW_OK || check_k(H) != QSW_OK || check_k(I) != QSW_OK)
    return 0;
  if (k > E || E > kMaxGroups || k > kMaxTopK || T > kMaxRows / k) return 0;
  return MoeWorkspace(T * k, H, I, E, fmt).total;
}

qsw_status qsw_fp4_moe_mlp(const void *x, int64_t T, int64_t H, int64_t I, int E, int k, int fmt, float x_scale,
                           float h_scale, const int *ids, const float *weights, const int *offsets,
                           const int *slots, const int *order, const uint8_t *wgu, const uint8_t *wgu_scales,
                           const float *gu_scale, const uint8_t *wd, const uint8_t *wd_scales, const float *d_scale,
                           const void *residual, int act_dtype, void *y, void *workspace, size_t workspace_bytes,
                           void *stream) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return QSW_ERR_INVALID_ARG;
  qsw_status st = check_format(fmt, x_scale);
  if (st != QSW_OK || (st = check_format(fmt, h_scale)) != QSW_OK) return st;
  if ((st = check_k(H)) != QSW_OK || (st = check_k(I)) != QSW_OK) return st;
  if (!act_ok(act_dtype)) return QSW_ERR_INVALID_ARG;
  if (E > kMaxGroups || k > kMaxTopK || T > kMaxRows / k) return QSW_ERR_UNSUPPORTED;
  if ((st = check_weights(wgu, wgu_scales, gu_scale, E, 2 * I)) != QSW_OK) return st;
  if ((st = check_weights(wd, wd_scales, d_scale, E, H)) != QSW_OK) return st;
  if (T == 0) return QSW_OK;
  if (!x || !y || !ids || !weights || !offsets || !slots || !order || !workspace) return QSW_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(workspace, 256) ||
      !aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(slots, 4) || !aligned(order, 4))
    return QSW_ERR_UNSUPPORTED;
  const int64_t R = T * k;
  const MoeWorkspace at(R, H, I, E, fmt);
  if (workspace_bytes < at.total) return QSW_ERR_INVALID_ARG;
  auto *ws = static_cast<uint8_t *>(workspace);
  const int sms = qsw::device_sm_count();
  const uint64_t timeout = qsw::wait_timeout_ns();
  auto s = static_cast<cudaStream_t>(stream);

  // rows sorted by expert, in 4 bits; gate and up with the SwiGLU, held in
  // 4 bits; down; the tokens' weighted sums
  cudaError_t e;
  qsw::Fp4GemmArgs a = {};
  const bool fuse = qsw::fp4_gemm_quantizes(T, H, fmt);
  if (fuse) {
    a.x = x;
    a.x_tokens = T;
    a.order = order;
    a.fan = k;
  } else {
    e = qsw::launch_fp4_quantize_fan(x, T, H, k, ids, slots, offsets, E, fmt, act_dtype, x_scale, ws + at.x_codes,
                                     ws + at.x_scales, s);
    if (e != cudaSuccess) return QSW_ERR_CUDA;
    a.x_codes = ws + at.x_codes;
    a.x_scales = ws + at.x_scales;
  }
  a.rows = R;
  a.max_group = T;      // a token's experts are distinct
  a.offsets = offsets;
  a.groups = E;
  a.w_codes = wgu;
  a.w_scales = wgu_scales;
  a.N = 2 * I;
  a.K = H;
  a.w_scale = gu_scale;
  a.x_scale = x_scale;
  a.fmt = fmt;
  a.act = act_dtype;
  a.swiglu = true;
  a.h_codes = ws + at.h_codes;
  a.h_scales = ws + at.h_scales;
  a.h_scale = h_scale;
  if ((e = qsw::launch_fp4_gemm(a, sms, timeout, s, !fuse)) != cudaSuccess) return QSW_ERR_CUDA;
  a.x = nullptr;
  a.x_codes = ws + at.h_codes;
  a.x_scales = ws + at.h_scales;
  a.w_codes = wd;
  a.w_scales = wd_scales;
  a.N = H;
  a.K = I;
  a.w_scale = d_scale;
  a.x_scale = h_scale;
  a.swiglu = false;
  a.out = ws + at.rows;
  a.out_f32 = true;
  if ((e = qsw::launch_fp4_gemm(a, sms, timeout, s, true)) != cudaSuccess) return QSW_ERR_CUDA;
  st = from_cuda(qsw::launch_moe_combine(reinterpret_cast<const float *>(ws + at.rows), R, slots, weights, residual, T,
                                         k, H, act_dtype, y, s, true));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_FP4_MOE);
  return st;
}

void qsw_debug_withhold_next_product(void) { qsw::fp4_gemm_withhold_next(); }

qsw_status qsw_rms_norm(const void *x, const void *weight, int64_t rows, int64_t H, float eps, int act_dtype,
                        void *out, void *stream) {
  if (rows < 0 || H <= 0 || !(eps >= 0.0f) || !std::isfinite(eps) || !act_ok(act_dtype)) return QSW_ERR_INVALID_ARG;
  if (H > kMaxNorm || rows > kMaxRows) return QSW_ERR_UNSUPPORTED;
  if (rows == 0) return QSW_OK;
  if (!x || !out) return QSW_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(out, 2)) return QSW_ERR_UNSUPPORTED;
  qsw::NormArgs a = {};
  a.h = x;
  a.w_next = weight;
  a.rows = rows;
  a.H = H;
  a.act = act_dtype;
  a.eps = eps;
  a.n_out = out;
  const qsw_status st = from_cuda(qsw::launch_norm(a, qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_NORM);
  return st;
}

qsw_status qsw_post_norm(const void *h, const void *y, int norm_y, const void *w_post, const void *gate,
                         int64_t gate_rows, int64_t gate_cols, float scale, const void *w_next, int64_t rows,
                         int64_t H, float eps, int act_dtype, void *h_out, void *n_out, void *stream) {
  if (rows < 0 || H <= 0 || !(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(scale) || !act_ok(act_dtype))
    return QSW_ERR_INVALID_ARG;
  if (!norm_y && w_post) return QSW_ERR_INVALID_ARG;
  if (H > kMaxNorm || rows > kMaxRows) return QSW_ERR_UNSUPPORTED;
  if (rows == 0) return QSW_OK;
  if (!h || !y || !h_out) return QSW_ERR_INVALID_ARG;
  if (gate && (gate_rows <= 0 || rows % gate_rows != 0 || (gate_cols != 1 && gate_cols != H)))
    return QSW_ERR_INVALID_ARG;
  if (!aligned(h, 2) || !aligned(y, 2) || !aligned(w_post, 2) || !aligned(gate, 2) || !aligned(w_next, 2) ||
      !aligned(h_out, 2) || !aligned(n_out, 2))
    return QSW_ERR_UNSUPPORTED;
  qsw::NormArgs a = {};
  a.h = h;
  a.y = y;
  a.norm_y = norm_y != 0;
  a.w_post = w_post;
  a.gate = gate;
  a.gate_rows = gate_rows;
  a.gate_cols = gate_cols;
  a.scale = scale;
  a.w_next = w_next;
  a.rows = rows;
  a.H = H;
  a.eps = eps;
  a.act = act_dtype;
  a.h_out = h_out;
  a.n_out = n_out;
  const qsw_status st = from_cuda(qsw::launch_norm(a, qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (st == QSW_OK) qsw::count_call(QSW_CNT_NORM);
  return st;
}

}  // extern "C"

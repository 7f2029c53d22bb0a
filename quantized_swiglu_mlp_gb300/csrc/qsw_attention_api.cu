// C entry points of the attention half of a block: rotary positions, the paged cache,
// attention over it (include/qswiglu.h).  Arguments are checked before anything is
// enqueued.
#include <cmath>

#include "qsw_internal.h"
#include "qswiglu.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxTokens = int64_t(1) << 22;     // of a plan
constexpr int64_t kMaxSequences = 65536;
constexpr int64_t kMaxHeads = 1024, kMaxRopeHeads = 4096;
constexpr int64_t kMaxHeadDim = 128, kMaxRopeDim = 1024;
constexpr int64_t kMaxWindow = int64_t(1) << 30;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
qsw_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSW_OK : QSW_ERR_CUDA; }
bool act_ok(int act) { return act == QSW_ACT_BF16 || act == QSW_ACT_F16; }

qsw_status check_cache(const qsw_kv_cache *c, int64_t D) {
  if (!c || c->pages <= 0 || c->kv_heads <= 0 || c->page_size <= 0 || D <= 0) return QSW_ERR_INVALID_ARG;
  if (!c->k || !c->v) return QSW_ERR_INVALID_ARG;
  if (c->page_size % 8 || D % 8 || D > kMaxHeadDim || c->kv_heads > kMaxHeads) return QSW_ERR_UNSUPPORTED;
  if (c->page_size > INT32_MAX || c->pages > INT32_MAX / c->page_size) return QSW_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QSW_ERR_UNSUPPORTED;
  // (strides as a copy takes them: below 2^40 bytes)
  for (int i = 0; i < 3; ++i) {
    if (c->k_strides[i] <= 0 || c->v_strides[i] <= 0) return QSW_ERR_INVALID_ARG;
    if (c->k_strides[i] % 8 || c->v_strides[i] % 8) return QSW_ERR_UNSUPPORTED;
    if (c->k_strides[i] >= (int64_t(1) << 39) || c->v_strides[i] >= (int64_t(1) << 39)) return QSW_ERR_UNSUPPORTED;
  }
  return QSW_OK;
}

qsw_status check_rotation(const int64_t *table, int64_t rot, int64_t D, float scale) {
  if (rot < 0 || rot % 2 || rot > D || !std::isfinite(scale)) return QSW_ERR_INVALID_ARG;
  if (rot > 0 && !table) return QSW_ERR_INVALID_ARG;
  return aligned(table, 8) ? QSW_OK : QSW_ERR_UNSUPPORTED;
}

// Sizes of a plan and of the calls that take it.
qsw_status check_step(int64_t B, int64_t T, int64_t heads, int64_t max_pages, int64_t table_stride, int64_t window,
                      const qsw_kv_cache *c) {
  if (B <= 0 || T < 0 || heads <= 0 || max_pages < 0 || table_stride < 0 || window < 0) return QSW_ERR_INVALID_ARG;
  if (heads % c->kv_heads) return QSW_ERR_INVALID_ARG;
  if (B > kMaxSequences || T > kMaxTokens || heads > kMaxHeads || T * heads > kMaxRows || window > kMaxWindow)
    return QSW_ERR_UNSUPPORTED;
  // (the end of a length's last tile is a 32-bit number too)
  return max_pages > (INT32_MAX - 1024) / c->page_size ? QSW_ERR_UNSUPPORTED : QSW_OK;
}

// Whether an element of the heads x [T, heads, D] lies in the `n` elements at p.
bool heads_meet(const qsw_heads &x, int64_t T, int64_t heads, int64_t D, const void *p, int64_t n) {
  using Wide = __int128;
  const Wide off = (static_cast<Wide>(reinterpret_cast<uintptr_t>(x.data)) - reinterpret_cast<uintptr_t>(p)) / 2;
  Wide ts = x.token_stride, hs = x.head_stride;
  const Wide t_span = (T - 1) * ts, h_span = (heads - 1) * hs;
  const Wide low = off + (t_span < 0 ? t_span : 0) + (h_span < 0 ? h_span : 0);
  const Wide high = off + (t_span > 0 ? t_span : 0) + (h_span > 0 ? h_span : 0) + D;
  if (low >= n || high <= 0) return false;
  // tokens counted so that they ascend
  const Wide first = off + (ts < 0 ? t_span : 0);
  ts = ts < 0 ? -ts : ts;
  for (int64_t h = 0; h < heads; ++h) {
    // a token t with -D < at + t ts < n
    const Wide at = first + h * hs;
    if (at >= n) continue;
    if (at > -D) return true;
    if (ts == 0) continue;
    const Wide t = (-D - at) / ts + 1;        // the first past -D
    if (t < T && at + t * ts < n) return true;
  }
  return false;
}

// Whether rows of heads [T, heads, D] share memory with each other (off 0), or with those of a
// tensor of the same strides `off` elements on.  (Differences of rows are of either sign: so may
// the strides be.)
bool rows_meet(int64_t T, int64_t heads, int64_t D, int64_t token_stride, int64_t head_stride, __int128 off) {
  using Wide = __int128;
  const auto size = [](Wide x) { return x < 0 ? -x : x; };
  const Wide ts = T == 1 ? 0 : size(token_stride), hs = heads == 1 ? 0 : size(head_stride);
  const Wide t_span = (T - 1) * ts, h_span = (heads - 1) * hs;
  if (off == 0) {
    // the usual: a token's heads one after the other, or a head's tokens
    if ((heads == 1 || hs >= D) && (T == 1 || ts >= h_span + D)) return false;
    if ((T == 1 || ts >= D) && (heads == 1 || hs >= t_span + D)) return false;
    if (T > 1 && ts < D) return true;
  } else if (size(off) >= t_span + h_span + D) {
    return false;
  }
  for (int64_t dh = off == 0 ? 1 : 1 - heads; dh < heads; ++dh) {
    // rows `dh` heads apart, and the number of tokens that brings them closest, or one more
    const Wide at = size(off + dh * hs);
    Wide dt = ts ? at / ts : 0;
    dt = dt < T ? dt : T - 1;
    if (at - dt * ts < D || (dt + 1 < T && (dt + 1) * ts - at < D)) return true;
  }
  return false;
}
// Whether `out` may take the heads of x: rows of its own, and either x's or none that meet them.
bool output_ok(const qsw_heads &x, int64_t T, int64_t heads, int64_t D, const void *out, int64_t token_stride,
               int64_t head_stride) {
  if (rows_meet(T, heads, D, token_stride, head_stride, 0)) return false;
  const bool alike = (T == 1 || token_stride == x.token_stride) && (heads == 1 || head_stride == x.head_stride);
  const __int128 off = static_cast<__int128>(reinterpret_cast<uintptr_t>(out)) - reinterpret_cast<uintptr_t>(x.data);
  return !alike || off == 0 || !rows_meet(T, heads, D, token_stride, head_stride, off / 2);
}

}  // namespace

extern "C" {

qsw_status qsw_rope(const qsw_heads *x, int64_t T, int64_t heads, int64_t D, const int *positions,
                    const int64_t *table, int64_t rot, int interleaved, float scale, int act_dtype, void *out,
                    int64_t out_token_stride, int64_t out_head_stride, void *stream) {
  if (!x || T < 0 || heads <= 0 || D <= 0 || !act_ok(act_dtype)) return QSW_ERR_INVALID_ARG;
  const qsw_status st = check_rotation(table, rot, D, scale);
  if (st != QSW_OK) return st;
  if (D > kMaxRopeDim || heads > kMaxRopeHeads || T > kMaxRows) return QSW_ERR_UNSUPPORTED;
  if (T == 0) return QSW_OK;
  if (!x->data || !out) return QSW_ERR_INVALID_ARG;
  if (!aligned(x->data, 2) || !aligned(out, 2) || !aligned(positions, 4)) return QSW_ERR_UNSUPPORTED;
  if (!output_ok(*x, T, heads, D, out, out_token_stride, out_head_stride)) return QSW_ERR_INVALID_ARG;
  qsw::RopeArgs a = {};
  a.q = *x;
  a.T = T, a.heads = heads, a.D = D, a.rot = rot;
  a.positions = positions;
  a.table = table;
  a.interleaved = interleaved != 0;
  a.act = act_dtype;
  a.scale = scale;
  a.out = out;
  a.out_token_stride = out_token_stride, a.out_head_stride = out_head_stride;
  const qsw_status r = from_cuda(qsw::launch_rope(a, qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (r == QSW_OK) qsw::count_call(QSW_CNT_ROPE);
  return r;
}

qsw_status qsw_kv_append(const qsw_heads *q, const qsw_heads *k, const qsw_heads *v, int64_t T, int64_t heads,
                         int64_t D, const int *slots, const int *positions, const int64_t *table, int64_t rot,
                         int interleaved, float scale, int act_dtype, const qsw_kv_cache *cache, void *q_out,
                         int64_t q_out_token_stride, int64_t q_out_head_stride, void *stream) {
  if (!k || !v || T < 0 || !act_ok(act_dtype) || (q && heads <= 0)) return QSW_ERR_INVALID_ARG;
  qsw_status st = check_cache(cache, D);
  if (st != QSW_OK || (st = check_rotation(table, rot, D, scale)) != QSW_OK) return st;
  if ((q && heads > kMaxRopeHeads) || T > kMaxRows) return QSW_ERR_UNSUPPORTED;
  if (T == 0) return QSW_OK;
  if (!k->data || !v->data || !slots || (q && (!q->data || !q_out))) return QSW_ERR_INVALID_ARG;
  if (!aligned(k->data, 2) || !aligned(v->data, 2) || !aligned(slots, 4) || !aligned(positions, 4) ||
      (q && (!aligned(q->data, 2) || !aligned(q_out, 2))))
    return QSW_ERR_UNSUPPORTED;
  if (q && !output_ok(*q, T, heads, D, q_out, q_out_token_stride, q_out_head_stride)) return QSW_ERR_INVALID_ARG;
  qsw::RopeArgs a = {};
  if (q) {
    a.q = *q;
    a.heads = heads;
    a.out = q_out;
    a.out_token_stride = q_out_token_stride, a.out_head_stride = q_out_head_stride;
  }
  a.k = *k, a.v = *v;
  a.T = T, a.D = D, a.rot = rot;
  a.positions = positions, a.slots = slots;
  a.table = table;
  a.interleaved = interleaved != 0;
  a.act = act_dtype;
  a.scale = scale;
  a.cache = *cache;
  const qsw_status r = from_cuda(qsw::launch_rope(a, qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (r == QSW_OK) qsw::count_call(QSW_CNT_KV_APPEND);
  return r;
}

size_t qsw_paged_plan_bytes(int64_t B, int64_t T) {
  if (B <= 0 || T < 0 || B > kMaxSequences || T > kMaxTokens) return 0;
  return static_cast<size_t>(qsw::paged_plan_bytes(B, T));
}

qsw_status qsw_paged_plan(const int *offsets, const int *lengths, int64_t B, const int *page_table,
                          int64_t table_stride, int64_t max_pages, int64_t T, int64_t heads, int64_t D, int64_t window,
                          const qsw_kv_cache *cache, int *positions, int *slots, void *plan, void *stream) {
  qsw_status st = check_cache(cache, D);
  if (st != QSW_OK || (st = check_step(B, T, heads, max_pages, table_stride, window, cache)) != QSW_OK) return st;
  if (T == 0) return QSW_OK;
  if (!offsets || !lengths || (max_pages > 0 && !page_table) || !positions || !slots || !plan)
    return QSW_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(lengths, 4) || !aligned(page_table, 4) || !aligned(positions, 4) ||
      !aligned(slots, 4) || !aligned(plan, 16))
    return QSW_ERR_UNSUPPORTED;
  qsw::PlanArgs a = {};
  a.offsets = offsets, a.lengths = lengths, a.page_table = page_table;
  a.B = B, a.T = T, a.table_stride = table_stride, a.max_pages = max_pages;
  a.heads = heads, a.D = D, a.window = window;
  a.cache = *cache;
  a.positions = positions, a.slots = slots;
  a.plan = plan;
  const qsw_status r = from_cuda(qsw::launch_paged_plan(a, qsw::device_sm_count(), static_cast<cudaStream_t>(stream)));
  if (r == QSW_OK) qsw::count_call(QSW_CNT_PAGED_PLAN);
  return r;
}

size_t qsw_paged_attention_workspace_bytes(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t D,
                                           int64_t max_len) {
  if (max_len < 0 || max_len > INT32_MAX || B <= 0 || T < 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads || D <= 0 || D % 8 || D > kMaxHeadDim) return 0;
  if (B > kMaxSequences || T > kMaxTokens || heads > kMaxHeads || T * heads > kMaxRows) return 0;
  return qsw::attention_workspace_bytes(T, B, heads, kv_heads, D, max_len, qsw::device_sm_count());
}

qsw_status qsw_paged_attention(const qsw_heads *q, const qsw_kv_cache *cache, const int *page_table,
                               int64_t table_stride, int64_t max_pages, const void *plan, int64_t B, int64_t T,
                               int64_t heads, int64_t D, int64_t window, float scale, int act_dtype, void *out,
                               void *workspace, size_t workspace_bytes, void *stream) {
  qsw_status st = check_cache(cache, D);
  if (st != QSW_OK || (st = check_step(B, T, heads, max_pages, table_stride, window, cache)) != QSW_OK) return st;
  if (!q || !act_ok(act_dtype) || !(scale > 0.0f) || !std::isfinite(scale * 1.5f)) return QSW_ERR_INVALID_ARG;
  if (T == 0) return QSW_OK;
  if (!q->data || !out || !plan || (max_pages > 0 && !page_table)) return QSW_ERR_INVALID_ARG;
  if (!aligned(q->data, 16) || !aligned(out, 16) || !aligned(plan, 16) || !aligned(page_table, 4) ||
      !aligned(workspace, 256) || q->token_stride % 8 || q->head_stride % 8)
    return QSW_ERR_UNSUPPORTED;
  const int sms = qsw::device_sm_count();
  if (sms <= 0) return QSW_ERR_CUDA;
  // (a row of q may be read after another is written)
  if (heads_meet(*q, T, heads, D, out, T * heads * D)) return QSW_ERR_INVALID_ARG;
  const size_t need =
      qsw_paged_attention_workspace_bytes(B, T, heads, cache->kv_heads, D, max_pages * cache->page_size);
  if (workspace_bytes < need || (need && !workspace)) return QSW_ERR_INVALID_ARG;
  qsw::AttentionArgs a = {};
  a.q = *q;
  a.cache = *cache;
  a.B = B, a.T = T, a.table_stride = table_stride, a.max_pages = max_pages;
  a.heads = heads, a.D = D, a.window = window;
  a.page_table = page_table;
  a.plan = plan;
  a.scale = scale;
  a.act = act_dtype;
  a.out = out;
  a.workspace = workspace;
  const qsw_status r = from_cuda(qsw::launch_paged_attention(a, sms, qsw::wait_timeout_ns(),
                                                             static_cast<cudaStream_t>(stream)));
  if (r == QSW_OK) qsw::count_call(QSW_CNT_PAGED_ATTENTION);
  return r;
}

void qsw_debug_withhold_next_attention(void) { qsw::attention_withhold_next(); }

}  // extern "C"

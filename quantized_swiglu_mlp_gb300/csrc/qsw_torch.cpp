// Python binding of the block operators (qsw_fp4_*, qsw_moe_*, qsw_rms_norm,
// qsw_post_norm, qsw_rope, qsw_kv_append, qsw_paged_*) for torch tensors: checks device, dtype, shape and contiguity,
// allocates results and scratch memory on the current stream, and calls the C entry
// points, whose addresses ops.py hands over from the library it loaded.
//
// These calls last a few microseconds on the device.  With the checks in Python
// and the call through ctypes, the host took 16 to 28 us for each.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

#include "qswiglu.h"

namespace {

// ------------------------------------------------------------ entry points --

#define QSW_ENTRIES(X)                                                                                       \
  X(qsw_fp4_quantize) X(qsw_fp4_dequantize) X(qsw_fp4_workspace_bytes) X(qsw_fp4_linear) X(qsw_fp4_grouped_linear) \
  X(qsw_moe_route) X(qsw_fp4_moe_workspace_bytes) X(qsw_fp4_moe_mlp) X(qsw_rms_norm) X(qsw_post_norm) \
  X(qsw_rope) X(qsw_kv_append) X(qsw_paged_plan_bytes) X(qsw_paged_plan) X(qsw_paged_attention_workspace_bytes)    \
  X(qsw_paged_attention)

struct Entries {
#define X(name) decltype(&::name) name##_;
  QSW_ENTRIES(X)
#undef X
};
Entries g_fn = {};
PyObject *g_raise = nullptr;   // raise_status(function name, status)

// A Python exception is set.
struct PyError {};

[[noreturn]] void fail(PyObject *type, const char *format, const char *name) {
  PyErr_Format(type, format, name);
  throw PyError();
}

void check_status(const char *fn, qsw_status st) {
  if (st == QSW_OK) return;
  PyObject *r = PyObject_CallFunction(g_raise, "si", fn, static_cast<int>(st));
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
  throw PyError();
}

// ------------------------------------------------------------------ checks --

bool is_act(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }
int act_code(at::ScalarType t) { return t == at::kBFloat16 ? QSW_ACT_BF16 : QSW_ACT_F16; }

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return t;
}

// A contiguous CUDA tensor of an activation type.
const at::Tensor &activation(PyObject *o, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (!is_act(t.scalar_type())) fail(PyExc_TypeError, "%s must be bfloat16 or float16", name);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

// A contiguous tensor of `dtype` on the device of `like`.
const at::Tensor &operand(PyObject *o, const char *name, at::ScalarType dtype, const at::Tensor &like) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != dtype) fail(PyExc_TypeError, "%s has the wrong dtype", name);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  if (t.device() != like.device()) fail(PyExc_ValueError, "%s is on another device", name);
  return t;
}

void *data(const at::Tensor &t) { return t.numel() ? t.data_ptr() : nullptr; }

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return v;
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return static_cast<float>(v);
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError();
  return v != 0;
}

int format(PyObject *o) {
  const int64_t f = integer(o);
  if (f != QSW_FP4_MX && f != QSW_FP4_NV) {
    PyErr_SetString(PyExc_ValueError, "fmt must be FP4_MX or FP4_NV");
    throw PyError();
  }
  return static_cast<int>(f);
}

// Row blocks of 128 and blocks of 4 scales of a [rows, K] matrix.
int64_t row_blocks(int64_t rows) { return (rows + 127) / 128; }
int64_t scale_blocks(int64_t K, int fmt) {
  const int64_t per = 4 * (fmt == QSW_FP4_MX ? 32 : 16);
  return (K + per - 1) / per;
}

// A 4-bit matrix (groups = -1) or stack with rows of K elements.
struct Weight {
  const at::Tensor *codes, *scales;
  const float *scale = nullptr;
  int64_t rows;
  Weight(PyObject *w, PyObject *s, PyObject *g, const char *name, const char *s_name, const char *g_name, int64_t K,
         int fmt, int64_t groups, const at::Tensor &like)
      : codes(&operand(w, name, at::kByte, like)), scales(&operand(s, s_name, at::kByte, like)) {
    const bool stack = groups >= 0;
    const int64_t d = stack ? 1 : 0;
    if (codes->dim() != d + 2 || (stack && codes->size(0) != groups) || codes->size(d + 1) * 2 != K)
      fail(PyExc_ValueError, "%s has the wrong shape: codes are [(groups,) rows, K/2]", name);
    rows = codes->size(d);
    if (scales->dim() != d + 3 || (stack && scales->size(0) != groups) || scales->size(d) != row_blocks(rows) ||
        scales->size(d + 1) != scale_blocks(K, fmt) || scales->size(d + 2) != 512)
      fail(PyExc_ValueError, "%s have the wrong shape: scales are [(groups,) row blocks, scale blocks, 512]", s_name);
    if (g != Py_None) {
      const at::Tensor &t = operand(g, g_name, at::kFloat, like);
      if (t.numel() != (stack ? groups : 1)) fail(PyExc_ValueError, "%s must have one value per matrix", g_name);
      scale = t.const_data_ptr<float>();
    }
  }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}
// The caller's output, or a new one.
at::Tensor output(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like) {
  if (o == Py_None) return empty(shape, dtype, like);
  const at::Tensor &t = operand(o, name, dtype, like);
  if (t.numel() != c10::multiply_integers(shape)) fail(PyExc_ValueError, "%s has the wrong size", name);
  return t;
}
// x's shape with its last dimension replaced.
c10::SmallVector<int64_t, 6> with_last(const at::Tensor &x, int64_t last) {
  c10::SmallVector<int64_t, 6> s(x.sizes().begin(), x.sizes().end());
  s.back() = last;
  return s;
}

void *current_stream(const at::Tensor &like) { return c10::cuda::getCurrentCUDAStream(like.get_device()).stream(); }

PyObject *wrap(at::Tensor t) {
  PyObject *o = THPVariable_Wrap(std::move(t));
  if (!o) throw PyError();
  return o;
}

// --------------------------------------------------------------- functions --

using Args = PyObject *const *;

// x, fmt, scale
PyObject *fp4_quantize(Args a) {
  const at::Tensor &x = activation(a[0], "x");
  const int fmt = format(a[1]);
  if (x.dim() != 2 && x.dim() != 3) fail(PyExc_ValueError, "%s must be [rows, K] or [groups, rows, K]", "x");
  const bool stack = x.dim() == 3;
  const int64_t groups = stack ? x.size(0) : 1, rows = x.size(-2), K = x.size(-1);
  c10::cuda::CUDAGuard guard(x.device());
  at::Tensor codes = empty(with_last(x, K / 2), at::kByte, x);
  const int64_t shape[4] = {groups, row_blocks(rows), scale_blocks(K, fmt), 512};
  at::Tensor scales = empty(at::IntArrayRef(shape + !stack, 3 + stack), at::kByte, x);
  check_status("qsw_fp4_quantize",
               g_fn.qsw_fp4_quantize_(data(x), groups, rows, K, fmt, number(a[2]), act_code(x.scalar_type()),
                                      static_cast<uint8_t *>(data(codes)), static_cast<uint8_t *>(data(scales)),
                                      current_stream(x)));
  PyObject *r = PyTuple_New(2);
  if (!r) throw PyError();
  PyTuple_SET_ITEM(r, 0, wrap(std::move(codes)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(scales)));
  return r;
}

// codes, scales, fmt, scale, act, out
PyObject *fp4_dequantize(Args a) {
  const at::Tensor &codes = tensor(a[0], "codes");
  if (codes.dim() != 2 && codes.dim() != 3) fail(PyExc_ValueError, "%s must be [rows, K/2] or [groups, rows, K/2]", "codes");
  const int fmt = format(a[2]);
  const bool stack = codes.dim() == 3;
  const int64_t K = codes.size(-1) * 2;
  const Weight w(a[0], a[1], Py_None, "codes", "scales", "", K, fmt, stack ? codes.size(0) : -1, codes);
  const int act = static_cast<int>(integer(a[4]));
  c10::cuda::CUDAGuard guard(codes.device());
  at::Tensor out = output(a[5], "out", with_last(codes, K), act == QSW_ACT_BF16 ? at::kBFloat16 : at::kHalf, codes);
  check_status("qsw_fp4_dequantize",
               g_fn.qsw_fp4_dequantize_(static_cast<uint8_t *>(data(codes)), static_cast<uint8_t *>(data(*w.scales)),
                                        stack ? codes.size(0) : 1, w.rows, K, fmt, number(a[3]), act, data(out),
                                        current_stream(codes)));
  return wrap(std::move(out));
}

// x, w, w_scales, fmt, x_scale, w_scale, out
PyObject *fp4_linear(Args a) {
  const at::Tensor &x = activation(a[0], "x");
  if (x.dim() < 1) fail(PyExc_ValueError, "%s must have at least one dimension", "x");
  const int fmt = format(a[3]);
  const int64_t K = x.size(-1), M = K ? x.numel() / K : 0;
  const Weight w(a[1], a[2], a[5], "w", "w scales", "w tensor scale", K, fmt, -1, x);
  c10::cuda::CUDAGuard guard(x.device());
  at::Tensor out = output(a[6], "out", with_last(x, w.rows), x.scalar_type(), x);
  const size_t bytes = g_fn.qsw_fp4_workspace_bytes_(M, K, 1, fmt);
  at::Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, x);
  check_status("qsw_fp4_linear",
               g_fn.qsw_fp4_linear_(data(x), M, K, w.rows, fmt, number(a[4]), w.codes->const_data_ptr<uint8_t>(),
                                    w.scales->const_data_ptr<uint8_t>(), w.scale, act_code(x.scalar_type()), data(out),
                                    data(ws), bytes, current_stream(x)));
  return wrap(std::move(out));
}

// x, offsets, w, w_scales, fmt, x_scale, w_scale, out
PyObject *fp4_grouped_linear(Args a) {
  const at::Tensor &x = activation(a[0], "x");
  const at::Tensor &offsets = operand(a[1], "offsets", at::kInt, x);
  const int fmt = format(a[4]);
  if (x.dim() != 2 || offsets.dim() != 1 || offsets.numel() < 2)
    fail(PyExc_ValueError, "%s must be [rows, K] and offsets [groups + 1]", "x");
  const int64_t rows = x.size(0), K = x.size(1), groups = offsets.numel() - 1;
  const Weight w(a[2], a[3], a[6], "w", "w scales", "w tensor scale", K, fmt, groups, x);
  c10::cuda::CUDAGuard guard(x.device());
  at::Tensor out = output(a[7], "out", {rows, w.rows}, x.scalar_type(), x);
  const int g32 = static_cast<int>(groups < INT32_MAX ? groups : INT32_MAX);
  const size_t bytes = g_fn.qsw_fp4_workspace_bytes_(rows, K, g32, fmt);
  at::Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, x);
  check_status("qsw_fp4_grouped_linear",
               g_fn.qsw_fp4_grouped_linear_(data(x), rows, K, w.rows, g32, offsets.const_data_ptr<int>(), fmt,
                                            number(a[5]), w.codes->const_data_ptr<uint8_t>(),
                                            w.scales->const_data_ptr<uint8_t>(), w.scale, act_code(x.scalar_type()),
                                            data(out), data(ws), bytes, current_stream(x)));
  return wrap(std::move(out));
}

// logits, k, scoring, renormalize, scale
PyObject *moe_route(Args a) {
  const at::Tensor &logits = tensor(a[0], "logits");
  const at::ScalarType t = logits.scalar_type();
  if (t != at::kFloat && !is_act(t)) fail(PyExc_TypeError, "%s must be float32, bfloat16 or float16", "logits");
  if (!logits.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", "logits");
  if (logits.dim() != 2) fail(PyExc_ValueError, "%s must be [T, E]", "logits");
  const int64_t T = logits.size(0), E = logits.size(1), k = integer(a[1]);
  if (k < 1 || k > E) fail(PyExc_ValueError, "%s must be between 1 and the number of experts", "k");
  c10::cuda::CUDAGuard guard(logits.device());
  at::Tensor ids = empty({T, k}, at::kInt, logits), weights = empty({T, k}, at::kFloat, logits),
             offsets = empty({E + 1}, at::kInt, logits), slots = empty({T, k}, at::kInt, logits),
             order = empty({T * k}, at::kInt, logits);
  const int E32 = static_cast<int>(E < INT32_MAX ? E : INT32_MAX), k32 = static_cast<int>(k < INT32_MAX ? k : INT32_MAX);
  check_status("qsw_moe_route",
               g_fn.qsw_moe_route_(data(logits), T, E32, k32, t == at::kFloat ? QSW_LOGITS_F32 : act_code(t),
                                   static_cast<int>(integer(a[2])), truth(a[3]), number(a[4]),
                                   static_cast<int *>(data(ids)), static_cast<float *>(data(weights)),
                                   offsets.data_ptr<int>(), static_cast<int *>(data(slots)),
                                   static_cast<int *>(data(order)), current_stream(logits)));
  PyObject *r = PyTuple_New(5);
  if (!r) throw PyError();
  at::Tensor *parts[5] = {&ids, &weights, &offsets, &slots, &order};
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, wrap(std::move(*parts[i])));
  return r;
}

// x, ids, weights, offsets, slots, order, wgu, wgu_scales, wd, wd_scales, fmt, x_scale, h_scale, gu_scale, d_scale,
// residual, out
PyObject *fp4_moe_mlp(Args a) {
  const at::Tensor &x = activation(a[0], "x");
  const at::Tensor &ids = operand(a[1], "route.ids", at::kInt, x), &weights = operand(a[2], "route.weights", at::kFloat, x),
                   &offsets = operand(a[3], "route.offsets", at::kInt, x),
                   &slots = operand(a[4], "route.slots", at::kInt, x), &order = operand(a[5], "route.order", at::kInt, x);
  const int fmt = format(a[10]);
  if (x.dim() != 2 || weights.dim() != 2) fail(PyExc_ValueError, "%s must be [T, H] and route moe_route's result", "x");
  const int64_t T = x.size(0), H = x.size(1), E = offsets.numel() - 1, k = weights.size(1);
  if (weights.size(0) != T || ids.sizes() != weights.sizes() || slots.sizes() != weights.sizes() || order.numel() != T * k ||
      E < 1 || E >= INT32_MAX || k >= INT32_MAX)
    fail(PyExc_ValueError, "%s does not belong to x", "route");
  const Weight gu(a[6], a[7], a[13], "wgu", "wgu scales", "wgu tensor scale", H, fmt, E, x);
  if (gu.rows % 2) fail(PyExc_ValueError, "%s must have 2 I rows", "wgu");
  const int64_t I = gu.rows / 2;
  const Weight d(a[8], a[9], a[14], "wd", "wd scales", "wd tensor scale", I, fmt, E, x);
  if (d.rows != H) fail(PyExc_ValueError, "%s must have H rows", "wd");
  const void *residual = nullptr;
  if (a[15] != Py_None) {
    const at::Tensor &r = operand(a[15], "residual", x.scalar_type(), x);
    if (r.numel() != T * H) fail(PyExc_ValueError, "%s has the wrong size", "residual");
    residual = data(r);
  }
  c10::cuda::CUDAGuard guard(x.device());
  at::Tensor out = output(a[16], "out", {T, H}, x.scalar_type(), x);
  const int E32 = static_cast<int>(E), k32 = static_cast<int>(k);
  const size_t bytes = g_fn.qsw_fp4_moe_workspace_bytes_(T, k32, H, I, E32, fmt);
  at::Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, x);
  check_status("qsw_fp4_moe_mlp",
               g_fn.qsw_fp4_moe_mlp_(data(x), T, H, I, E32, k32, fmt, number(a[11]), number(a[12]),
                                     static_cast<int *>(data(ids)), static_cast<float *>(data(weights)),
                                     offsets.const_data_ptr<int>(), static_cast<int *>(data(slots)),
                                     static_cast<int *>(data(order)), gu.codes->const_data_ptr<uint8_t>(),
                                     gu.scales->const_data_ptr<uint8_t>(), gu.scale, d.codes->const_data_ptr<uint8_t>(),
                                     d.scales->const_data_ptr<uint8_t>(), d.scale, residual, act_code(x.scalar_type()),
                                     data(out), data(ws), bytes, current_stream(x)));
  return wrap(std::move(out));
}

const void *norm_vector(PyObject *o, const char *name, int64_t H, const at::Tensor &like) {
  if (o == Py_None) return nullptr;
  const at::Tensor &w = operand(o, name, like.scalar_type(), like);
  if (w.dim() != 1 || w.size(0) != H) fail(PyExc_ValueError, "%s must have one value per column", name);
  return data(w);
}

// x, weight, eps, out
PyObject *rms_norm(Args a) {
  const at::Tensor &x = activation(a[0], "x");
  if (x.dim() < 1) fail(PyExc_ValueError, "%s must have at least one dimension", "x");
  const int64_t H = x.size(-1);
  const void *w = norm_vector(a[1], "weight", H, x);
  c10::cuda::CUDAGuard guard(x.device());
  at::Tensor out = output(a[3], "out", x.sizes(), x.scalar_type(), x);
  check_status("qsw_rms_norm", g_fn.qsw_rms_norm_(data(x), w, H ? x.numel() / H : 0, H, number(a[2]),
                                                  act_code(x.scalar_type()), data(out), current_stream(x)));
  return wrap(std::move(out));
}

// h, y, weight, gate, scale, next_weight, eps, norm, next_norm, out, next_out
PyObject *post_norm(Args a) {
  const at::Tensor &h = activation(a[0], "h");
  const at::Tensor &y = operand(a[1], "y", h.scalar_type(), h);
  if (h.dim() < 1 || y.sizes() != h.sizes()) fail(PyExc_ValueError, "%s and y must have the same shape", "h");
  const int64_t H = h.size(-1), rows = H ? h.numel() / H : 0;
  const void *w = norm_vector(a[2], "weight", H, h), *wn = norm_vector(a[5], "next_weight", H, h), *gate = nullptr;
  int64_t gate_rows = 0, gate_cols = 0;
  if (a[3] != Py_None) {
    const at::Tensor &g = operand(a[3], "gate", h.scalar_type(), h);
    if (g.dim() != 1 && g.dim() != 2) fail(PyExc_ValueError, "%s must be [H], [gate_rows, H] or [gate_rows, 1]", "gate");
    gate_rows = g.dim() == 1 ? 1 : g.size(0);
    gate_cols = g.size(-1);
    // (its pointer would be null, which is no gate)
    if (rows > 0 && g.numel() == 0) fail(PyExc_ValueError, "%s must not be empty", "gate");
    gate = data(g);
  }
  const bool norm = truth(a[7]), next_norm = truth(a[8]);
  c10::cuda::CUDAGuard guard(h.device());
  at::Tensor out = output(a[9], "out", h.sizes(), h.scalar_type(), h), next;
  if (next_norm) next = output(a[10], "next_out", h.sizes(), h.scalar_type(), h);
  check_status("qsw_post_norm",
               g_fn.qsw_post_norm_(data(h), data(y), norm, w, gate, gate_rows, gate_cols, number(a[4]), wn, rows, H,
                                   number(a[6]), act_code(h.scalar_type()), data(out), next_norm ? data(next) : nullptr,
                                   current_stream(h)));
  if (!next_norm) return wrap(std::move(out));
  PyObject *r = PyTuple_New(2);
  if (!r) throw PyError();
  PyTuple_SET_ITEM(r, 0, wrap(std::move(out)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(next)));
  return r;
}

// The attention's operators have no derivatives: a tensor that autograd would follow is
// refused instead of cut off.
void check_no_grad(const at::Tensor &t, const char *name) {
  if (c10::GradMode::is_enabled() && t.requires_grad())
    fail(PyExc_RuntimeError, "%s requires grad, and this operator has no derivative; detach it or use torch.no_grad()", name);
}
// What a call has written: autograd then knows that a value saved before is gone.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Heads [T, heads, D] of an activation type, a head's elements contiguous.
const at::Tensor &heads_of(PyObject *o, const char *name, const at::Tensor *like) {
  const at::Tensor &t = tensor(o, name);
  if (like ? t.scalar_type() != like->scalar_type() : !is_act(t.scalar_type()))
    fail(PyExc_TypeError, like ? "%s has the wrong dtype" : "%s must be bfloat16 or float16", name);
  if (like && t.device() != like->device()) fail(PyExc_ValueError, "%s is on another device", name);
  if (t.dim() != 3) fail(PyExc_ValueError, "%s must be [tokens, heads, head_dim]", name);
  if (t.size(2) > 1 && t.stride(2) != 1) fail(PyExc_ValueError, "%s must have contiguous heads", name);
  check_no_grad(t, name);
  return t;
}
// The stride of dimension d, for one of a single element that of a dense tensor.
int64_t step_of(const at::Tensor &t, int64_t d) {
  if (t.size(d) > 1) return t.stride(d);
  int64_t s = 1;
  for (int64_t i = d + 1; i < t.dim(); ++i) s *= t.size(i);
  return s;
}
qsw_heads heads_arg(const at::Tensor &t) { return qsw_heads{data(t), step_of(t, 0), step_of(t, 1)}; }

// k and v [pages, kv_heads, page_size, D] of the same type, shape and device as `like`'s.
qsw_kv_cache cache_arg(PyObject *ko, PyObject *vo, const at::Tensor *like) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  if (like ? k.scalar_type() != like->scalar_type() : !is_act(k.scalar_type()))
    fail(PyExc_TypeError, like ? "%s has the wrong dtype" : "%s must be bfloat16 or float16", "k_cache");
  if (v.scalar_type() != k.scalar_type()) fail(PyExc_TypeError, "%s has the wrong dtype", "v_cache");
  if (like && k.device() != like->device()) fail(PyExc_ValueError, "%s is on another device", "k_cache");
  if (v.device() != k.device()) fail(PyExc_ValueError, "%s is on another device", "v_cache");
  if (k.dim() != 4 || v.sizes() != k.sizes())
    fail(PyExc_ValueError, "%s and v_cache must be [pages, kv_heads, page_size, head_dim]", "k_cache");
  if (k.size(3) > 1 && (k.stride(3) != 1 || v.stride(3) != 1))
    fail(PyExc_ValueError, "%s and v_cache must have contiguous rows", "k_cache");
  check_no_grad(k, "k_cache");
  check_no_grad(v, "v_cache");
  qsw_kv_cache c = {data(k), data(v), k.size(0), k.size(1), k.size(2), {}, {}};
  for (int i = 0; i < 3; ++i) {
    c.k_strides[i] = step_of(k, i);
    c.v_strides[i] = step_of(v, i);
  }
  return c;
}
const int *indices(PyObject *o, const char *name, int64_t n, const at::Tensor &like) {
  const at::Tensor &t = operand(o, name, at::kInt, like);
  if (t.dim() != 1 || t.size(0) != n) fail(PyExc_ValueError, "%s has the wrong size", name);
  return static_cast<const int *>(data(t));
}
// The caller's output for heads like `x`, of any strides, or a new one.
at::Tensor heads_output(PyObject *o, const char *name, const at::Tensor &x) {
  if (o == Py_None) return empty(x.sizes(), x.scalar_type(), x);
  const at::Tensor &t = heads_of(o, name, &x);
  if (t.sizes() != x.sizes()) fail(PyExc_ValueError, "%s has the wrong size", name);
  return t;
}
struct Rotation {
  const int *positions = nullptr;
  const int64_t *table = nullptr;
  int64_t rot = 0;
  Rotation(PyObject *pos, PyObject *tab, int64_t T, const at::Tensor &like) {
    if (pos != Py_None) positions = indices(pos, "positions", T, like);
    if (tab == Py_None) return;
    const at::Tensor &t = operand(tab, "table", at::kLong, like);
    if (t.dim() != 1 || 2 * t.size(0) > like.size(2)) fail(PyExc_ValueError, "%s must have at most half as many values as a head", "table");
    if (T > 0 && t.size(0) && !positions) fail(PyExc_ValueError, "%s must be given where heads turn", "positions");
    table = static_cast<const int64_t *>(data(t));
    rot = 2 * t.size(0);
  }
};

// x, positions, table, interleaved, scale, out
PyObject *rope(Args a) {
  const at::Tensor &x = heads_of(a[0], "x", nullptr);
  const int64_t T = x.size(0), heads = x.size(1), D = x.size(2);
  const Rotation r(a[1], a[2], T, x);
  c10::cuda::CUDAGuard guard(x.device());
  at::Tensor out = heads_output(a[5], "out", x);
  const qsw_heads in = heads_arg(x);
  check_status("qsw_rope",
               g_fn.qsw_rope_(&in, heads ? T : 0, heads ? heads : 1, D, r.positions, r.table, r.rot, truth(a[3]),
                              number(a[4]), act_code(x.scalar_type()), data(out), step_of(out, 0), step_of(out, 1),
                              current_stream(x)));
  written(out);
  return wrap(std::move(out));
}

// k, v, k_cache, v_cache, slots, positions, table, q, interleaved, scale, q_out
PyObject *kv_append(Args a) {
  const at::Tensor &k = heads_of(a[0], "k", nullptr), &v = heads_of(a[1], "v", &k);
  const qsw_kv_cache cache = cache_arg(a[2], a[3], &k);
  const at::Tensor &kc = THPVariable_Unpack(a[2]);
  const int64_t T = k.size(0), D = k.size(2);
  if (v.sizes() != k.sizes()) fail(PyExc_ValueError, "%s and v must have the same shape", "k");
  if (k.size(1) != cache.kv_heads || D != kc.size(3)) fail(PyExc_ValueError, "%s does not fit the cache", "k");
  const int *slots = indices(a[4], "slots", T, k);
  const Rotation r(a[5], a[6], T, k);
  c10::cuda::CUDAGuard guard(k.device());
  const qsw_heads ka = heads_arg(k), va = heads_arg(v);
  qsw_heads qa = {};
  at::Tensor q_out;
  int64_t heads = 0;
  if (a[7] != Py_None) {
    const at::Tensor &q = heads_of(a[7], "q", &k);
    heads = q.size(1);
    if (q.size(0) != T || q.size(2) != D || heads < 1) fail(PyExc_ValueError, "%s does not fit k", "q");
    qa = heads_arg(q);
    q_out = heads_output(a[10], "q_out", q);
  } else if (a[10] != Py_None) {
    fail(PyExc_ValueError, "%s is given without q", "q_out");
  }
  check_status("qsw_kv_append",
               g_fn.qsw_kv_append_(heads ? &qa : nullptr, &ka, &va, T, heads, D, slots, r.positions, r.table, r.rot,
                                   truth(a[8]), number(a[9]), act_code(k.scalar_type()), &cache,
                                   heads ? data(q_out) : nullptr, heads ? step_of(q_out, 0) : 0,
                                   heads ? step_of(q_out, 1) : 0, current_stream(k)));
  written(kc);
  written(THPVariable_Unpack(a[3]));
  if (!heads) Py_RETURN_NONE;
  written(q_out);
  return wrap(std::move(q_out));
}

// A page table [B, max_pages], a sequence's pages contiguous.
const at::Tensor &page_table_of(PyObject *o, const at::Tensor &like) {
  const at::Tensor &t = tensor(o, "page_table");
  if (t.scalar_type() != at::kInt) fail(PyExc_TypeError, "%s has the wrong dtype", "page_table");
  if (t.device() != like.device()) fail(PyExc_ValueError, "%s is on another device", "page_table");
  if (t.dim() != 2) fail(PyExc_ValueError, "%s must be [sequences, pages]", "page_table");
  if (t.size(1) > 1 && t.stride(1) != 1) fail(PyExc_ValueError, "%s must have contiguous rows", "page_table");
  return t;
}

// offsets, lengths, page_table, k_cache, tokens, heads, window -> positions, slots, plan
PyObject *paged_plan(Args a) {
  const qsw_kv_cache cache = cache_arg(a[3], a[3], nullptr);
  const at::Tensor &kc = THPVariable_Unpack(a[3]);
  const at::Tensor &table = page_table_of(a[2], kc), &offsets = operand(a[0], "offsets", at::kInt, kc);
  const int64_t B = table.size(0), T = integer(a[4]), heads = integer(a[5]), D = kc.size(3);
  if (offsets.dim() != 1 || offsets.size(0) != B + 1 || B < 1)
    fail(PyExc_ValueError, "%s must have one value more than there are sequences", "offsets");
  const int *lengths = indices(a[1], "lengths", B, kc);
  if (T < 0) fail(PyExc_ValueError, "%s must not be negative", "tokens");
  c10::cuda::CUDAGuard guard(kc.device());
  const size_t bytes = g_fn.qsw_paged_plan_bytes_(B, T);
  const int64_t rows = bytes ? T : 0;     // (sizes that the call below refuses)
  at::Tensor positions = empty({rows}, at::kInt, kc), slots = empty({rows}, at::kInt, kc),
             plan = empty({static_cast<int64_t>(bytes)}, at::kByte, kc);
  check_status("qsw_paged_plan",
               g_fn.qsw_paged_plan_(offsets.const_data_ptr<int>(), lengths, B, static_cast<int *>(data(table)),
                                    step_of(table, 0), table.size(1), T, heads, D, integer(a[6]), &cache,
                                    static_cast<int *>(data(positions)), static_cast<int *>(data(slots)), data(plan),
                                    current_stream(kc)));
  PyObject *r = PyTuple_New(3);
  if (!r) throw PyError();
  at::Tensor *parts[3] = {&positions, &slots, &plan};
  for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(r, i, wrap(std::move(*parts[i])));
  return r;
}

// q, k_cache, v_cache, page_table, plan, plan's (tokens, heads, window, pages, kv_heads, page_size, head_dim), scale, out
PyObject *paged_attention(Args a) {
  const at::Tensor &q = heads_of(a[0], "q", nullptr);
  const qsw_kv_cache cache = cache_arg(a[1], a[2], &q);
  const at::Tensor &kc = THPVariable_Unpack(a[1]);
  const at::Tensor &table = page_table_of(a[3], q), &plan = operand(a[4], "plan", at::kByte, q);
  const int64_t T = q.size(0), heads = q.size(1), D = q.size(2), B = table.size(0);
  if (D != kc.size(3)) fail(PyExc_ValueError, "%s does not fit the cache", "q");
  const int64_t made[6] = {T, heads, cache.pages, cache.kv_heads, cache.page_size, D};
  const int at_arg[6] = {5, 6, 8, 9, 10, 11};
  for (int i = 0; i < 6; ++i)
    if (integer(a[at_arg[i]]) != made[i]) fail(PyExc_ValueError, "%s was made for other sizes", "plan");
  if (static_cast<size_t>(plan.numel()) != g_fn.qsw_paged_plan_bytes_(B, T))
    fail(PyExc_ValueError, "%s was made for other sizes", "plan");
  c10::cuda::CUDAGuard guard(q.device());
  at::Tensor out = output(a[13], "out", q.sizes(), q.scalar_type(), q);
  check_no_grad(out, "out");
  const size_t bytes = g_fn.qsw_paged_attention_workspace_bytes_(B, T, heads, cache.kv_heads, D,
                                                                  table.size(1) * cache.page_size);
  at::Tensor ws;
  if (bytes) ws = empty({static_cast<int64_t>(bytes)}, at::kByte, q);
  const qsw_heads in = heads_arg(q);
  check_status("qsw_paged_attention",
               g_fn.qsw_paged_attention_(&in, &cache, static_cast<int *>(data(table)), step_of(table, 0), table.size(1),
                                         data(plan), B, T, heads, D, integer(a[7]), number(a[12]),
                                         act_code(q.scalar_type()), data(out), bytes ? data(ws) : nullptr, bytes,
                                         current_stream(q)));
  written(out);
  return wrap(std::move(out));
}

// {name: address}, raise_status
PyObject *bind(Args a) {
#define X(name)                                                        \
  {                                                                    \
    PyObject *v = PyDict_GetItemString(a[0], #name);                   \
    if (!v) fail(PyExc_KeyError, "%s is not bound", #name);            \
    g_fn.name##_ = reinterpret_cast<decltype(&::name)>(PyLong_AsVoidPtr(v)); \
    if (PyErr_Occurred()) throw PyError();                             \
  }
  QSW_ENTRIES(X)
#undef X
  Py_INCREF(a[1]);
  Py_XDECREF(g_raise);
  g_raise = a[1];
  Py_RETURN_NONE;
}

// Argument count, and every C++ exception as a Python one.
template <PyObject *(*F)(Args), Py_ssize_t N>
PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
  try {
    return F(a);
  } catch (const PyError &) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());   // torch's own, out of memory among them
  }
  return nullptr;
}

#define METHOD(name, args) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name, args>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(bind, 2),        METHOD(fp4_quantize, 3),       METHOD(fp4_dequantize, 6),
                           METHOD(fp4_linear, 7),  METHOD(fp4_grouped_linear, 8), METHOD(moe_route, 5),
                           METHOD(fp4_moe_mlp, 17), METHOD(rms_norm, 4),          METHOD(post_norm, 11),
                           METHOD(rope, 6),        METHOD(kv_append, 11),         METHOD(paged_plan, 7),
                           METHOD(paged_attention, 14),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_qsw_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qsw_torch(void) { return PyModule_Create(&g_module); }

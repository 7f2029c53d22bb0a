// Python binding of the block operators (qsw_fp4_*, qsw_moe_*, qsw_rms_norm,
// qsw_post_norm) for torch tensors: checks device, dtype, shape and contiguity,
// allocates results and scratch memory on the current stream, and calls the C entry
// points, whose addresses ops.py hands over from the library it loaded.
//
// These calls last a few microseconds on the device.  With the checks in Python
// and the call through ctypes, the host took 16 to 28 us for each.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
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
  X(qsw_moe_route) X(qsw_fp4_moe_workspace_bytes) X(qsw_fp4_moe_mlp) X(qsw_rms_norm) X(qsw_post_norm)

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
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_qsw_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qsw_torch(void) { return PyModule_Create(&g_module); }

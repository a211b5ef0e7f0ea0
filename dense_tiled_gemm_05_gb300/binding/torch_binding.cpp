// torch_binding.cpp -- the calls of the feed-forward operators, of the operators of experts and
// of dropout on torch tensors, compiled.
//
// A generation step calls them with a few microseconds of work each, so the host's part of a
// call is part of its latency: marshalled in Python a layer norm took 11 us on the host (Grace
// CPU), here 3.4, a torch addition 4.4. Like the ctypes binding this only marshals: it checks
// and reads shapes, strides, types and streams, allocates outputs and calls the C ABI, whose
// functions Python hands over as addresses (init), so that this module links to torch only.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstring>
#include <initializer_list>
#include <optional>

#include "gemm.h"

namespace {

decltype(&gemm_run_epilogue) run_epilogue = nullptr;
decltype(&gemm_run_epilogue_backward) run_epilogue_backward = nullptr;
decltype(&gemm_run_gated) run_gated = nullptr;
decltype(&gemm_run_gated_backward) run_gated_backward = nullptr;
decltype(&gemm_layer_norm) run_layer_norm = nullptr;
decltype(&gemm_layer_norm_backward) run_layer_norm_backward = nullptr;
decltype(&gemm_expert_sort) run_expert_sort = nullptr;
decltype(&gemm_expert_gather) run_expert_gather = nullptr;
decltype(&gemm_expert_combine) run_expert_combine = nullptr;
decltype(&gemm_expert_combine_backward) run_expert_combine_backward = nullptr;
decltype(&gemm_run_expert) run_expert = nullptr;
decltype(&gemm_run_expert_backward) run_expert_backward = nullptr;
decltype(&gemm_run_expert_gated) run_expert_gated = nullptr;
decltype(&gemm_run_expert_gated_backward) run_expert_gated_backward = nullptr;
decltype(&gemm_dropout) run_dropout = nullptr;
PyObject *raise_status = nullptr;  // raise_status(code, function name) raises

using at::Tensor;

// Leaves the call with a Python exception (PyErr_Format's formats).
[[noreturn]] void fail(PyObject *type, const char *format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw python_error();
}

// ------------------------------------------------------------------ arguments

Tensor tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", what);
  return THPVariable_Unpack(o);
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return GEMM_F32;
    case at::kHalf: return GEMM_F16;
    case at::kBFloat16: return GEMM_BF16;
    default: fail(PyExc_TypeError, "unsupported dtype %s", c10::toString(t));
  }
}
int code_of(const Tensor &t) { return code_of(t.scalar_type()); }

const char *text(PyObject *o) {
  const char *s = PyUnicode_AsUTF8(o);
  if (!s) throw python_error();
  return s;
}

// A torch dtype or one of the library's names; `otherwise` for None.
at::ScalarType dtype_arg(PyObject *o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (THPDtype_Check(o)) {
    const at::ScalarType t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    code_of(t);
    return t;
  }
  if (PyUnicode_Check(o)) {
    const char *s = text(o);
    if (!std::strcmp(s, "f32")) return at::kFloat;
    if (!std::strcmp(s, "f16")) return at::kHalf;
    if (!std::strcmp(s, "bf16")) return at::kBFloat16;
  }
  fail(PyExc_TypeError, "unsupported dtype");
}

int name_arg(PyObject *o, const char *const *names, int n, const char *what) {
  if (o == Py_None) return 0;
  if (!PyUnicode_Check(o)) fail(PyExc_TypeError, "%s must be a string or None", what);
  const char *s = text(o);
  for (int i = 0; i < n; ++i)
    if (!std::strcmp(s, names[i])) return i;
  fail(PyExc_ValueError, "unknown %s '%s'", what, s);
}
gemm_activation_t activation_arg(PyObject *o) {
  static const char *const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"};
  return static_cast<gemm_activation_t>(name_arg(o, names, 6, "activation"));
}
gemm_precision_t precision_arg(PyObject *o) {
  static const char *const names[] = {"default", "tf32", "exact", "f16acc"};
  return static_cast<gemm_precision_t>(name_arg(o, names, 4, "precision"));
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
struct Need {
  bool v[3];
  explicit Need(PyObject *o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3)
      fail(PyExc_ValueError, "need must be a tuple of three truth values");
    for (int i = 0; i < 3; ++i) v[i] = truth(PyTuple_GET_ITEM(o, i));
  }
};

gemm_handle_t handle_arg(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<gemm_handle_t>(p);
}

// The stream of a call: the current one, or another that the caller names. On another, the call
// does what it would with that stream current -- its outputs come from that stream's memory, or
// they could lie where the current stream's work is not done yet -- and the allocator learns of
// every tensor that two streams use.
class CallStream {
 public:
  CallStream(PyObject *o, int dev)
      : current_(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev))) {
    ptr_ = current_.stream();
    if (o == Py_None) return;
    PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw python_error();
    void *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw python_error();
    if (s == ptr_) return;
    ptr_ = s;
    other_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s),
                                                    static_cast<c10::DeviceIndex>(dev)));
  }
  void *get() const { return ptr_; }
  // The caller's tensors, before the call; its new ones, after.
  void uses(std::initializer_list<const Tensor *> tensors) const { record(tensors, true); }
  void gives(std::initializer_list<const Tensor *> tensors) const { record(tensors, false); }

 private:
  void record(std::initializer_list<const Tensor *> tensors, bool on_call) const {
    if (!other_) return;
    const c10::Stream s = on_call ? other_->current_stream().unwrap() : current_.unwrap();
    for (const Tensor *t : tensors)
      if (t->defined() && t->numel() > 0) t->record_stream(s);
  }
  c10::cuda::CUDAStream current_;
  std::optional<c10::cuda::CUDAStreamGuard> other_;
  void *ptr_;
};

// ------------------------------------------------------------------- operands

int device_of(const Tensor &t, const char *what) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", what);
  return t.get_device();
}
void on_device(const Tensor &t, int dev, const char *what) {
  if (!t.is_cuda() || t.get_device() != dev)
    fail(PyExc_ValueError, "%s must be a CUDA tensor on the operands' device", what);
}

// A matrix with contiguous rows.
struct Rows {
  int64_t rows, cols, ld;
  Rows(const Tensor &t, const char *what) {
    if (t.dim() != 2) fail(PyExc_ValueError, "%s must be 2-D", what);
    rows = t.size(0), cols = t.size(1);
    const int64_t s0 = t.stride(0), s1 = t.stride(1);
    if ((s1 != 1 && cols > 1) || (s0 < cols && rows > 1))
      fail(PyExc_ValueError, "rows of %s must be contiguous", what);
    ld = rows > 1 ? s0 : cols > 0 ? cols : 1;
  }
};
int64_t row_ld(const Tensor &t, int64_t rows, int64_t cols, const char *what, int dev) {
  const Rows r(t, what);
  if (r.rows != rows || r.cols != cols)
    fail(PyExc_ValueError, "%s must be a %lld x %lld tensor, got %lld x %lld", what,
                     static_cast<long long>(rows), static_cast<long long>(cols),
                     static_cast<long long>(r.rows), static_cast<long long>(r.cols));
  on_device(t, dev, what);
  return r.ld;
}

// A row- or column-major operand (the rule of the ctypes binding's operand_layout; a single row
// or column may also have any stride along itself).
struct Layout {
  gemm_layout_t layout;
  int64_t ld;
  explicit Layout(const Tensor &t) : Layout(t.size(0), t.size(1), t.stride(0), t.stride(1)) {}
  Layout(int64_t r, int64_t c, int64_t s0, int64_t s1) {
    auto most = [](int64_t a, int64_t b) { return a > b ? a : b; };
    if (s1 == 1 && (s0 >= most(c, 1) || r <= 1)) {
      layout = GEMM_ROW_MAJOR, ld = most(most(s0, c), 1);
    } else if (s0 == 1 && (s1 >= most(r, 1) || c <= 1)) {
      layout = GEMM_COL_MAJOR, ld = most(most(s1, r), 1);
    } else if (c == 1 && s0 >= 1) {
      layout = GEMM_ROW_MAJOR, ld = s0;
    } else if (r == 1 && s1 >= 1) {
      layout = GEMM_COL_MAJOR, ld = s1;
    } else {
      fail(PyExc_ValueError, "operand must be row- or column-major, got stride (%lld, %lld)",
                       static_cast<long long>(s0), static_cast<long long>(s1));
    }
  }
  // The same operand in the other layout, where a single row or column of it has both.
  void become(gemm_layout_t other, const Tensor &t) {
    if (layout == other) return;
    if (other == GEMM_COL_MAJOR ? t.size(0) != 1 : t.size(1) != 1) return;
    layout = other, ld = most1(t.stride(other == GEMM_COL_MAJOR ? 1 : 0));
  }

 private:
  static int64_t most1(int64_t v) { return v > 1 ? v : 1; }
};

const void *vector(const Tensor &t, int64_t n, const char *what, int dev) {
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be a contiguous vector of %lld values", what, static_cast<long long>(n));
  on_device(t, dev, what);
  return t.data_ptr();
}

Tensor empty(const Tensor &like, at::IntArrayRef sizes, at::ScalarType t) {
  return at::empty(sizes, like.options().dtype(t));
}
int64_t least1(int64_t v) { return v > 0 ? v : 1; }
// An empty tensor of t's shape, tight in the layout t was read in, and its leading dimension. (The
// layout cannot be read back from the new tensor: a matrix of one row or column has both.)
Tensor empty_like_layout(const Tensor &t, gemm_layout_t layout) {
  if (layout == GEMM_ROW_MAJOR) return empty(t, {t.size(0), t.size(1)}, t.scalar_type());
  return empty(t, {t.size(1), t.size(0)}, t.scalar_type()).t();
}
int64_t tight_ld(gemm_layout_t layout, int64_t rows, int64_t cols) {
  return least1(layout == GEMM_ROW_MAJOR ? cols : rows);
}

struct Product {
  int64_t M, N, K;
  int dev;
  Product(const Tensor &a, const Tensor &b) {
    if (!a.is_cuda() || !b.is_cuda() || a.get_device() != b.get_device())
      fail(PyExc_ValueError, "operands must be CUDA tensors on one device");
    if (a.scalar_type() != b.scalar_type()) fail(PyExc_TypeError, "operands must share a dtype");
    if (a.dim() != 2 || b.dim() != 2) fail(PyExc_ValueError, "operands must be 2-D");
    if (a.size(1) != b.size(0))
      fail(PyExc_ValueError, "inner dimensions differ: %lld vs %lld", static_cast<long long>(a.size(1)),
                       static_cast<long long>(b.size(0)));
    M = a.size(0), N = b.size(1), K = a.size(1);
    dev = a.get_device();
  }
};

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject *wrap(const Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject *wrap3(const Tensor &a, const Tensor &b, const Tensor &c) {
  PyObject *r = PyTuple_New(3);
  if (!r) return nullptr;
  const Tensor *t[3] = {&a, &b, &c};
  for (int i = 0; i < 3; ++i) {
    PyObject *o = wrap(*t[i]);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

void check(gemm_status_t st, const char *name) {
  if (st == GEMM_OK) return;
  PyObject *r = PyObject_CallFunction(raise_status, "is", static_cast<int>(st), name);
  Py_XDECREF(r);
  throw python_error();
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "expected %lld arguments, got %lld", static_cast<long long>(want),
                                 static_cast<long long>(n));
}

// ------------------------------------------------------------------- operators

// handle, a, b, bias, activation, residual, out, out_dtype, precision, save, stream
PyObject *matmul_epilogue(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const Tensor a = tensor(v[1], "a"), b = tensor(v[2], "b");
  const Product p(a, b);
  const int in = code_of(a);
  Tensor out;
  at::ScalarType od;
  int64_t ldc;
  if (v[6] != Py_None) {
    out = tensor(v[6], "out");
    od = out.scalar_type();
    ldc = row_ld(out, p.M, p.N, "out", p.dev);
  } else {
    od = dtype_arg(v[7], a.scalar_type());
    ldc = least1(p.N);
  }
  gemm_epilogue_t ep;
  std::memset(&ep, 0, sizeof ep);
  ep.activation = activation_arg(v[4]);
  Tensor bias, residual, pre;
  if (v[3] != Py_None) {
    bias = tensor(v[3], "bias");
    ep.bias = vector(bias, p.N, "bias", p.dev);
    ep.bias_dtype = code_of(bias);
  }
  if (v[5] != Py_None) {
    residual = tensor(v[5], "residual");
    if (residual.scalar_type() != od) fail(PyExc_TypeError, "residual must have the output's dtype");
    ep.ld_residual = row_ld(residual, p.M, p.N, "residual", p.dev);
    ep.residual = residual.data_ptr();
  }
  const Layout la(a), lb(b);
  const gemm_precision_t prec = precision_arg(v[8]);
  const bool save = truth(v[9]);
  const CallStream stream(v[10], p.dev);
  stream.uses({&a, &b, &bias, &residual, &out});
  if (!out.defined()) out = empty(a, {p.M, p.N}, od);
  if (save) {
    pre = empty(a, {p.M, p.N}, od);
    ep.pre = pre.data_ptr();
    ep.ld_pre = least1(p.N);
  }
  check(run_epilogue(handle_arg(v[0]), p.M, p.N, p.K, a.data_ptr(), la.ld, b.data_ptr(), lb.ld,
                     out.data_ptr(), ldc, static_cast<gemm_dtype_t>(in),
                     static_cast<gemm_dtype_t>(code_of(od)), prec, la.layout, lb.layout, &ep, stream.get()),
        "gemm_run_epilogue");
  stream.gives({&out, &pre});
  if (!save) return wrap(out);
  PyObject *x = wrap(out), *y = wrap(pre);
  return x && y ? Py_BuildValue("(NN)", x, y) : nullptr;
  END_HANDLE_TH_ERRORS
}

// handle, grad, a, b, pre, activation, need, bias_dtype, precision, stream
PyObject *matmul_epilogue_backward(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor grad = tensor(v[1], "grad"), a = tensor(v[2], "a"), b = tensor(v[3], "b");
  const Product p(a, b);
  const gemm_activation_t act = activation_arg(v[5]);
  const int64_t lddy = row_ld(grad, p.M, p.N, "grad", p.dev);
  Tensor pre;
  int64_t ldz = 0;
  if (act != GEMM_ACT_NONE) {
    if (v[4] == Py_None) fail(PyExc_ValueError, "the backward pass of an activation needs the saved pre");
    pre = tensor(v[4], "pre");
    if (pre.scalar_type() != grad.scalar_type()) fail(PyExc_TypeError, "pre must have grad's dtype");
    ldz = row_ld(pre, p.M, p.N, "pre", p.dev);
  }
  const Need need(v[6]);
  const at::ScalarType bd = dtype_arg(v[7], a.scalar_type());
  const gemm_precision_t prec = precision_arg(v[8]);
  const Layout la(a), lb(b);
  const CallStream stream(v[9], p.dev);
  stream.uses({&grad, &a, &b, &pre});
  Tensor da, db, dbias;
  if (need.v[0]) da = empty_like_layout(a, la.layout);
  if (need.v[1]) db = empty_like_layout(b, lb.layout);
  if (need.v[2]) dbias = empty(a, {p.N}, bd);
  check(run_epilogue_backward(
            handle_arg(v[0]), p.M, p.N, p.K, grad.data_ptr(), lddy, ptr(pre), ldz, a.data_ptr(),
            la.ld, b.data_ptr(), lb.ld, ptr(da), tight_ld(la.layout, p.M, p.K), ptr(db),
            tight_ld(lb.layout, p.K, p.N), ptr(dbias), static_cast<gemm_dtype_t>(code_of(bd)),
            static_cast<gemm_dtype_t>(code_of(a)), static_cast<gemm_dtype_t>(code_of(grad)), prec,
            la.layout, lb.layout, act, stream.get()),
        "gemm_run_epilogue_backward");
  stream.gives({&da, &db, &dbias});
  return wrap3(da, db, dbias);
  END_HANDLE_TH_ERRORS
}

// The operands of a gated pair.
struct Gated {
  Product p;
  int64_t ldx;
  Layout g, u;
  Gated(const Tensor &x, const Tensor &wg, const Tensor &wu)
      : p(x, wg), ldx(Rows(x, "x").ld), g(wg), u((Product(x, wu), wu)) {
    if (wu.size(1) != p.N) fail(PyExc_ValueError, "w_gate and w_up must have one shape");
    g.become(u.layout, wg);
    u.become(g.layout, wu);
    if (g.layout != u.layout) fail(PyExc_ValueError, "w_gate and w_up must have one layout");
  }
};

// handle, x, w_gate, w_up, activation, out, precision, save, stream
PyObject *gated(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor x = tensor(v[1], "x"), wg = tensor(v[2], "w_gate"), wu = tensor(v[3], "w_up");
  const Gated q(x, wg, wu);
  const Product &p = q.p;
  const gemm_activation_t act = activation_arg(v[4]);
  const gemm_precision_t prec = precision_arg(v[6]);
  const bool save = truth(v[7]);
  const auto dt = static_cast<gemm_dtype_t>(code_of(x));
  const CallStream stream(v[8], p.dev);
  Tensor out, gate, up;
  int64_t ldh = least1(p.N);
  if (v[5] != Py_None) {
    out = tensor(v[5], "out");
    if (out.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    ldh = row_ld(out, p.M, p.N, "out", p.dev);
  }
  stream.uses({&x, &wg, &wu, &out});
  if (!out.defined()) out = empty(x, {p.M, p.N}, x.scalar_type());
  if (save) {  // column ranges of one buffer, as the backward pass keeps their gradients
    const Tensor both = empty(x, {p.M, 2 * p.N}, x.scalar_type());
    gate = both.narrow(1, 0, p.N);
    up = both.narrow(1, p.N, p.N);
  }
  check(run_gated(handle_arg(v[0]), p.M, p.N, p.K, x.data_ptr(), q.ldx, wg.data_ptr(), q.g.ld,
                  wu.data_ptr(), q.u.ld, out.data_ptr(), ldh, ptr(gate), 2 * p.N, ptr(up), 2 * p.N,
                  dt, prec, q.g.layout, act, stream.get()),
        "gemm_run_gated");
  stream.gives({&out, &gate, &up});
  return save ? wrap3(out, gate, up) : wrap(out);
  END_HANDLE_TH_ERRORS
}

// handle, grad, x, w_gate, w_up, gate, up, activation, need, precision, stream
PyObject *gated_backward(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const Tensor grad = tensor(v[1], "grad"), x = tensor(v[2], "x"), wg = tensor(v[3], "w_gate"),
               wu = tensor(v[4], "w_up"), gate = tensor(v[5], "gate"), up = tensor(v[6], "up");
  const Gated q(x, wg, wu);
  const Product &p = q.p;
  for (const Tensor *t : {&grad, &gate, &up})
    if (t->scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "grad, gate and up must have x's dtype");
  const int64_t ldh = row_ld(grad, p.M, p.N, "grad", p.dev);
  const int64_t ldg = row_ld(gate, p.M, p.N, "gate", p.dev), ldu = row_ld(up, p.M, p.N, "up", p.dev);
  const gemm_activation_t act = activation_arg(v[7]);
  const Need need(v[8]);
  const gemm_precision_t prec = precision_arg(v[9]);
  const auto dt = static_cast<gemm_dtype_t>(code_of(x));
  const CallStream stream(v[10], p.dev);
  stream.uses({&grad, &x, &wg, &wu, &gate, &up});
  Tensor dx, dwg, dwu;
  if (need.v[0]) dx = empty(x, {p.M, p.K}, x.scalar_type());
  if (need.v[1] && need.v[2] && q.g.layout == GEMM_COL_MAJOR) {
    // one buffer, so that both gradients are one product
    const Tensor both = empty(x, {2 * p.N, p.K}, x.scalar_type());
    dwg = both.narrow(0, 0, p.N).t();
    dwu = both.narrow(0, p.N, p.N).t();
  } else {
    if (need.v[1]) dwg = empty_like_layout(wg, q.g.layout);
    if (need.v[2]) dwu = empty_like_layout(wu, q.u.layout);
  }
  const int64_t ldw = tight_ld(q.g.layout, p.K, p.N);
  check(run_gated_backward(handle_arg(v[0]), p.M, p.N, p.K, grad.data_ptr(), ldh, gate.data_ptr(),
                           ldg, up.data_ptr(), ldu, x.data_ptr(), q.ldx, wg.data_ptr(), q.g.ld,
                           wu.data_ptr(), q.u.ld, ptr(dx), least1(p.K), ptr(dwg), ldw, ptr(dwu), ldw,
                           dt, prec, q.g.layout, act, stream.get()),
        "gemm_run_gated_backward");
  stream.gives({&dx, &dwg, &dwu});
  return wrap3(dx, dwg, dwu);
  END_HANDLE_TH_ERRORS
}

// handle, x, weight, bias, eps, out, out_dtype, save, stream
PyObject *layer_norm(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor x = tensor(v[1], "x");
  const int dev = device_of(x, "x");
  const Rows r(x, "x");
  const int in = code_of(x);
  Tensor weight, bias, out, mean, rstd;
  const void *wp = nullptr, *bp = nullptr;
  int params = GEMM_F32;
  if (v[3] != Py_None) {
    bias = tensor(v[3], "bias");
    bp = vector(bias, r.cols, "bias", dev);
    params = code_of(bias);
  }
  if (v[2] != Py_None) {
    weight = tensor(v[2], "weight");
    wp = vector(weight, r.cols, "weight", dev);
    params = code_of(weight);
    if (bias.defined() && bias.scalar_type() != weight.scalar_type())
      fail(PyExc_TypeError, "weight and bias must share a dtype");
  }
  const double eps = PyFloat_AsDouble(v[4]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  int64_t ldy = least1(r.cols);
  if (v[5] != Py_None) {
    out = tensor(v[5], "out");
    ldy = row_ld(out, r.rows, r.cols, "out", dev);
  }
  const bool save = truth(v[7]);
  const CallStream stream(v[8], dev);
  stream.uses({&x, &weight, &bias, &out});
  if (!out.defined()) out = empty(x, {r.rows, r.cols}, dtype_arg(v[6], x.scalar_type()));
  if (save) {
    const Tensor both = empty(x, {2, r.rows}, at::kFloat);
    mean = both.select(0, 0);
    rstd = both.select(0, 1);
  }
  check(run_layer_norm(handle_arg(v[0]), r.rows, r.cols, x.data_ptr(), r.ld, wp, bp, out.data_ptr(),
                       ldy, static_cast<float *>(ptr(mean)), static_cast<float *>(ptr(rstd)),
                       static_cast<float>(eps), static_cast<gemm_dtype_t>(in),
                       static_cast<gemm_dtype_t>(params), static_cast<gemm_dtype_t>(code_of(out)),
                       stream.get()),
        "gemm_layer_norm");
  stream.gives({&out, &mean, &rstd});
  return save ? wrap3(out, mean, rstd) : wrap(out);
  END_HANDLE_TH_ERRORS
}

// handle, grad, x, weight, mean, rstd, need, param_dtype, stream
PyObject *layer_norm_backward(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor grad = tensor(v[1], "grad"), x = tensor(v[2], "x");
  const int dev = device_of(x, "x");
  const Rows r(x, "x");
  const int64_t lddy = row_ld(grad, r.rows, r.cols, "grad", dev);
  const Tensor mean = tensor(v[4], "mean"), rstd = tensor(v[5], "rstd");
  if (mean.scalar_type() != at::kFloat || rstd.scalar_type() != at::kFloat)
    fail(PyExc_TypeError, "mean and rstd must be float32");
  const float *mp = static_cast<const float *>(vector(mean, r.rows, "mean", dev));
  const float *rp = static_cast<const float *>(vector(rstd, r.rows, "rstd", dev));
  at::ScalarType pd = at::kFloat;
  const void *wp = nullptr;
  Tensor weight;
  if (v[3] != Py_None) {
    weight = tensor(v[3], "weight");
    wp = vector(weight, r.cols, "weight", dev);
    pd = weight.scalar_type();
  }
  if (v[7] != Py_None) {
    const at::ScalarType asked = dtype_arg(v[7], pd);
    if (weight.defined() && asked != pd) fail(PyExc_TypeError, "param_dtype must be weight's dtype");
    pd = asked;
  }
  const Need need(v[6]);
  const int in = code_of(x), params = code_of(pd), g = code_of(grad);
  const CallStream stream(v[8], dev);
  stream.uses({&grad, &x, &weight, &mean, &rstd});
  Tensor dx, dw, db;
  if (need.v[0]) dx = empty(x, {r.rows, r.cols}, x.scalar_type());
  if (need.v[1]) dw = empty(x, {r.cols}, pd);
  if (need.v[2]) db = empty(x, {r.cols}, pd);
  check(run_layer_norm_backward(handle_arg(v[0]), r.rows, r.cols, grad.data_ptr(), lddy,
                                x.data_ptr(), r.ld, wp, mp, rp, ptr(dx), least1(r.cols), ptr(dw),
                                ptr(db), static_cast<gemm_dtype_t>(in),
                                static_cast<gemm_dtype_t>(params), static_cast<gemm_dtype_t>(g),
                                stream.get()),
        "gemm_layer_norm_backward");
  stream.gives({&dx, &dw, &db});
  return wrap3(dx, dw, db);
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------- operators of experts

// The tokens' positions: int32, tokens x k.
struct Pairs {
  int64_t tokens, k;
  int dev;
  const int32_t *ptr;
  explicit Pairs(const Tensor &t) {
    dev = device_of(t, "position");
    if (t.scalar_type() != at::kInt) fail(PyExc_TypeError, "position must be int32");
    if (t.dim() != 2 || !t.is_contiguous())
      fail(PyExc_ValueError, "position must be a contiguous tokens x k tensor");
    tokens = t.size(0), k = t.size(1);
    ptr = static_cast<const int32_t *>(t.data_ptr());
  }
};
// One value for every pair.
const void *pair_values(const Tensor &t, const Pairs &p, const char *what) {
  if (t.dim() != 2 || t.size(0) != p.tokens || t.size(1) != p.k || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be a contiguous %lld x %lld tensor", what,
         static_cast<long long>(p.tokens), static_cast<long long>(p.k));
  on_device(t, p.dev, what);
  return t.data_ptr();
}
gemm_dtype_t type_of(const Tensor &t) { return static_cast<gemm_dtype_t>(code_of(t)); }

// handle, ids, experts, stream
PyObject *expert_sort(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  const Tensor ids = tensor(v[1], "ids");
  const int dev = device_of(ids, "ids");
  if (ids.scalar_type() != at::kLong && ids.scalar_type() != at::kInt)
    fail(PyExc_TypeError, "ids must be int64 or int32");
  const Rows r(ids, "ids");
  const long long experts = PyLong_AsLongLong(v[2]);
  if (experts == -1 && PyErr_Occurred()) throw python_error();
  if (experts < 1) fail(PyExc_ValueError, "experts must be at least 1");
  const CallStream stream(v[3], dev);
  stream.uses({&ids});
  const Tensor position = empty(ids, {r.rows, r.cols}, at::kInt);
  const Tensor offsets = empty(ids, {experts + 1}, at::kInt);
  check(run_expert_sort(handle_arg(v[0]), r.rows, r.cols, experts, ids.data_ptr(), r.ld,
                        static_cast<int32_t>(ids.element_size()),
                        static_cast<int32_t *>(position.data_ptr()),
                        static_cast<int32_t *>(offsets.data_ptr()), stream.get()),
        "gemm_expert_sort");
  stream.gives({&position, &offsets});
  PyObject *a = wrap(position), *b = wrap(offsets);
  return a && b ? Py_BuildValue("(NN)", a, b) : nullptr;
  END_HANDLE_TH_ERRORS
}

// handle, x, position, out, stream
PyObject *expert_gather(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  const Tensor x = tensor(v[1], "x"), position = tensor(v[2], "position");
  const Pairs p(position);
  const Rows r(x, "x");
  on_device(x, p.dev, "x");
  if (r.rows != p.tokens) fail(PyExc_ValueError, "x and position must have one row a token");
  const gemm_dtype_t dt = type_of(x);
  Tensor out;
  int64_t rows = p.tokens * p.k, ldy = least1(r.cols);
  if (v[3] != Py_None) {
    out = tensor(v[3], "out");
    if (out.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    if (out.dim() != 2) fail(PyExc_ValueError, "out must be 2-D");
    rows = out.size(0);
    ldy = row_ld(out, rows, r.cols, "out", p.dev);
  }
  const CallStream stream(v[4], p.dev);
  stream.uses({&x, &position, &out});
  if (!out.defined()) out = empty(x, {rows, r.cols}, x.scalar_type());
  check(run_expert_gather(handle_arg(v[0]), p.tokens, p.k, r.cols, x.data_ptr(), r.ld, p.ptr, rows,
                          out.data_ptr(), ldy, dt, stream.get()),
        "gemm_expert_gather");
  stream.gives({&out});
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// handle, rows, position, weights, residual, out, out_dtype, stream
PyObject *expert_combine(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Tensor z = tensor(v[1], "rows"), position = tensor(v[2], "position");
  const Pairs p(position);
  const Rows r(z, "rows");
  on_device(z, p.dev, "rows");
  const gemm_dtype_t in = type_of(z);
  Tensor weights, residual, out;
  const void *wp = nullptr;
  gemm_dtype_t wd = GEMM_F32;
  if (v[3] != Py_None) {
    weights = tensor(v[3], "weights");
    wp = pair_values(weights, p, "weights");
    wd = type_of(weights);
  }
  at::ScalarType od;
  int64_t ldy = least1(r.cols), ldr = 0;
  if (v[5] != Py_None) {
    out = tensor(v[5], "out");
    od = out.scalar_type();
    code_of(od);
    ldy = row_ld(out, p.tokens, r.cols, "out", p.dev);
  } else {
    od = dtype_arg(v[6], z.scalar_type());
  }
  if (v[4] != Py_None) {
    residual = tensor(v[4], "residual");
    if (residual.scalar_type() != od) fail(PyExc_TypeError, "residual must have the output's dtype");
    ldr = row_ld(residual, p.tokens, r.cols, "residual", p.dev);
  }
  const CallStream stream(v[7], p.dev);
  stream.uses({&z, &position, &weights, &residual, &out});
  if (!out.defined()) out = empty(z, {p.tokens, r.cols}, od);
  check(run_expert_combine(handle_arg(v[0]), p.tokens, p.k, r.cols, z.data_ptr(), r.ld, r.rows, p.ptr,
                           wp, wd, ptr(residual), ldr, out.data_ptr(), ldy, in,
                           static_cast<gemm_dtype_t>(code_of(od)), stream.get()),
        "gemm_expert_combine");
  stream.gives({&out});
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// handle, grad, rows, position, weights, need, out, stream
PyObject *expert_combine_backward(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Tensor grad = tensor(v[1], "grad"), z = tensor(v[2], "rows"), position = tensor(v[3], "position");
  const Pairs p(position);
  const Rows r(z, "rows");
  on_device(z, p.dev, "rows");
  const int64_t lddy = row_ld(grad, p.tokens, r.cols, "grad", p.dev);
  const gemm_dtype_t in = type_of(z), gt = type_of(grad);
  if (!PyTuple_Check(v[5]) || PyTuple_GET_SIZE(v[5]) != 2)
    fail(PyExc_ValueError, "need must be a tuple of two truth values");
  const bool need_rows = truth(PyTuple_GET_ITEM(v[5], 0));
  bool need_weights = truth(PyTuple_GET_ITEM(v[5], 1));
  Tensor weights, dz, dw;
  const void *wp = nullptr;
  gemm_dtype_t wd = GEMM_F32;
  if (v[4] != Py_None) {
    weights = tensor(v[4], "weights");
    wp = pair_values(weights, p, "weights");
    wd = type_of(weights);
  } else {
    need_weights = false;
  }
  int64_t ldd = least1(r.cols);
  if (need_rows && v[6] != Py_None) {
    dz = tensor(v[6], "out");
    if (dz.scalar_type() != z.scalar_type()) fail(PyExc_TypeError, "out must have rows' dtype");
    ldd = row_ld(dz, r.rows, r.cols, "out", p.dev);
  }
  const CallStream stream(v[7], p.dev);
  stream.uses({&grad, &z, &position, &weights, &dz});
  if (need_rows && !dz.defined()) dz = empty(z, {r.rows, r.cols}, z.scalar_type());
  if (need_weights) dw = empty(z, {p.tokens, p.k}, weights.scalar_type());
  check(run_expert_combine_backward(handle_arg(v[0]), p.tokens, p.k, r.cols, grad.data_ptr(), lddy,
                                    z.data_ptr(), r.ld, r.rows, p.ptr, wp, wd, ptr(dz), ldd, ptr(dw),
                                    in, gt, stream.get()),
        "gemm_expert_combine_backward");
  stream.gives({&dz, &dw});
  PyObject *a = wrap(dz), *b = wrap(dw);
  return a && b ? Py_BuildValue("(NN)", a, b) : nullptr;
  END_HANDLE_TH_ERRORS
}

// The experts' weights: experts x K x N, each K x N row- or column-major.
struct Weights {
  int64_t experts, K, N, stride;
  Layout layout;
  explicit Weights(const Tensor &w)
      : experts(w.dim() == 3 ? w.size(0) : 0),
        K(w.dim() == 3 ? w.size(1) : 0),
        N(w.dim() == 3 ? w.size(2) : 0),
        stride(w.dim() == 3 ? w.stride(0) : 0),
        layout(w.dim() == 3 ? Layout(K, N, w.stride(1), w.stride(2)) : Layout(0, 0, 1, 1)) {
    if (w.dim() != 3) fail(PyExc_ValueError, "weights must be 3-D (experts x inputs x outputs)");
    if (experts < 1) fail(PyExc_ValueError, "weights must have at least one expert");
  }
  // A gradient of the weights' shape in their layout, tight.
  Tensor gradient(const Tensor &w) const {
    if (layout.layout == GEMM_ROW_MAJOR) return empty(w, {experts, K, N}, w.scalar_type());
    return empty(w, {experts, N, K}, w.scalar_type()).transpose(1, 2);
  }
  int64_t gradient_ld() const { return tight_ld(layout.layout, K, N); }
  int64_t gradient_stride() const { return K * N; }
};

// The operands of an expert product: rows (rows x K), weights, offsets.
struct ExpertOperands {
  Weights w;
  int dev;
  int64_t rows, ldx;
  const int32_t *offsets;
  gemm_dtype_t dt;
  ExpertOperands(const Tensor &x, const Tensor &wt, const Tensor &o) : w(wt) {
    dev = device_of(x, "x");
    on_device(wt, dev, "weights");
    if (x.scalar_type() != wt.scalar_type()) fail(PyExc_TypeError, "operands must share a dtype");
    dt = type_of(x);
    const Rows r(x, "x");
    if (r.cols != w.K)
      fail(PyExc_ValueError, "inner dimensions differ: %lld vs %lld", static_cast<long long>(r.cols),
           static_cast<long long>(w.K));
    rows = r.rows, ldx = r.ld;
    if (o.scalar_type() != at::kInt) fail(PyExc_TypeError, "offsets must be int32");
    offsets = static_cast<const int32_t *>(vector(o, w.experts + 1, "offsets", dev));
  }
};

// handle, x, w, offsets, out, stream
PyObject *expert_matmul(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  const Tensor x = tensor(v[1], "x"), w = tensor(v[2], "w"), offsets = tensor(v[3], "offsets");
  const ExpertOperands q(x, w, offsets);
  Tensor out;
  int64_t ldy = least1(q.w.N);
  if (v[4] != Py_None) {
    out = tensor(v[4], "out");
    if (out.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    ldy = row_ld(out, q.rows, q.w.N, "out", q.dev);
  }
  const CallStream stream(v[5], q.dev);
  stream.uses({&x, &w, &offsets, &out});
  if (!out.defined()) out = empty(x, {q.rows, q.w.N}, x.scalar_type());
  check(run_expert(handle_arg(v[0]), q.w.experts, q.rows, q.w.N, q.w.K, x.data_ptr(), q.ldx, w.data_ptr(),
                   q.w.layout.ld, q.w.stride, q.offsets, out.data_ptr(), ldy, q.dt, q.w.layout.layout,
                   stream.get()),
        "gemm_run_expert");
  stream.gives({&out});
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// handle, grad, x, w, offsets, need, out, stream
PyObject *expert_matmul_backward(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Tensor grad = tensor(v[1], "grad"), x = tensor(v[2], "x"), w = tensor(v[3], "w"),
               offsets = tensor(v[4], "offsets");
  const ExpertOperands q(x, w, offsets);
  if (grad.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "grad must have x's dtype");
  const int64_t lddy = row_ld(grad, q.rows, q.w.N, "grad", q.dev);
  if (!PyTuple_Check(v[5]) || PyTuple_GET_SIZE(v[5]) != 2)
    fail(PyExc_ValueError, "need must be a tuple of two truth values");
  const bool need_x = truth(PyTuple_GET_ITEM(v[5], 0)), need_w = truth(PyTuple_GET_ITEM(v[5], 1));
  Tensor dx, dw;
  int64_t lddx = least1(q.w.K);
  if (need_x && v[6] != Py_None) {
    dx = tensor(v[6], "out");
    if (dx.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    lddx = row_ld(dx, q.rows, q.w.K, "out", q.dev);
  }
  const CallStream stream(v[7], q.dev);
  stream.uses({&grad, &x, &w, &offsets, &dx});
  if (need_x && !dx.defined()) dx = empty(x, {q.rows, q.w.K}, x.scalar_type());
  if (need_w) dw = q.w.gradient(w);
  check(run_expert_backward(handle_arg(v[0]), q.w.experts, q.rows, q.w.N, q.w.K, grad.data_ptr(), lddy,
                            x.data_ptr(), q.ldx, w.data_ptr(), q.w.layout.ld, q.w.stride, q.offsets,
                            ptr(dx), lddx, ptr(dw), q.w.gradient_ld(), q.w.gradient_stride(), q.dt,
                            q.w.layout.layout, stream.get()),
        "gemm_run_expert_backward");
  stream.gives({&dx, &dw});
  PyObject *a = wrap(dx), *b = wrap(dw);
  return a && b ? Py_BuildValue("(NN)", a, b) : nullptr;
  END_HANDLE_TH_ERRORS
}

// The operands of the experts' gated pair.
struct ExpertGated {
  ExpertOperands q;
  Weights u;
  ExpertGated(const Tensor &x, const Tensor &wg, const Tensor &wu, const Tensor &offsets)
      : q(x, wg, offsets), u(wu) {
    if (wu.scalar_type() != wg.scalar_type()) fail(PyExc_TypeError, "operands must share a dtype");
    on_device(wu, q.dev, "w_up");
    if (u.experts != q.w.experts || u.K != q.w.K || u.N != q.w.N)
      fail(PyExc_ValueError, "w_gate and w_up must have one shape");
    if (u.layout.layout != q.w.layout.layout) {  // (a single row or column has both layouts)
      const Tensor g0 = wg.select(0, 0), u0 = wu.select(0, 0);
      q.w.layout.become(u.layout.layout, g0);
      u.layout.become(q.w.layout.layout, u0);
    }
    if (u.layout.layout != q.w.layout.layout)
      fail(PyExc_ValueError, "w_gate and w_up must have one layout");
  }
};

// handle, x, w_gate, w_up, offsets, activation, out, save, stream
PyObject *expert_gated(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor x = tensor(v[1], "x"), wg = tensor(v[2], "w_gate"), wu = tensor(v[3], "w_up"),
               offsets = tensor(v[4], "offsets");
  const ExpertGated e(x, wg, wu, offsets);
  const ExpertOperands &q = e.q;
  const int64_t F = q.w.N;
  const gemm_activation_t act = activation_arg(v[5]);
  const bool save = truth(v[7]);
  Tensor out, gate, up;
  int64_t ldh = least1(F);
  if (v[6] != Py_None) {
    out = tensor(v[6], "out");
    if (out.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    ldh = row_ld(out, q.rows, F, "out", q.dev);
  }
  const CallStream stream(v[8], q.dev);
  stream.uses({&x, &wg, &wu, &offsets, &out});
  if (!out.defined()) out = empty(x, {q.rows, F}, x.scalar_type());
  if (save) {  // column ranges of one buffer
    const Tensor both = empty(x, {q.rows, 2 * F}, x.scalar_type());
    gate = both.narrow(1, 0, F);
    up = both.narrow(1, F, F);
  }
  check(run_expert_gated(handle_arg(v[0]), q.w.experts, q.rows, F, q.w.K, x.data_ptr(), q.ldx,
                         wg.data_ptr(), q.w.layout.ld, q.w.stride, wu.data_ptr(), e.u.layout.ld,
                         e.u.stride, q.offsets, out.data_ptr(), ldh, ptr(gate), 2 * F, ptr(up), 2 * F,
                         q.dt, q.w.layout.layout, act, stream.get()),
        "gemm_run_expert_gated");
  stream.gives({&out, &gate, &up});
  return save ? wrap3(out, gate, up) : wrap(out);
  END_HANDLE_TH_ERRORS
}

// handle, grad, x, w_gate, w_up, gate, up, offsets, activation, need, out, stream
PyObject *expert_gated_backward(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Tensor grad = tensor(v[1], "grad"), x = tensor(v[2], "x"), wg = tensor(v[3], "w_gate"),
               wu = tensor(v[4], "w_up"), gate = tensor(v[5], "gate"), up = tensor(v[6], "up"),
               offsets = tensor(v[7], "offsets");
  const ExpertGated e(x, wg, wu, offsets);
  const ExpertOperands &q = e.q;
  const int64_t F = q.w.N;
  for (const Tensor *t : {&grad, &gate, &up})
    if (t->scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "grad, gate and up must have x's dtype");
  const int64_t lddh = row_ld(grad, q.rows, F, "grad", q.dev);
  const int64_t ldg = row_ld(gate, q.rows, F, "gate", q.dev), ldu = row_ld(up, q.rows, F, "up", q.dev);
  const gemm_activation_t act = activation_arg(v[8]);
  const Need need(v[9]);
  Tensor dx, dwg, dwu;
  int64_t lddx = least1(q.w.K);
  if (need.v[0] && v[10] != Py_None) {
    dx = tensor(v[10], "out");
    if (dx.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    lddx = row_ld(dx, q.rows, q.w.K, "out", q.dev);
  }
  const CallStream stream(v[11], q.dev);
  stream.uses({&grad, &x, &wg, &wu, &gate, &up, &offsets, &dx});
  if (need.v[0] && !dx.defined()) dx = empty(x, {q.rows, q.w.K}, x.scalar_type());
  if (need.v[1]) dwg = q.w.gradient(wg);
  if (need.v[2]) dwu = e.u.gradient(wu);
  const int64_t ldw = q.w.gradient_ld(), step = q.w.gradient_stride();
  check(run_expert_gated_backward(
            handle_arg(v[0]), q.w.experts, q.rows, F, q.w.K, grad.data_ptr(), lddh, gate.data_ptr(), ldg,
            up.data_ptr(), ldu, x.data_ptr(), q.ldx, wg.data_ptr(), q.w.layout.ld, q.w.stride,
            wu.data_ptr(), e.u.layout.ld, e.u.stride, q.offsets, ptr(dx), lddx, ptr(dwg), ldw, step,
            ptr(dwu), ldw, step, q.dt, q.w.layout.layout, act, stream.get()),
        "gemm_run_expert_gated_backward");
  stream.gives({&dx, &dwg, &dwu});
  return wrap3(dx, dwg, dwu);
  END_HANDLE_TH_ERRORS
}

// handle, x, p, key, residual, out, stream
PyObject *dropout(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const Tensor x = tensor(v[1], "x"), key = tensor(v[3], "key");
  const int dev = device_of(x, "x");
  const Rows r(x, "x");
  const gemm_dtype_t dt = type_of(x);
  const double p = PyFloat_AsDouble(v[2]);
  if (p == -1.0 && PyErr_Occurred()) throw python_error();
  if (key.scalar_type() != at::kLong) fail(PyExc_TypeError, "key must be int64");
  const void *kp = vector(key, 2, "key", dev);
  Tensor residual, out;
  int64_t ldr = 0, ldy = least1(r.cols);
  if (v[4] != Py_None) {
    residual = tensor(v[4], "residual");
    if (residual.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "residual must have x's dtype");
    ldr = row_ld(residual, r.rows, r.cols, "residual", dev);
  }
  if (v[5] != Py_None) {
    out = tensor(v[5], "out");
    if (out.scalar_type() != x.scalar_type()) fail(PyExc_TypeError, "out must have x's dtype");
    ldy = row_ld(out, r.rows, r.cols, "out", dev);
  }
  const CallStream stream(v[6], dev);
  stream.uses({&x, &key, &residual, &out});
  if (!out.defined()) out = empty(x, {r.rows, r.cols}, x.scalar_type());
  check(run_dropout(handle_arg(v[0]), r.rows, r.cols, x.data_ptr(), r.ld, ptr(residual), ldr,
                    out.data_ptr(), ldy, p, static_cast<const uint64_t *>(kp), dt, stream.get()),
        "gemm_dropout");
  stream.gives({&out});
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// Addresses of the C functions, in the order of the operators above, and the callable that
// raises a status code.
PyObject *init(PyObject *, PyObject *const *v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int kFunctions = 15;
  count(n, kFunctions + 1);
  void *f[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(v[i]);
    if (!f[i]) fail(PyExc_ValueError, "address of a library function missing");
  }
  run_epilogue = reinterpret_cast<decltype(run_epilogue)>(f[0]);
  run_epilogue_backward = reinterpret_cast<decltype(run_epilogue_backward)>(f[1]);
  run_gated = reinterpret_cast<decltype(run_gated)>(f[2]);
  run_gated_backward = reinterpret_cast<decltype(run_gated_backward)>(f[3]);
  run_layer_norm = reinterpret_cast<decltype(run_layer_norm)>(f[4]);
  run_layer_norm_backward = reinterpret_cast<decltype(run_layer_norm_backward)>(f[5]);
  run_expert_sort = reinterpret_cast<decltype(run_expert_sort)>(f[6]);
  run_expert_gather = reinterpret_cast<decltype(run_expert_gather)>(f[7]);
  run_expert_combine = reinterpret_cast<decltype(run_expert_combine)>(f[8]);
  run_expert_combine_backward = reinterpret_cast<decltype(run_expert_combine_backward)>(f[9]);
  run_expert = reinterpret_cast<decltype(run_expert)>(f[10]);
  run_expert_backward = reinterpret_cast<decltype(run_expert_backward)>(f[11]);
  run_expert_gated = reinterpret_cast<decltype(run_expert_gated)>(f[12]);
  run_expert_gated_backward = reinterpret_cast<decltype(run_expert_gated_backward)>(f[13]);
  run_dropout = reinterpret_cast<decltype(run_dropout)>(f[14]);
  Py_INCREF(v[kFunctions]);
  Py_XDECREF(raise_status);
  raise_status = v[kFunctions];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init), FAST(matmul_epilogue), FAST(matmul_epilogue_backward),
                         FAST(gated), FAST(gated_backward), FAST(layer_norm),
                         FAST(layer_norm_backward), FAST(expert_sort), FAST(expert_gather),
                         FAST(expert_combine), FAST(expert_combine_backward), FAST(expert_matmul),
                         FAST(expert_matmul_backward), FAST(expert_gated),
                         FAST(expert_gated_backward), FAST(dropout),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gemm_gb300_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gemm_gb300_torch() { return PyModule_Create(&module); }

// Python module sparse_moe_router_amd._ops: the calls of ops.py on torch
// tensors.  Checks the arguments, allocates what the caller did not pass and
// calls the C ABI of moe_ops.h on the current stream of the tensors' device.
//
// Compiled, and not ctypes as for the layer's own entry points: a decode step
// makes several of these calls for one token, and reading a dozen tensor
// attributes through the interpreter costs 13-20 us a call where the kernels
// take 3-9 us; here a call costs 5-8 us of the host's time.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <c10/core/GradMode.h>

#include <initializer_list>
#include <string>
#include <vector>

#include "moe_ops.h"

extern "C" int hipGetDevice(int*);
extern "C" int hipSetDevice(int);

namespace {

using at::Tensor;

constexpr auto BF16 = at::kBFloat16;
constexpr auto F32 = at::kFloat;
constexpr auto I8 = at::kChar;
constexpr auto I32 = at::kInt;

struct Error {
  PyObject* type;
  std::string text;
};
[[noreturn]] void value_error(const std::string& s) { throw Error{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Error{PyExc_TypeError, s}; }
struct PythonError {};  // the interpreter's error is set already

PyObject* g_raw_stream = nullptr;  // torch._C._cuda_getCurrentRawStream
PyObject* g_check = nullptr;       // moe._check
PyObject* g_oom = nullptr;         // torch.OutOfMemoryError

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

typedef std::initializer_list<at::ScalarType> Types;

// One call: its device, made current while the call lasts, and its stream.
struct Call {
  int device = -1, before = -1;
  hipStream_t stream = nullptr;
  bool warned = false;

  // a tensor argument; the first one fixes the device
  const Tensor& tensor(PyObject* o, Types types, int dims, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error(std::string(name) + " must be on the GPU, got " + t.device().str());
    const int d = t.get_device();
    if (device < 0)
      device = d;
    else if (d != device)
      value_error(std::string(name) + " is on " + t.device().str() + ", the call on cuda:" + std::to_string(device));
    bool ok = false;
    for (auto s : types) ok = ok || t.scalar_type() == s;
    if (!ok) {
      std::string want;
      for (auto s : types) want += (want.empty() ? "" : " or ") + std::string(c10::toString(s));
      type_error(std::string(name) + " must be " + want + ", got " + c10::toString(t.scalar_type()));
    }
    if (t.dim() != dims)
      value_error(std::string(name) + " must have " + std::to_string(dims) + " dimension(s), got " + shape_of(t));
    if (t.requires_grad() && c10::GradMode::is_enabled())
      warn(std::string(name) + " requires a gradient, which this call does not record: use its gradient call, from "
                               "torch.no_grad() or a torch.autograd.Function");
    return t;
  }
  // once a call, at the line that calls ops.py, whose own frames there are `frames` of
  void warn(const std::string& text, int frames = 2) {
    if (warned) return;
    warned = true;
    if (PyErr_WarnEx(PyExc_UserWarning, text.c_str(), frames + 1) != 0) throw PythonError{};
  }
  // a contiguous tensor of exactly this shape; its address
  void* flat(PyObject* o, Types types, std::initializer_list<int64_t> shape, const char* name) {
    const Tensor& t = tensor(o, types, (int)shape.size(), name);
    if (!std::equal(shape.begin(), shape.end(), t.sizes().begin())) {
      std::string want;
      for (int64_t v : shape) want += (want.empty() ? "" : ", ") + std::to_string(v);
      value_error(std::string(name) + " must have shape (" + want + "), got " + shape_of(t));
    }
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  // a matrix with contiguous rows (rows < 0: any number of them)
  moe_mat_t rows(PyObject* o, Types types, int64_t rows, int64_t cols, const char* name) {
    const Tensor& t = tensor(o, types, 2, name);
    if (t.size(1) != cols || (rows >= 0 && t.size(0) != rows))
      value_error(std::string(name) + " must have shape (" + (rows < 0 ? "rows" : std::to_string(rows)) + ", " +
                  std::to_string(cols) + "), got " + shape_of(t));
    if (t.stride(1) != 1 && t.numel() > 0) value_error(std::string(name) + " must have contiguous rows");
    // a matrix of one row (or none) has no row stride of its own
    const int64_t ld = t.size(0) > 1 ? t.stride(0) : cols;
    if (ld < cols) value_error(std::string(name) + " must not have overlapping rows");
    return moe_mat_t{t.data_ptr(), ld};
  }
  // makes the device current and takes its current stream; before any allocation
  void begin() {
    int cur = 0;
    if (hipGetDevice(&cur) == 0 && cur != device) {
      if (hipSetDevice(device) != 0) value_error("cannot make cuda:" + std::to_string(device) + " current");
      before = cur;
    }
    PyObject* idx = PyLong_FromLong(device);
    if (!idx) throw PythonError{};
    PyObject* s = PyObject_CallOneArg(g_raw_stream, idx);
    Py_DECREF(idx);
    if (!s) throw PythonError{};
    stream = (hipStream_t)PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) throw PythonError{};
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::empty(shape, at::TensorOptions().dtype(t).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
  }
  ~Call() {
    if (before >= 0) hipSetDevice(before);
  }
};

moe_dtype_t dt(const Tensor& t) { return t.scalar_type() == F32 ? MOE_DT_FP32 : MOE_DT_BF16; }

at::ScalarType out_type(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v ? F32 : BF16;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < INT32_MIN || v > INT32_MAX) value_error("integer argument out of range");
  return (int)v;
}
bool given(PyObject* o) { return o != Py_None; }

void check(moe_status_t st, const char* what) {
  if (st == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, what);
  Py_XDECREF(r);
  throw PythonError{};
}

// the caller's workspace, or one of the call's own: calls on different streams and captured graphs
// never share one
void* workspace(Call& c, PyObject* o, size_t need, Tensor* own, size_t* have) {
  if (given(o)) {
    const Tensor& t = c.tensor(o, {at::kByte}, 1, "workspace");
    if (!t.is_contiguous()) value_error("workspace must be contiguous");
    *have = (size_t)t.numel();
    return t.data_ptr();
  }
  *own = c.empty({(int64_t)need}, at::kByte);
  *have = need;
  return need ? own->data_ptr() : nullptr;
}

// group offsets and permutation into g
void set_groups(Call& c, moe_groups_t* g, PyObject* offsets, PyObject* perm, PyObject* top_k) {
  if (given(offsets))
    g->offsets = (const int32_t*)c.flat(offsets, {I32}, {(int64_t)g->E + 1}, "offsets");
  else if (g->E != 1)
    value_error("offsets may be left out with one expert only");
  if (given(perm)) g->perm = (const int32_t*)c.flat(perm, {I32}, {g->rows}, "perm");
  g->top_k = integer(top_k);
}

int32_t dim32(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(std::string(name) + " is too large");
  return (int32_t)v;
}

// rows of the grouped order: those of perm, else of x.  An out of another number of rows is refused
// with the permutation's shape, here (fewer than x: its last rows would not be computed) or by the
// library (more than x).
int64_t forward_rows(Call& c, PyObject* out, PyObject* perm, const Tensor& x) {
  if (given(out)) {
    const Tensor& t = c.tensor(out, {BF16, F32}, 2, "out");
    if (!given(perm) && t.size(0) < x.size(0))
      value_error("out must have a row for each of x's " + std::to_string(x.size(0)) + ", got " + shape_of(t));
    return t.size(0);
  }
  if (given(perm)) return c.tensor(perm, {I32}, 1, "perm").size(0);
  return x.size(0);
}

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
// A tensor of the caller's has other values now: a graph of torch's differentiation that had saved it
// refuses to use them.  (A tensor of the inference mode has no version.)
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
PyObject* result(PyObject* o, Tensor& own) {
  if (!given(o)) return wrap(std::move(own));
  written(THPVariable_Unpack(o));
  Py_INCREF(o);
  return o;
}

// Runs body with C++ errors turned into Python's; nothing is thrown through the interpreter.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Error& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_oom, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

typedef PyObject* const* Args;

// x, w, offsets, perm, top_k, out, fp32
PyObject* grouped_matmul(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[0], {BF16}, 2, "x");
    const Tensor& w = c.tensor(a[1], {BF16}, 3, "w");
    moe_groups_t g{};
    g.E = dim32(w.size(0), "w"), g.N = dim32(w.size(1), "w"), g.K = dim32(w.size(2), "w");
    void* wp = c.flat(a[1], {BF16}, {g.E, g.N, g.K}, "w");
    const moe_mat_t xm = c.rows(a[0], {BF16}, -1, g.K, "x");
    g.rows = forward_rows(c, a[5], a[3], x);
    g.x_rows = x.size(0);
    set_groups(c, &g, a[2], a[3], a[4]);
    c.begin();
    Tensor own;
    if (!given(a[5])) own = c.empty({g.rows, g.N}, out_type(a[6]));
    const moe_mat_t ym = given(a[5]) ? c.rows(a[5], {BF16, F32}, -1, g.N, "out") : moe_mat_t{own.data_ptr(), g.N};
    g.ldx = xm.ld, g.ldy = ym.ld;
    check(moe_grouped_matmul(&g, xm.data, wp, ym.data, dt(given(a[5]) ? THPVariable_Unpack(a[5]) : own), c.stream),
          "moe_grouped_matmul");
    return result(a[5], own);
  });
}

// dy, w, offsets, out, fp32
PyObject* grouped_matmul_grad_input(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Call c;
    const Tensor& dy = c.tensor(a[0], {BF16}, 2, "dy");
    const Tensor& w = c.tensor(a[1], {BF16}, 3, "w");
    moe_groups_t g{};
    g.E = dim32(w.size(0), "w"), g.N = dim32(w.size(1), "w"), g.K = dim32(w.size(2), "w");
    void* wp = c.flat(a[1], {BF16}, {g.E, g.N, g.K}, "w");
    const moe_mat_t dym = c.rows(a[0], {BF16}, -1, g.N, "dy");
    g.rows = g.x_rows = dy.size(0);
    PyObject* one = PyLong_FromLong(1);
    set_groups(c, &g, a[2], Py_None, one);
    Py_XDECREF(one);
    c.begin();
    Tensor own;
    if (!given(a[3])) own = c.empty({g.rows, g.K}, out_type(a[4]));
    const moe_mat_t dxm = given(a[3]) ? c.rows(a[3], {BF16, F32}, g.rows, g.K, "out") : moe_mat_t{own.data_ptr(), g.K};
    g.ldx = dxm.ld, g.ldy = dym.ld;
    check(moe_grouped_matmul_grad_input(&g, dym.data, wp, dxm.data,
                                        dt(given(a[3]) ? THPVariable_Unpack(a[3]) : own), c.stream),
          "moe_grouped_matmul_grad_input");
    return result(a[3], own);
  });
}

// x, dy, offsets, perm, top_k, out, fp32
PyObject* grouped_matmul_grad_weight(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[0], {BF16}, 2, "x");
    const Tensor& dy = c.tensor(a[1], {BF16}, 2, "dy");
    moe_groups_t g{};
    g.E = given(a[2]) ? dim32(c.tensor(a[2], {I32}, 1, "offsets").size(0) - 1, "offsets") : 1;
    g.N = dim32(dy.size(1), "dy"), g.K = dim32(x.size(1), "x");
    const moe_mat_t xm = c.rows(a[0], {BF16}, -1, g.K, "x"), dym = c.rows(a[1], {BF16}, -1, g.N, "dy");
    g.rows = dy.size(0);
    g.x_rows = x.size(0);
    g.ldx = xm.ld, g.ldy = dym.ld;
    set_groups(c, &g, a[2], a[3], a[4]);
    if (g.E < 1) value_error("offsets must have at least two entries");
    c.begin();
    Tensor own;
    if (!given(a[5])) own = c.empty({g.E, g.N, g.K}, out_type(a[6]));
    void* dw = given(a[5]) ? c.flat(a[5], {BF16, F32}, {g.E, g.N, g.K}, "out") : own.data_ptr();
    check(moe_grouped_matmul_grad_weight(&g, xm.data, dym.data, dw, dt(given(a[5]) ? THPVariable_Unpack(a[5]) : own),
                                         c.stream),
          "moe_grouped_matmul_grad_weight");
    return result(a[5], own);
  });
}

// x, codes, scale
PyObject* quantize_i8(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[0], {BF16}, 2, "x");
    const int64_t M = x.size(0), K = x.size(1);
    const moe_mat_t xm = c.rows(a[0], {BF16}, M, K, "x");
    c.begin();
    Tensor q, s;
    void* qp = given(a[1]) ? c.flat(a[1], {I8}, {M, K}, "codes") : (q = c.empty({M, K}, I8)).data_ptr();
    void* sp = given(a[2]) ? c.flat(a[2], {F32}, {M}, "scale") : (s = c.empty({M}, F32)).data_ptr();
    check(moe_quantize_i8(M, dim32(K, "x"), xm.ld, xm.data, qp, (float*)sp, c.stream), "moe_quantize_i8");
    PyObject* r0 = result(a[1], q);
    PyObject* r1 = result(a[2], s);
    PyObject* r = PyTuple_Pack(2, r0, r1);
    Py_XDECREF(r0);
    Py_XDECREF(r1);
    return r;
  });
}

// x, w [N][K] or [E][N][K], w_scale, offsets, perm, top_k, x_scale, bias, out, fp32, workspace
PyObject* matmul_i8(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[0], {BF16, I8}, 2, "x");
    if ((x.scalar_type() == I8) != given(a[6]))
      value_error("x is either bf16, quantised by the call, or int8 codes with x_scale");
    const bool one = THPVariable_Check(a[1]) && THPVariable_Unpack(a[1]).dim() == 2;
    const Tensor& w = c.tensor(a[1], {I8}, one ? 2 : 3, "w");
    moe_groups_t g{};
    g.E = one ? 1 : dim32(w.size(0), "w");
    g.N = dim32(w.size(one ? 0 : 1), "w"), g.K = dim32(w.size(one ? 1 : 2), "w");
    if (!w.is_contiguous()) value_error("w must be contiguous");
    const float* ws = (const float*)(one ? c.flat(a[2], {F32}, {g.N}, "w_scale")
                                         : c.flat(a[2], {F32}, {g.E, g.N}, "w_scale"));
    const moe_mat_t xm = c.rows(a[0], {BF16, I8}, -1, g.K, "x");
    g.x_rows = x.size(0);
    g.rows = forward_rows(c, a[8], a[4], x);
    set_groups(c, &g, a[3], a[4], a[5]);
    const float* xs = given(a[6]) ? (const float*)c.flat(a[6], {F32}, {g.x_rows}, "x_scale") : nullptr;
    const float* bias = given(a[7]) ? (const float*)c.flat(a[7], {F32}, {g.N}, "bias") : nullptr;
    c.begin();
    Tensor own, wk;
    if (!given(a[8])) own = c.empty({g.rows, g.N}, out_type(a[9]));
    const moe_mat_t ym =
        given(a[8]) ? c.rows(a[8], {BF16, F32}, one ? g.x_rows : -1, g.N, "out") : moe_mat_t{own.data_ptr(), g.N};
    g.ldx = xm.ld, g.ldy = ym.ld;
    void* wkp = nullptr;
    size_t have = 0;
    if (!given(a[6])) wkp = workspace(c, a[10], moe_matmul_i8_workspace_size(&g), &wk, &have);
    check(moe_matmul_i8(&g, xm.data, xs, w.data_ptr(), ws, bias, ym.data,
                        dt(given(a[8]) ? THPVariable_Unpack(a[8]) : own), wkp, have, c.stream),
          "moe_matmul_i8");
    return result(a[8], own);
  });
}

// gate mode and matrix (or vector) of a gate
moe_gate_t gate_arg(Call& c, PyObject* o, int64_t M, int64_t H, moe_mat_t* m) {
  *m = moe_mat_t{nullptr, 0};
  if (!given(o)) return MOE_GATE_NONE;
  if (THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 1) {
    m->data = c.flat(o, {BF16}, {M}, "gate");
    return MOE_GATE_TOKEN;
  }
  *m = c.rows(o, {BF16}, M, H, "gate");
  return MOE_GATE_ELEMENT;
}

moe_mat_t opt_rows(Call& c, PyObject* o, at::ScalarType t, int64_t M, int64_t H, const char* name) {
  return given(o) ? c.rows(o, {t}, M, H, name) : moe_mat_t{nullptr, 0};
}

// x, weight, eps, out
PyObject* block_norm(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[0], {BF16, F32}, 2, "x");
    const int64_t M = x.size(0), H = x.size(1);
    const moe_mat_t xm = c.rows(a[0], {BF16, F32}, M, H, "x");
    const void* w = c.flat(a[1], {BF16, F32}, {H}, "weight");
    moe_norm_t d{M, dim32(H, "x"), dt(x), dt(THPVariable_Unpack(a[1])), MOE_GATE_NONE, (float)number(a[2]), 1.0f};
    c.begin();
    Tensor own;
    const moe_mat_t h = given(a[3]) ? c.rows(a[3], {BF16}, M, H, "out")
                                    : moe_mat_t{(own = c.empty({M, H}, BF16)).data_ptr(), H};
    check(moe_block_norm(&d, xm, w, h, c.stream), "moe_block_norm");
    return result(a[3], own);
  });
}

// d_h, x, weight, eps, d_add, workspace
PyObject* block_norm_grad(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[1], {BF16, F32}, 2, "x");
    const int64_t M = x.size(0), H = x.size(1);
    const moe_mat_t xm = c.rows(a[1], {BF16, F32}, M, H, "x"), dh = c.rows(a[0], {BF16}, M, H, "d_h");
    const moe_mat_t da = opt_rows(c, a[4], x.scalar_type(), M, H, "d_add");
    const void* w = c.flat(a[2], {BF16, F32}, {H}, "weight");
    moe_norm_t d{M, dim32(H, "x"), dt(x), dt(THPVariable_Unpack(a[2])), MOE_GATE_NONE, (float)number(a[3]), 1.0f};
    c.begin();
    Tensor dx = c.empty({M, H}, x.scalar_type()), dw = c.empty({H}, F32), wk;
    size_t have = 0;
    void* wkp = workspace(c, a[5], moe_norm_grad_workspace_size(&d), &wk, &have);
    check(moe_block_norm_grad(&d, dh, xm, w, da, moe_mat_t{dx.data_ptr(), H}, (float*)dw.data_ptr(), wkp, have,
                              c.stream),
          "moe_block_norm_grad");
    return Py_BuildValue("{sNsN}", "x", wrap(dx), "weight", wrap(dw));
  });
}

// residual, y, weight, eps, gate, scale, next_weight, out, h
PyObject* block_merge(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call c;
    const Tensor& r = c.tensor(a[0], {BF16, F32}, 2, "residual");
    const int64_t M = r.size(0), H = r.size(1);
    const auto st = r.scalar_type();
    const moe_mat_t rm = c.rows(a[0], {st}, M, H, "residual"), ym = c.rows(a[1], {BF16}, M, H, "y");
    const void* w = c.flat(a[2], {BF16, F32}, {H}, "weight");
    const Tensor& wt = THPVariable_Unpack(a[2]);
    moe_mat_t gm;
    const moe_gate_t mode = gate_arg(c, a[4], M, H, &gm);
    const void* wn = given(a[6]) ? c.flat(a[6], {wt.scalar_type()}, {H}, "next_weight") : nullptr;
    if (!given(a[6]) && given(a[8])) value_error("h needs next_weight");
    moe_norm_t d{M, dim32(H, "residual"), dt(r), dt(wt), mode, (float)number(a[3]), (float)number(a[5])};
    c.begin();
    Tensor out, h;
    const moe_mat_t om =
        given(a[7]) ? c.rows(a[7], {st}, M, H, "out") : moe_mat_t{(out = c.empty({M, H}, st)).data_ptr(), H};
    moe_mat_t hm{nullptr, 0};
    if (given(a[6]))
      hm = given(a[8]) ? c.rows(a[8], {BF16}, M, H, "h") : moe_mat_t{(h = c.empty({M, H}, BF16)).data_ptr(), H};
    check(moe_block_merge(&d, rm, ym, w, gm, wn, om, hm, c.stream), "moe_block_merge");
    PyObject* ro = result(a[7], out);
    if (!given(a[6])) return ro;
    PyObject* rh = result(a[8], h);
    PyObject* res = PyTuple_Pack(2, ro, rh);
    Py_XDECREF(ro);
    Py_XDECREF(rh);
    return res;
  });
}

// d_out, y, weight, eps, gate, scale, next_weight, out, d_h, workspace
PyObject* block_merge_grad(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c;
    const Tensor& y = c.tensor(a[1], {BF16}, 2, "y");
    const int64_t M = y.size(0), H = y.size(1);
    const bool next = given(a[6]);
    if (next != given(a[8]) || next != given(a[7])) value_error("next_weight, out and d_h are given together");
    if (!given(a[0]) && !next) value_error("d_out or d_h must be given");
    const bool from_out = !given(a[0]);
    const auto st = c.tensor(a[from_out ? 7 : 0], {BF16, F32}, 2, from_out ? "out" : "d_out").scalar_type();
    const moe_mat_t ym = c.rows(a[1], {BF16}, M, H, "y"), dom = opt_rows(c, a[0], st, M, H, "d_out"),
                    om = opt_rows(c, a[7], st, M, H, "out"), dhm = opt_rows(c, a[8], BF16, M, H, "d_h");
    const void* w = c.flat(a[2], {BF16, F32}, {H}, "weight");
    const Tensor& wt = THPVariable_Unpack(a[2]);
    const void* wn = next ? c.flat(a[6], {wt.scalar_type()}, {H}, "next_weight") : nullptr;
    moe_mat_t gm;
    const moe_gate_t mode = gate_arg(c, a[4], M, H, &gm);
    moe_norm_t d{M,    dim32(H, "y"), st == F32 ? MOE_DT_FP32 : MOE_DT_BF16, dt(wt),
                 mode, (float)number(a[3]), (float)number(a[5])};
    c.begin();
    Tensor dr = c.empty({M, H}, st), dy = c.empty({M, H}, BF16), dw = c.empty({H}, F32), dg, dwn, wk;
    if (mode == MOE_GATE_TOKEN) dg = c.empty({M}, BF16);
    if (mode == MOE_GATE_ELEMENT) dg = c.empty({M, H}, BF16);
    if (next) dwn = c.empty({H}, F32);
    size_t have = 0;
    void* wkp = workspace(c, a[9], moe_norm_grad_workspace_size(&d), &wk, &have);
    check(moe_block_merge_grad(&d, dom, dhm, ym, w, gm, om, wn, moe_mat_t{dr.data_ptr(), H},
                               moe_mat_t{dy.data_ptr(), H}, moe_mat_t{mode ? dg.data_ptr() : nullptr, H},
                               (float*)dw.data_ptr(), next ? (float*)dwn.data_ptr() : nullptr, wkp, have, c.stream),
          "moe_block_merge_grad");
    PyObject* res = Py_BuildValue("{sNsNsN}", "residual", wrap(dr), "y", wrap(dy), "weight", wrap(dw));
    auto put = [&](const char* key, Tensor& t) {
      PyObject* v = wrap(t);
      if (!v || PyDict_SetItemString(res, key, v) != 0) {
        Py_XDECREF(v);
        Py_DECREF(res);
        throw PythonError{};
      }
      Py_DECREF(v);
    };
    if (!res) return nullptr;
    if (mode != MOE_GATE_NONE) put("gate", dg);
    if (next) put("next_weight", dwn);
    return res;
  });
}

// x, w, offsets, perm, top_k, save, out, gate_up
PyObject* gated_matmul(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call c;
    const Tensor& x = c.tensor(a[0], {BF16}, 2, "x");
    const Tensor& w = c.tensor(a[1], {BF16}, 3, "w");
    if (w.size(1) % 2) value_error("w must have the rows of two matrices, got " + shape_of(w));
    moe_groups_t g{};
    g.E = dim32(w.size(0), "w"), g.N = dim32(w.size(1) / 2, "w"), g.K = dim32(w.size(2), "w");
    void* wp = c.flat(a[1], {BF16}, {g.E, 2 * (int64_t)g.N, g.K}, "w");
    const moe_mat_t xm = c.rows(a[0], {BF16}, -1, g.K, "x");
    g.rows = forward_rows(c, a[6], a[3], x);
    g.x_rows = x.size(0);
    set_groups(c, &g, a[2], a[3], a[4]);
    const int save = PyObject_IsTrue(a[5]);
    if (save < 0) throw PythonError{};
    if (given(a[7]) && !save) value_error("gate_up is written with save only");
    c.begin();
    Tensor own, pre;
    if (!given(a[6])) own = c.empty({g.rows, g.N}, BF16);
    const moe_mat_t hm = given(a[6]) ? c.rows(a[6], {BF16}, -1, g.N, "out") : moe_mat_t{own.data_ptr(), g.N};
    moe_mat_t pm{nullptr, 0};
    const int64_t cols = 2 * (int64_t)g.N;
    if (save)
      pm = given(a[7]) ? c.rows(a[7], {BF16}, g.rows, cols, "gate_up")
                       : moe_mat_t{(pre = c.empty({g.rows, cols}, BF16)).data_ptr(), cols};
    g.ldx = xm.ld, g.ldy = hm.ld;
    check(moe_gated_matmul(&g, xm.data, wp, hm.data, pm, c.stream), "moe_gated_matmul");
    PyObject* h = result(a[6], own);
    if (!save) return h;
    PyObject* q = result(a[7], pre);
    PyObject* r = PyTuple_Pack(2, h, q);
    Py_XDECREF(h);
    Py_XDECREF(q);
    return r;
  });
}

// dy, w, gate_up, offsets
PyObject* gated_matmul_grad(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    Call c;
    const Tensor& dy = c.tensor(a[0], {BF16}, 2, "dy");
    const Tensor& w = c.tensor(a[1], {BF16}, 3, "w");
    moe_groups_t g{};
    g.E = dim32(w.size(0), "w"), g.N = dim32(w.size(1), "w"), g.K = dim32(w.size(2), "w");
    void* wp = c.flat(a[1], {BF16}, {g.E, g.N, g.K}, "w");
    const moe_mat_t dym = c.rows(a[0], {BF16}, -1, g.N, "dy");
    g.rows = g.x_rows = dy.size(0);
    g.top_k = 1;
    const int64_t cols = 2 * (int64_t)g.K;
    const moe_mat_t pm = c.rows(a[2], {BF16}, g.rows, cols, "gate_up");
    if (given(a[3]))
      g.offsets = (const int32_t*)c.flat(a[3], {I32}, {(int64_t)g.E + 1}, "offsets");
    else if (g.E != 1)
      value_error("offsets may be left out with one expert only");
    c.begin();
    Tensor d = c.empty({g.rows, cols}, BF16), h = c.empty({g.rows, g.K}, BF16);
    g.ldx = g.K, g.ldy = dym.ld;
    check(moe_gated_matmul_grad(&g, dym.data, wp, pm, moe_mat_t{d.data_ptr(), cols}, h.data_ptr(), c.stream),
          "moe_gated_matmul_grad");
    return Py_BuildValue("{sNsN}", "gate_up", wrap(d), "h", wrap(h));
  });
}

// dy, x, w_gate_up, w_down, gate_up, offsets, perm, top_k, dw fp32, workspace
PyObject* feed_forward_grad(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c;
    const Tensor& dy = c.tensor(a[0], {BF16}, 2, "dy");
    const Tensor& x = c.tensor(a[1], {BF16}, 2, "x");
    const Tensor& w = c.tensor(a[2], {BF16}, 3, "w_gate_up");
    if (w.size(1) % 2) value_error("w_gate_up must have the rows of two matrices, got " + shape_of(w));
    moe_feed_forward_t d{};
    d.E = dim32(w.size(0), "w_gate_up"), d.I = dim32(w.size(1) / 2, "w_gate_up"), d.K = dim32(w.size(2), "w_gate_up");
    d.H = dim32(dy.size(1), "dy");
    const int64_t I2 = 2 * (int64_t)d.I;
    const void* wp = c.flat(a[2], {BF16}, {d.E, I2, d.K}, "w_gate_up");
    const void* wd = c.flat(a[3], {BF16}, {d.E, d.H, d.I}, "w_down");
    const moe_mat_t dym = c.rows(a[0], {BF16}, -1, d.H, "dy"), xm = c.rows(a[1], {BF16}, -1, d.K, "x");
    d.rows = dy.size(0), d.x_rows = x.size(0), d.ldx = xm.ld, d.ld_dy = dym.ld;
    const moe_mat_t pm = c.rows(a[4], {BF16}, d.rows, I2, "gate_up");
    moe_groups_t g{};
    g.rows = d.rows, g.E = d.E;
    set_groups(c, &g, a[5], a[6], a[7]);
    d.offsets = g.offsets, d.perm = g.perm, d.top_k = g.top_k;
    const auto type = out_type(a[8]);
    c.begin();
    Tensor dx = c.empty({d.rows, d.K}, BF16), dgu = c.empty({d.E, I2, d.K}, type), dwd = c.empty({d.E, d.H, d.I}, type), wk;
    size_t have = 0;
    void* wkp = workspace(c, a[9], moe_feed_forward_grad_workspace_size(&d), &wk, &have);
    check(moe_feed_forward_grad(&d, dym.data, xm.data, wp, wd, pm, moe_mat_t{dx.data_ptr(), d.K}, dgu.data_ptr(),
                                dwd.data_ptr(), dt(dgu), wkp, have, c.stream),
          "moe_feed_forward_grad");
    return Py_BuildValue("{sNsNsN}", "x", wrap(dx), "w_gate_up", wrap(dgu), "w_down", wrap(dwd));
  });
}

// group offsets of any number of experts; their number
const int32_t* any_offsets(Call& c, PyObject* o, int32_t* E) {
  if (!given(o)) return nullptr;
  const Tensor& t = c.tensor(o, {I32}, 1, "offsets");
  if (t.size(0) < 2) value_error("offsets must have at least two entries");
  *E = dim32(t.size(0) - 1, "offsets");
  return (const int32_t*)c.flat(o, {I32}, {t.size(0)}, "offsets");
}

// perm, assignments (None: as many as perm), offsets, out
PyObject* invert_permutation(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    Call c;
    const int64_t rows = c.tensor(a[0], {I32}, 1, "perm").size(0);
    const void* perm = c.flat(a[0], {I32}, {rows}, "perm");
    int64_t num = rows;
    if (given(a[1])) {
      num = PyLong_AsLongLong(a[1]);
      if (num == -1 && PyErr_Occurred()) throw PythonError{};
      if (num < 0) value_error("assignments must not be negative");
    }
    int32_t E = 0;
    const int32_t* offsets = any_offsets(c, a[2], &E);
    c.begin();
    Tensor own;
    void* out = given(a[3]) ? c.flat(a[3], {I32}, {num}, "out") : (own = c.empty({num}, I32)).data_ptr();
    check(moe_invert_permutation(rows, (const int32_t*)perm, offsets, E, num, (int32_t*)out, c.stream),
          "moe_invert_permutation");
    return result(a[3], own);
  });
}

// tokens of a combine: inverse holds top_k assignments of each
void set_combine(Call& c, moe_combine_t* d, const Tensor& inverse, PyObject* top_k) {
  d->top_k = integer(top_k);
  if (d->top_k < 1 || inverse.size(0) % d->top_k) value_error("inverse must hold top_k entries for each token");
  d->tokens = inverse.size(0) / d->top_k;
}

// y, inverse, top_k, weight, add, out, fp32
PyObject* combine(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c;
    const Tensor& y = c.tensor(a[0], {BF16}, 2, "y");
    moe_combine_t d{};
    const Tensor& inv = c.tensor(a[1], {I32}, 1, "inverse");
    set_combine(c, &d, inv, a[2]);
    d.inverse = (const int32_t*)c.flat(a[1], {I32}, {inv.size(0)}, "inverse");
    d.rows = y.size(0), d.H = dim32(y.size(1), "y");
    const moe_mat_t ym = c.rows(a[0], {BF16}, d.rows, d.H, "y");
    const float* w = given(a[3]) ? (const float*)c.flat(a[3], {F32}, {d.tokens, d.top_k}, "weight") : nullptr;
    const auto type = given(a[5]) ? c.tensor(a[5], {BF16, F32}, 2, "out").scalar_type() : out_type(a[6]);
    const moe_mat_t am = opt_rows(c, a[4], type, d.tokens, d.H, "add");
    d.out_type = type == F32 ? MOE_DT_FP32 : MOE_DT_BF16;
    c.begin();
    Tensor own;
    const moe_mat_t om = given(a[5]) ? c.rows(a[5], {type}, d.tokens, d.H, "out")
                                     : moe_mat_t{(own = c.empty({d.tokens, d.H}, type)).data_ptr(), d.H};
    check(moe_combine(&d, ym, w, am, om, c.stream), "moe_combine");
    return result(a[5], own);
  });
}

// d_out, y, perm, inverse, weight, top_k, offsets, dy
PyObject* combine_grad(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call c;
    const Tensor& dout = c.tensor(a[0], {BF16}, 2, "d_out");
    moe_combine_t d{};
    d.H = dim32(dout.size(1), "d_out");
    const moe_mat_t dm = c.rows(a[0], {BF16}, -1, d.H, "d_out");
    d.rows = c.tensor(a[2], {I32}, 1, "perm").size(0);
    d.perm = (const int32_t*)c.flat(a[2], {I32}, {d.rows}, "perm");
    const Tensor& inv = c.tensor(a[3], {I32}, 1, "inverse");
    d.inverse = (const int32_t*)c.flat(a[3], {I32}, {inv.size(0)}, "inverse");
    const float* w = nullptr;
    moe_mat_t ym{nullptr, 0};
    if (given(a[4])) {
      const Tensor& wt = c.tensor(a[4], {F32}, 2, "weight");
      d.top_k = dim32(wt.size(1), "weight");
      if (given(a[5]) && integer(a[5]) != d.top_k) value_error("weight must have top_k columns, got " + shape_of(wt));
      d.tokens = dout.size(0);
      w = (const float*)c.flat(a[4], {F32}, {d.tokens, d.top_k}, "weight");
      if (!given(a[1])) value_error("y must be given with weight");
      ym = c.rows(a[1], {BF16}, d.rows, d.H, "y");
    } else {
      if (!given(a[5])) value_error("top_k must be given without weight");
      set_combine(c, &d, inv, a[5]);
    }
    if (dout.size(0) != d.tokens || inv.size(0) != d.tokens * d.top_k)
      value_error("d_out must have a row, and inverse top_k entries, for each token, got " + shape_of(dout) + " and " +
                  shape_of(inv));
    d.offsets = any_offsets(c, a[6], &d.E);
    c.begin();
    Tensor own, dw;
    const moe_mat_t dym = given(a[7]) ? c.rows(a[7], {BF16}, d.rows, d.H, "dy")
                                      : moe_mat_t{(own = c.empty({d.rows, d.H}, BF16)).data_ptr(), d.H};
    if (w) dw = c.empty({d.tokens, d.top_k}, F32);
    check(moe_combine_grad(&d, dm, ym, w, dym, w ? (float*)dw.data_ptr() : nullptr, c.stream), "moe_combine_grad");
    PyObject* res = Py_BuildValue("{sN}", "y", result(a[7], own));
    if (res && w) {
      PyObject* v = wrap(dw);
      if (!v || PyDict_SetItemString(res, "weight", v) != 0) {
        Py_XDECREF(v);
        Py_DECREF(res);
        throw PythonError{};
      }
      Py_DECREF(v);
    }
    return res;
  });
}

// One of many gradients: any shape, contiguous.
const Tensor& gradient(Call& c, PyObject* o, const char* name, Py_ssize_t i) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must hold torch tensors");
  const Tensor& t = THPVariable_Unpack(o);
  auto fail = [&](const std::string& s) { value_error(std::string(name) + "[" + std::to_string(i) + "] " + s); };
  if (!t.is_cuda()) fail("must be on the GPU, got " + t.device().str());
  const int d = t.get_device();
  if (c.device < 0)
    c.device = d;
  else if (d != c.device)
    fail("is on " + t.device().str() + ", the call on cuda:" + std::to_string(c.device));
  if (t.scalar_type() != BF16 && t.scalar_type() != F32)
    type_error(std::string(name) + "[" + std::to_string(i) + "] must be BFloat16 or Float, got " +
               c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) fail("must be contiguous");
  if (t.requires_grad() && c10::GradMode::is_enabled())
    c.warn(std::string(name) + "[" + std::to_string(i) + "] requires a gradient, which this call does not record: call it "
           "from torch.no_grad()", 3);
  return t;
}
// The list's tensors; with outs (None: in place) as their results.
std::vector<moe_tensor_t> gradients(Call& c, PyObject* list, PyObject* outs, bool scaled) {
  if (!PyList_Check(list) && !PyTuple_Check(list)) type_error("grads must be a list or tuple of tensors");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
  if (n == 0) value_error("grads must hold at least one tensor");
  const bool apart = scaled && given(outs);
  if (apart) {
    if (!PyList_Check(outs) && !PyTuple_Check(outs)) type_error("out must be a list or tuple of tensors");
    if (PySequence_Fast_GET_SIZE(outs) != n) value_error("out must hold a tensor for each gradient");
  }
  std::vector<moe_tensor_t> v((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor& t = gradient(c, PySequence_Fast_GET_ITEM(list, i), "grads", i);
    moe_tensor_t& m = v[(size_t)i];
    m.in = t.data_ptr();
    m.n = t.numel();
    m.in_type = m.out_type = dt(t);
    m.out = (void*)m.in;
    if (!apart) continue;
    const Tensor& o = gradient(c, PySequence_Fast_GET_ITEM(outs, i), "out", i);
    if (o.sizes() != t.sizes())
      value_error("out[" + std::to_string(i) + "] must have shape " + shape_of(t) + ", got " + shape_of(o));
    m.out = o.data_ptr();
    m.out_type = dt(o);
  }
  return v;
}
int32_t count_of(const std::vector<moe_tensor_t>& v) { return dim32((int64_t)v.size(), "grads"); }

// grads, workspace
PyObject* grad_norm(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    Call c;
    const auto v = gradients(c, a[0], Py_None, false);
    c.begin();
    Tensor norm = c.empty({}, F32), wk;
    size_t have = 0;
    void* wkp = workspace(c, a[1], moe_grad_norm_workspace_size(v.data(), count_of(v)), &wk, &have);
    check(moe_grad_norm(v.data(), count_of(v), (float*)norm.data_ptr(), wkp, have, c.stream), "moe_grad_norm");
    return wrap(norm);
  });
}

// grads, max_norm, norm, eps, out, workspace
PyObject* clip_grads(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Call c;
    const auto v = gradients(c, a[0], a[4], true);
    const double max_norm = number(a[1]), eps = number(a[3]);
    float* np = nullptr;
    if (given(a[2])) {
      const Tensor& t = THPVariable_Check(a[2]) ? c.tensor(a[2], {F32}, (int)THPVariable_Unpack(a[2]).dim(), "norm")
                                                : c.tensor(a[2], {F32}, 0, "norm");
      if (t.numel() != 1) value_error("norm must have one element, got " + shape_of(t));
      np = (float*)t.data_ptr();
    }
    c.begin();
    Tensor norm, wk;
    void* wkp = nullptr;
    size_t have = 0;
    if (!np) {
      norm = c.empty({}, F32);
      wkp = workspace(c, a[5], moe_grad_norm_workspace_size(v.data(), count_of(v)), &wk, &have);
    }
    check(moe_clip_grads(v.data(), count_of(v), (float)max_norm, (float)eps, np ? np : (float*)norm.data_ptr(), np != nullptr,
                         wkp, have, c.stream),
          "moe_clip_grads");
    PyObject* const outs = given(a[4]) ? a[4] : a[0];
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(outs); ++i)
      written(THPVariable_Unpack(PySequence_Fast_GET_ITEM(outs, i)));
    if (!np) return wrap(norm);
    Py_INCREF(a[2]);  // read only
    return a[2];
  });
}

// x, w, targets, ignore_index into a descriptor
struct Loss {
  moe_loss_t d{};
  moe_mat_t x;
  const void* w;
  const int64_t* target;
  Loss(Call& c, PyObject* xo, PyObject* wo, PyObject* to, PyObject* ignore) {
    const Tensor& xt = c.tensor(xo, {BF16}, 2, "x");
    const Tensor& wt = c.tensor(wo, {BF16}, 2, "w");
    d.rows = xt.size(0), d.H = dim32(xt.size(1), "x"), d.V = dim32(wt.size(0), "w");
    x = c.rows(xo, {BF16}, d.rows, d.H, "x");
    w = c.flat(wo, {BF16}, {d.V, d.H}, "w");
    target = (const int64_t*)c.flat(to, {at::kLong}, {d.rows}, "targets");
    d.ldx = x.ld;
    d.ignore_index = PyLong_AsLongLong(ignore);
    if (d.ignore_index == -1 && PyErr_Occurred()) throw PythonError{};
  }
};

// x, w, targets, ignore_index, workspace
PyObject* cross_entropy(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Call c;
    const Loss l(c, a[0], a[1], a[2], a[3]);
    c.begin();
    Tensor loss = c.empty({l.d.rows}, F32), lse = c.empty({l.d.rows}, F32), wk;
    size_t have = 0;
    void* wkp = workspace(c, a[4], moe_cross_entropy_workspace_size(&l.d), &wk, &have);
    check(moe_cross_entropy(&l.d, l.x.data, l.w, l.target, (float*)loss.data_ptr(), (float*)lse.data_ptr(), wkp, have,
                            c.stream),
          "moe_cross_entropy");
    PyObject* r0 = wrap(loss);
    PyObject* r1 = wrap(lse);
    PyObject* r = PyTuple_Pack(2, r0, r1);
    Py_XDECREF(r0);
    Py_XDECREF(r1);
    return r;
  });
}

// d_loss, x, w, targets, lse, ignore_index, dx fp32 (None: no dx), dw fp32 (None: no dw), workspace
PyObject* cross_entropy_grad(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call c;
    const Loss l(c, a[1], a[2], a[3], a[5]);
    const float* dl = (const float*)c.flat(a[0], {F32}, {l.d.rows}, "d_loss");
    const float* lse = (const float*)c.flat(a[4], {F32}, {l.d.rows}, "lse");
    c.begin();
    Tensor dx, dw, wk;
    moe_mat_t dxm{nullptr, 0};
    if (given(a[6])) {
      dx = c.empty({l.d.rows, l.d.H}, out_type(a[6]));
      dxm = moe_mat_t{dx.data_ptr(), l.d.H};
    }
    if (given(a[7])) dw = c.empty({l.d.V, l.d.H}, out_type(a[7]));
    size_t have = 0;
    void* wkp = workspace(c, a[8], moe_cross_entropy_grad_workspace_size(&l.d), &wk, &have);
    check(moe_cross_entropy_grad(&l.d, dl, l.x.data, l.w, l.target, lse, dxm, given(a[6]) ? dt(dx) : MOE_DT_BF16,
                                 given(a[7]) ? dw.data_ptr() : nullptr, given(a[7]) ? dt(dw) : MOE_DT_BF16, wkp, have,
                                 c.stream),
          "moe_cross_entropy_grad");
    PyObject* res = PyDict_New();
    auto put = [&](const char* key, Tensor& t) {
      PyObject* v = wrap(t);
      if (!v || PyDict_SetItemString(res, key, v) != 0) {
        Py_XDECREF(v);
        Py_DECREF(res);
        throw PythonError{};
      }
      Py_DECREF(v);
    };
    if (!res) return nullptr;
    if (given(a[6])) put("x", dx);
    if (given(a[7])) put("w", dw);
    return res;
  });
}

#define FAST(name) \
  { #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FAST(grouped_matmul),
                         FAST(grouped_matmul_grad_input),
                         FAST(grouped_matmul_grad_weight),
                         FAST(quantize_i8),
                         FAST(matmul_i8),
                         FAST(block_norm),
                         FAST(block_norm_grad),
                         FAST(block_merge),
                         FAST(block_merge_grad),
                         FAST(gated_matmul),
                         FAST(gated_matmul_grad),
                         FAST(feed_forward_grad),
                         FAST(invert_permutation),
                         FAST(combine),
                         FAST(combine_grad),
                         FAST(grad_norm),
                         FAST(clip_grads),
                         FAST(cross_entropy),
                         FAST(cross_entropy_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

PyObject* attribute(const char* mod, const char* name) {
  PyObject* m = PyImport_ImportModule(mod);
  if (!m) return nullptr;
  PyObject* a = PyObject_GetAttrString(m, name);
  Py_DECREF(m);
  return a;
}

}  // namespace

PyMODINIT_FUNC PyInit__ops() {
  g_raw_stream = attribute("torch._C", "_cuda_getCurrentRawStream");
  if (!g_raw_stream) return nullptr;
  g_check = attribute("sparse_moe_router_amd.moe", "_check");
  if (!g_check) return nullptr;
  g_oom = attribute("torch", "OutOfMemoryError");
  if (!g_oom) return nullptr;
  return PyModule_Create(&module);
}

// tg_torch.cpp -- Python's calls of the products with fused epilogues on torch tensors: checks of
// types, shapes and strides, new tensors for the results and the workspace, and the C entry point
// (include/tg.h) on torch's current stream.
//
// A CPython module instead of ctypes because a call is short: one gated projection of a token takes the
// GPU 4 us; by ctypes it took the host 15 us and a backward pass with three results 34, of which
// the entry points themselves need 5 and 10.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "../../include/tg.h"

namespace {

PyObject* g_error = nullptr;   // the package's TgError

struct PythonError {};   // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw PythonError();
}

// rc, or the package's exception for a negative one.
int64_t checked(int64_t rc) {
  if (rc >= 0) return rc;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(rc), tg_last_error());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

std::string sizes(int64_t rows, int64_t cols) {
  return "[" + std::to_string(rows) + ", " + std::to_string(cols) + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// A float16 or bfloat16 matrix with unit stride along its rows.
struct Matrix {
  at::Tensor t;
  int64_t rows, cols, ld;
  int code;   // TG_F16 or TG_BF16

  Matrix(PyObject* o, const char* name, const Matrix* like = nullptr)
      : t(tensor(o, name)) {
    const at::ScalarType type = t.scalar_type();
    if ((type != at::kHalf && type != at::kBFloat16) ||
        (like != nullptr && type != like->t.scalar_type()))
      raise(PyExc_TypeError, std::string(name) + " must be float16 or bfloat16" +
                                 (like ? ", the other matrices' type" : ""));
    code = type == at::kHalf ? TG_F16 : TG_BF16;
    if (t.dim() != 2) raise(PyExc_ValueError, std::string(name) + " must be a 2-D tensor");
    rows = t.size(0);
    cols = t.size(1);
    ld = t.stride(0);
    if (t.stride(1) != 1 && cols > 1)
      raise(PyExc_ValueError, std::string(name) + " must have unit stride along its rows");
    if (rows <= 1 || cols == 0)
      ld = cols;
    else if (ld < cols)
      raise(PyExc_ValueError, std::string("the rows of ") + name + " overlap");
  }

  Matrix(PyObject* o, const char* name, const Matrix& like, int64_t want_rows, int64_t want_cols)
      : Matrix(o, name, &like) {
    if (rows != want_rows || cols != want_cols)
      raise(PyExc_ValueError, std::string(name) + " must be " + sizes(want_rows, want_cols) +
                                  ", not " + sizes(rows, cols));
  }

  // a new one of ``like``'s type, on its device
  Matrix(const Matrix& like, int64_t r, int64_t c)
      : t(at::empty({r, c}, like.t.options())), rows(r), cols(c), ld(c), code(like.code) {}

  void* p() const { return t.data_ptr(); }
};

// A value for each row, next to each other: the tensor itself, or a copy where it lies otherwise (an
// expanded gradient, as sum() hands it back, or a column of a matrix).  A copy goes back to torch's
// allocator as a workspace does.
at::Tensor row_values(PyObject* o, const char* name, at::ScalarType type, int64_t rows) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != rows)
    raise(PyExc_ValueError, std::string(name) + " must be " +
                                (type == at::kLong ? "an int64" : "a float32") + " tensor of " +
                                std::to_string(rows) + " values");
  return t.contiguous();
}

at::Tensor new_rows(const Matrix& like, int64_t rows) {
  return at::empty({rows}, like.t.options().dtype(at::kFloat));
}

// A workspace of ``bytes`` (none: an undefined tensor).  It goes back to torch's allocator when the
// call returns, which hands it out again only to work that follows on this stream.
struct Workspace {
  at::Tensor t;
  int64_t bytes;
  Workspace(const Matrix& like, int64_t n) : bytes(n) {
    if (n > 0) t = at::empty({n}, like.t.options().dtype(at::kByte));
  }
  void* p() const { return bytes > 0 ? t.data_ptr() : nullptr; }
};

void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

// Runs the C entry point without the interpreter's lock: it may wait for room in the launch queue.
template <typename F>
void enqueue(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  checked(rc);
}

template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* const wrapped[] = {THPVariable_Wrap(t)...};
  PyObject* out = PyTuple_New(sizeof...(T));
  for (size_t i = 0; i < sizeof...(T); ++i) PyTuple_SET_ITEM(out, i, wrapped[i]);
  return out;
}

// (dy, w, out or None) -> dx
PyObject* input_grad(PyObject* const* a) {
  const Matrix dy(a[0], "dy"), w(a[1], "w", &dy);
  if (w.cols != dy.cols)
    raise(PyExc_ValueError, "dy has " + std::to_string(dy.cols) + " columns and w " +
                                std::to_string(w.cols));
  const Matrix dx = a[2] == Py_None ? Matrix(dy, dy.rows, w.rows)
                                    : Matrix(a[2], "out", dy, dy.rows, w.rows);
  const Workspace ws(dy, checked(tg_input_grad_workspace_bytes(dy.rows, w.rows, dy.cols)));
  void* const s = stream();
  enqueue([&] {
    return tg_input_grad(dy.p(), w.p(), dx.p(), dy.rows, w.rows, dy.cols, dy.ld, w.ld, dx.ld, dy.code,
                         ws.p(), ws.bytes, s);
  });
  return THPVariable_Wrap(dx.t);
}

// (x, w_gate, w_up, act, keep, out or None) -> h, or (h, g, u)
PyObject* gated_forward(PyObject* const* a) {
  const Matrix x(a[0], "x"), wg(a[1], "w_gate", &x);
  if (wg.rows != x.cols)
    raise(PyExc_ValueError, "w_gate must have " + std::to_string(x.cols) + " rows, not " +
                                std::to_string(wg.rows));
  const int64_t rows = x.rows, cols = x.cols, outs = wg.cols;
  const Matrix wu(a[2], "w_up", x, cols, outs);
  const int act = static_cast<int>(integer(a[3]));
  const int kept = PyObject_IsTrue(a[4]);
  if (kept < 0) throw PythonError();
  const bool keep = kept != 0;
  const Matrix h = a[5] == Py_None ? Matrix(x, rows, outs) : Matrix(a[5], "out", x, rows, outs);
  const Workspace ws(x, checked(tg_gated_fwd_workspace_bytes(rows, cols, outs)));
  void* const s = stream();
  auto run = [&](void* g, void* u) {
    enqueue([&] {
      return tg_gated_fwd(x.p(), wg.p(), wu.p(), h.p(), g, u, rows, cols, outs, x.ld, wg.ld, wu.ld,
                          h.ld, outs, outs, act, x.code, ws.p(), ws.bytes, s);
    });
  };
  if (!keep) {
    run(nullptr, nullptr);
    return THPVariable_Wrap(h.t);
  }
  const Matrix g(x, rows, outs), u(x, rows, outs);
  run(g.p(), u.p());
  return tuple(h.t, g.t, u.t);
}

// (dh, g, u, x, w_gate, w_up, act) -> (dx, dw_gate, dw_up)
PyObject* gated_backward(PyObject* const* a) {
  const Matrix dh(a[0], "dh");
  const int64_t rows = dh.rows, outs = dh.cols;
  const Matrix g(a[1], "g", dh, rows, outs), u(a[2], "u", dh, rows, outs), x(a[3], "x", &dh);
  if (x.rows != rows)
    raise(PyExc_ValueError, "x must have " + std::to_string(rows) + " rows, not " +
                                std::to_string(x.rows));
  const int64_t cols = x.cols;
  const Matrix wg(a[4], "w_gate", dh, cols, outs), wu(a[5], "w_up", dh, cols, outs);
  const int act = static_cast<int>(integer(a[6]));
  const Matrix dx(dh, rows, cols), dwg(dh, cols, outs), dwu(dh, cols, outs);
  const Workspace ws(dh, checked(tg_gated_bwd_workspace_bytes(rows, cols, outs)));
  void* const s = stream();
  enqueue([&] {
    return tg_gated_bwd(dh.p(), g.p(), u.p(), x.p(), wg.p(), wu.p(), dx.p(), dwg.p(), dwu.p(), rows,
                        cols, outs, dh.ld, g.ld, u.ld, x.ld, wg.ld, wu.ld, cols, outs, outs, act,
                        dh.code, ws.p(), ws.bytes, s);
  });
  return tuple(dx.t, dwg.t, dwu.t);
}

// (x, w, targets, ignore_index) -> (loss, lse)
PyObject* linear_cross_entropy(PyObject* const* a) {
  const Matrix x(a[0], "x"), w(a[1], "w", &x);
  if (w.cols != x.cols)
    raise(PyExc_ValueError, "x has " + std::to_string(x.cols) + " columns and w " +
                                std::to_string(w.cols));
  const at::Tensor targets = row_values(a[2], "targets", at::kLong, x.rows);
  const int64_t ignore = integer(a[3]);
  const at::Tensor loss = new_rows(x, x.rows), lse = new_rows(x, x.rows);
  const Workspace ws(x, checked(tg_xent_fwd_workspace_bytes(x.rows, x.cols, w.rows)));
  void* const s = stream();
  enqueue([&] {
    return tg_xent_fwd(x.p(), w.p(), static_cast<const int64_t*>(targets.data_ptr()),
                       static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()),
                       x.rows, x.cols, w.rows, x.ld, w.ld, ignore, x.code, ws.p(), ws.bytes, s);
  });
  return tuple(loss, lse);
}

// (dloss, x, w, targets, lse, ignore_index) -> (dx, dw)
PyObject* linear_cross_entropy_backward(PyObject* const* a) {
  const Matrix x(a[1], "x"), w(a[2], "w", &x);
  if (w.cols != x.cols)
    raise(PyExc_ValueError, "x has " + std::to_string(x.cols) + " columns and w " +
                                std::to_string(w.cols));
  const at::Tensor dloss = row_values(a[0], "dloss", at::kFloat, x.rows);
  const at::Tensor targets = row_values(a[3], "targets", at::kLong, x.rows);
  const at::Tensor lse = row_values(a[4], "lse", at::kFloat, x.rows);
  const int64_t ignore = integer(a[5]);
  const Matrix dx(x, x.rows, x.cols), dw(x, w.rows, w.cols);
  const Workspace ws(x, checked(tg_xent_bwd_workspace_bytes(x.rows, x.cols, w.rows)));
  void* const s = stream();
  enqueue([&] {
    return tg_xent_bwd(static_cast<const float*>(dloss.data_ptr()), x.p(), w.p(),
                       static_cast<const int64_t*>(targets.data_ptr()),
                       static_cast<const float*>(lse.data_ptr()), dx.p(), dw.p(), x.rows, x.cols,
                       w.rows, x.ld, w.ld, dx.ld, dw.ld, ignore, x.code, ws.p(), ws.bytes, s);
  });
  return tuple(dx.t, dw.t);
}

// The Python function of one of the above, which takes ``N`` arguments.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<input_grad, 3>("input_grad"),
    method<gated_forward, 6>("gated_forward"),
    method<gated_backward, 7>("gated_backward"),
    method<linear_cross_entropy, 4>("linear_cross_entropy"),
    method<linear_cross_entropy_backward, 6>("linear_cross_entropy_backward"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "tg_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tg_torch() { return PyModule_Create(&g_module); }

// ggrn_python.cpp -- the Python entry of the mixer's operators, of layer norm and
// of the backward passes: checks tensors,
// fills the call structures of ggrn.h and makes the calls.
//
// A decode step's kernels take 2 to 4 microseconds; reading the sizes, strides
// and pointers of ten tensors from Python takes 12 to 18.  Here it takes about
// one.  Everything is positional: the documented functions with their keywords
// are in binding.py.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>

#include "../../include/ggrn.h"

namespace {

PyObject* g_error = nullptr;  // callable (status, what): raises

struct Refused {
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse(std::string(name) + " must be a tensor");
  return *t;
}

// (rows, row stride) of a tensor viewed as [rows, width]; an axis of one
// element may have any stride.
void rows_of(const at::Tensor& t, int64_t width, const char* name, int64_t* rows, int64_t* stride) {
  const auto shape = t.sizes();
  const auto strides = t.strides();
  const size_t n = shape.size();
  if (n == 0 || shape[n - 1] != width)
    refuse(std::string(name) + " must have " + std::to_string(width) + " columns");
  if (width != 1 && strides[n - 1] != 1)
    refuse(std::string(name) + " needs unit stride on its last dimension");
  *rows = 1;
  *stride = width;
  if (t.numel() == 0) {
    *rows = 0;
    return;
  }
  for (size_t i = n - 1; i-- > 0;) {
    if (shape[i] == 1) continue;
    if (*rows == 1) *stride = strides[i];
    else if (strides[i] != *stride * *rows)
      refuse(std::string(name) + ": leading axes do not fold into one row axis");
    *rows *= shape[i];
  }
}

int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return GGRN_F32;
    case at::kHalf: return GGRN_F16;
    case at::kBFloat16: return GGRN_BF16;
    default: refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
  }
}

// Pointer of an optional contiguous vector of n elements on x's device.
template <typename T>
const T* vector(PyObject* o, int64_t n, at::ScalarType type, const at::Tensor& x, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->numel() != n || t->device() != x.device() ||
      !t->is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of " +
           std::to_string(n) + " elements on " + x.device().str());
  return static_cast<const T*>(t->const_data_ptr());
}

// The output: given, or made like x.
at::Tensor output(PyObject* o, const at::Tensor& x, const char* name = "out",
                  const char* like = "x") {
  const at::Tensor* t = tensor(o, name);
  if (!t) return at::empty(x.sizes(), x.options().memory_format(c10::nullopt));
  if (t->sizes() != x.sizes() || t->scalar_type() != x.scalar_type() || t->device() != x.device())
    refuse(std::string(name) + " must have the shape, dtype and device of " + like);
  return *t;
}

// A tensor that has to be like x: its address, and its row stride.
const void* alike(PyObject* o, const at::Tensor& x, const char* name, int64_t* stride,
                  const char* like = "x") {
  const at::Tensor& t = needed(o, name);
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.device() != x.device())
    refuse(std::string(name) + " must have the shape, dtype and device of " + like);
  int64_t rows;
  rows_of(t, x.size(-1), name, &rows, stride);
  return t.const_data_ptr();
}
// An output like x: the tensor, its address and its row stride.
at::Tensor output_rows(PyObject* o, const at::Tensor& x, const char* name, void** p,
                       int64_t* stride, const char* like = "x") {
  at::Tensor t = output(o, x, name, like);
  int64_t rows;
  rows_of(t, x.size(-1), name, &rows, stride);
  *p = t.data_ptr();
  return t;
}
at::Tensor new_floats(at::IntArrayRef sizes, const at::Tensor& x) {
  return at::empty(sizes, x.options().dtype(at::kFloat).memory_format(c10::nullopt));
}

// The interpreter's lock given up for a scope (taken again on an exception too).
struct WithoutLock {
  PyThreadState* state = PyEval_SaveThread();
  WithoutLock() = default;
  WithoutLock(const WithoutLock&) = delete;
  ~WithoutLock() { PyEval_RestoreThread(state); }
};

// Sequences and pool of a call: the fields both structures share.
template <typename Call>
void fill_seqs(Call* k, const at::Tensor& x, PyObject* cu_seqlens, PyObject* state_o,
               PyObject* slots, PyObject* resume, at::IntArrayRef held, at::ScalarType type,
               bool step) {
  int64_t n;
  if (step) {
    n = k->rows;
  } else if (cu_seqlens != Py_None) {
    n = needed(cu_seqlens, "cu_seqlens").numel() - 1;
    if (n < 0) refuse("cu_seqlens holds one offset more than there are sequences");
    k->cu_seqlens = vector<int32_t>(cu_seqlens, n + 1, at::kInt, x, "cu_seqlens");
  } else {
    n = 1;
    const auto shape = x.sizes();
    for (size_t i = 0; i + 2 < shape.size(); ++i) n *= shape[i];
  }
  k->seqs = n;
  const at::Tensor* state = tensor(state_o, "state");
  if (!state) {
    if (slots != Py_None || resume != Py_None)
      refuse("slots and resume name entries of a state: pass one");
    return;
  }
  if (state->scalar_type() != type || state->device() != x.device())
    refuse(std::string("state must be a ") + c10::toString(type) + " tensor on " + x.device().str());
  const auto shape = state->sizes();
  const auto strides = state->strides();
  bool fits = shape.size() == held.size() + 1;
  for (size_t i = 0; fits && i < held.size(); ++i) fits = shape[i + 1] == held[i];
  if (!fits) {
    std::string s = "state must be [slots";
    for (int64_t v : held) s += ", " + std::to_string(v);
    refuse(s + "]");
  }
  int64_t expect = 1;
  for (size_t i = shape.size(); i-- > 1;) {
    if (shape[i] != 1 && strides[i] != expect) refuse("the entries of state must be contiguous");
    expect *= shape[i];
  }
  if (slots == Py_None && shape[0] < n)
    refuse("state has " + std::to_string(shape[0]) + " entries for " + std::to_string(n) +
           " sequences");
  using State = decltype(k->state);
  k->state = static_cast<State>(state->data_ptr());
  k->state_slots = shape[0];
  k->state_slot_stride = shape[0] > 1 ? strides[0] : expect;
  k->slots = vector<int32_t>(slots, n, at::kInt, x, "slots");
  if (resume != Py_None) {
    const at::Tensor& r = needed(resume, "resume");
    if (r.scalar_type() != at::kBool && r.scalar_type() != at::kByte)
      refuse("resume must be a bool or uint8 tensor");
    k->resume = vector<uint8_t>(resume, n, r.scalar_type(), x, "resume");
  }
}

// x, weight, bias, activation, cu_seqlens, state, slots, resume, out, step
at::Tensor fill_conv(ggrn_conv_call* k, const at::Tensor*& x_out, PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x");
  x_out = &x;
  if (!x.is_cuda()) refuse("the convolution runs on CUDA tensors only (no CPU path)");
  const bool step = PyObject_IsTrue(a[9]) == 1;
  std::memset(k, 0, sizeof(*k));
  k->dtype = dtype_code(x);
  k->activation = static_cast<int32_t>(PyLong_AsLong(a[3]));
  if (x.dim() < 2) refuse("x must be [rows, width] or [batch, length, width]");
  const at::Tensor& w = needed(a[1], "weight");
  if (w.dim() != 2) refuse("weight must be [width, taps]");
  const int64_t width = x.size(-1), taps = w.size(1);
  rows_of(x, width, "x", &k->rows, &k->x_row_stride);
  k->x = x.const_data_ptr();
  k->width = width;
  k->taps = static_cast<int32_t>(taps);
  k->w = vector<float>(a[1], width * taps, at::kFloat, x, "weight");
  k->bias = vector<float>(a[2], width, at::kFloat, x, "bias");
  at::Tensor out = output(a[8], x);
  int64_t rows;
  rows_of(out, width, "out", &rows, &k->out_row_stride);
  k->out = out.data_ptr();
  const int64_t held[2] = {taps - 1, width};
  fill_seqs(k, x, a[4], a[5], a[6], a[7], held, x.scalar_type(), step);
  return out;
}

// x, dt, a, b, c, head_dim, state_size, d, dt_bias, dt_softplus, dt_min, dt_max,
// cu_seqlens, state, slots, resume, out, step.  Without `make_out` an output that
// is not given is not made either: its address stays NULL and its rows are taken
// for contiguous ones, as those of a new tensor are.
at::Tensor fill_scan(ggrn_scan_call* k, const at::Tensor*& x_out, PyObject* const* a,
                     bool make_out = true) {
  const at::Tensor& x = needed(a[0], "x");
  x_out = &x;
  if (!x.is_cuda()) refuse("the scan runs on CUDA tensors only (no CPU path)");
  const bool step = PyObject_IsTrue(a[17]) == 1;
  std::memset(k, 0, sizeof(*k));
  k->dtype = dtype_code(x);
  if (x.dim() < 2) refuse("x must be [rows, width] or [batch, length, width]");
  const at::Tensor &dt = needed(a[1], "dt"), &b = needed(a[3], "b"), &c = needed(a[4], "c");
  const int64_t width = x.size(-1), heads = needed(a[2], "a").numel();
  if (b.dim() == 0) refuse("b must have the leading shape of x");
  const int64_t gn = b.size(-1), head_dim = PyLong_AsLongLong(a[5]),
                state_size = PyLong_AsLongLong(a[6]);
  if (heads == 0 || head_dim <= 0 || width / head_dim != heads || width % head_dim != 0)
    refuse("x has " + std::to_string(width) + " columns, not " + std::to_string(heads) +
           " heads of " + std::to_string(head_dim));
  if (state_size <= 0 || gn == 0 || gn % state_size != 0)
    refuse("b has " + std::to_string(gn) + " columns, not a multiple of state_size " +
           std::to_string(state_size));
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  const struct { const at::Tensor* t; int64_t n; const char* name; int64_t* stride; } ins[] = {
      {&dt, heads, "dt", &k->dt_row_stride}, {&b, gn, "b", &k->b_row_stride},
      {&c, gn, "c", &k->c_row_stride}};
  int64_t rows;
  rows_of(x, width, "x", &k->rows, &k->x_row_stride);
  for (const auto& i : ins) {
    if (i.t->scalar_type() != x.scalar_type() || i.t->device() != x.device())
      refuse(std::string(i.name) + " must have the dtype and device of x");
    if (i.t->dim() != x.dim() || i.t->size(-1) != i.n ||
        i.t->sizes().slice(0, i.t->dim() - 1) != lead)
      refuse(std::string(i.name) + " must have the leading shape of x and " +
             std::to_string(i.n) + " columns");
    rows_of(*i.t, i.n, i.name, &rows, i.stride);
  }
  k->x = x.const_data_ptr();
  k->dt = dt.const_data_ptr();
  k->b = b.const_data_ptr();
  k->c = c.const_data_ptr();
  k->heads = heads;
  k->head_dim = head_dim;
  k->groups = gn / state_size;
  k->state_size = state_size;
  k->a = vector<float>(a[2], heads, at::kFloat, x, "a");
  k->d = vector<float>(a[7], heads, at::kFloat, x, "d");
  k->dt_bias = vector<float>(a[8], heads, at::kFloat, x, "dt_bias");
  k->dt_softplus = PyObject_IsTrue(a[9]) == 1;
  k->dt_min = static_cast<float>(PyFloat_AsDouble(a[10]));
  k->dt_max = static_cast<float>(PyFloat_AsDouble(a[11]));
  if (PyErr_Occurred()) throw python_error();
  at::Tensor out;
  k->out_row_stride = width;
  if (make_out || a[16] != Py_None) {
    out = output(a[16], x);
    rows_of(out, width, "out", &rows, &k->out_row_stride);
    k->out = out.data_ptr();
  }
  const int64_t held[3] = {heads, head_dim, state_size};
  fill_seqs(k, x, a[12], a[13], a[14], a[15], held, at::kFloat, step);
  return out;
}

// x, input_gate, decay_gate, a, cu_seqlens, state, slots, resume, saved, out, step
at::Tensor fill_recur(ggrn_recur_call* k, const at::Tensor*& x_out, PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x");
  x_out = &x;
  if (!x.is_cuda()) refuse("the recurrence runs on CUDA tensors only (no CPU path)");
  const bool step = PyObject_IsTrue(a[10]) == 1;
  std::memset(k, 0, sizeof(*k));
  k->dtype = dtype_code(x);
  if (x.dim() < 2) refuse("x must be [rows, width] or [batch, length, width]");
  const int64_t width = x.size(-1);
  rows_of(x, width, "x", &k->rows, &k->x_row_stride);
  k->x = x.const_data_ptr();
  k->width = width;
  k->input_gate = alike(a[1], x, "input_gate", &k->input_gate_row_stride);
  k->decay_gate = alike(a[2], x, "decay_gate", &k->decay_gate_row_stride);
  needed(a[3], "a");
  k->a = vector<float>(a[3], width, at::kFloat, x, "a");
  const int64_t kept = (k->rows + GGRN_RECUR_SAVED_ROWS - 1) / GGRN_RECUR_SAVED_ROWS;
  k->saved = const_cast<float*>(vector<float>(a[8], kept * width, at::kFloat, x, "saved"));
  const int64_t held[1] = {width};
  fill_seqs(k, x, a[4], a[5], a[6], a[7], held, at::kFloat, step);
  return output_rows(a[9], x, "out", &k->out, &k->out_row_stride);
}

// x, w, b, eps, out
at::Tensor fill_layer_norm(ggrn_layer_norm_call* k, const at::Tensor*& x_out, PyObject* const* a) {
  const at::Tensor& x = needed(a[0], "x");
  x_out = &x;
  if (!x.is_cuda()) refuse("layer_norm runs on CUDA tensors only (no CPU path)");
  std::memset(k, 0, sizeof(*k));
  k->dtype = dtype_code(x);
  if (x.dim() < 1) refuse("x must have rank >= 1");
  k->width = x.size(-1);
  rows_of(x, k->width, "x", &k->rows, &k->x_row_stride);
  k->x = x.const_data_ptr();
  needed(a[1], "w");
  k->w = vector<float>(a[1], k->width, at::kFloat, x, "w");
  k->b = vector<float>(a[2], k->width, at::kFloat, x, "b");
  k->eps = static_cast<float>(PyFloat_AsDouble(a[3]));
  if (PyErr_Occurred()) throw python_error();
  return output_rows(a[4], x, "out", &k->out, &k->out_row_stride);
}

// A call on its tensors' device and that device's current stream.  The
// interpreter's lock is released for it: a launch waits while the stream's queue
// is full, and other Python threads go on meanwhile.
template <typename Call>
bool made(int (*fn)(const Call*, void*), const Call& k, const at::Tensor& x, const char* what) {
  int st;
  {
    const WithoutLock released;
    const c10::DeviceIndex here = c10::cuda::current_device(), dev = x.device().index();
    if (here == dev) {
      st = fn(&k, c10::cuda::getCurrentCUDAStream(dev).stream());
    } else {
      c10::cuda::CUDAGuard guard(dev);
      st = fn(&k, c10::cuda::getCurrentCUDAStream(dev).stream());
    }
  }
  if (st != GGRN_OK) {
    PyObject* r = PyObject_CallFunction(g_error, "is", st, what);
    Py_XDECREF(r);
    return false;
  }
  return true;
}
template <typename Call>
PyObject* launch(int (*fn)(const Call*, void*), const Call& k, const at::Tensor& x,
                 const at::Tensor& out, const char* what) {
  return made(fn, k, x, what) ? THPVariable_Wrap(out) : nullptr;
}

// A tuple of tensors; an undefined one is None.
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = Py_None;
    if (t.defined()) o = THPVariable_Wrap(t);
    else Py_INCREF(o);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// The workspace that a call asks for, from torch's allocator on x's device.
template <typename Call>
at::Tensor workspace_for(Call* k, int64_t (*bytes_of)(const Call*), const at::Tensor& x) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != x.device().index()) guard.set_device(x.device());
  at::Tensor ws;
  const int64_t bytes = bytes_of(k);
  if (bytes > 0) {
    ws = at::empty({bytes}, x.options().dtype(at::kByte).memory_format(c10::nullopt));
    k->workspace = ws.data_ptr();
    k->workspace_bytes = bytes;
  }
  return ws;
}

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
  return false;
}

PyObject* py_conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_conv_call k;
    const at::Tensor* x;
    const at::Tensor out = fill_conv(&k, x, a);
    const bool step = a[9] == Py_True;
    return launch(step ? ggrn_conv_step : ggrn_conv, k, *x, out,
                  step ? "ggrn_conv_step" : "ggrn_conv");
  });
}

// as fill_scan, and the workspace
PyObject* py_scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 19)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_scan_call k;
    const at::Tensor* x;
    const at::Tensor out = fill_scan(&k, x, a);
    if (a[17] == Py_True) return launch(ggrn_scan_step, k, *x, out, "ggrn_scan_step");
    at::Tensor ws;
    if (a[18] != Py_None) {
      ws = needed(a[18], "workspace");
      if (ws.device() != x->device() || !ws.is_contiguous())
        refuse("workspace must be a contiguous tensor on the device of x");
    } else {
      c10::cuda::OptionalCUDAGuard guard;
      if (c10::cuda::current_device() != x->device().index()) guard.set_device(x->device());
      const int64_t bytes = ggrn_scan_workspace_bytes(&k);
      if (bytes > 0) ws = at::empty({bytes}, x->options().dtype(at::kByte));
    }
    if (ws.defined()) {
      k.workspace = ws.data_ptr();
      k.workspace_bytes = static_cast<int64_t>(ws.nbytes());
    }
    return launch(ggrn_scan, k, *x, out, "ggrn_scan");
  });
}

PyObject* py_scan_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 18)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_scan_call k;
    const at::Tensor* x;
    fill_scan(&k, x, a, /*make_out=*/false);
    c10::cuda::CUDAGuard guard(x->device());
    return PyLong_FromLongLong(ggrn_scan_workspace_bytes(&k));
  });
}

// The call structures as bytes, for decode graphs.
PyObject* py_conv_call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_conv_call k;
    const at::Tensor* x;
    fill_conv(&k, x, a);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&k), sizeof(k));
  });
}
PyObject* py_scan_call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 18)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_scan_call k;
    const at::Tensor* x;
    fill_scan(&k, x, a);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&k), sizeof(k));
  });
}

PyObject* py_recur(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_recur_call k;
    const at::Tensor* x;
    const at::Tensor out = fill_recur(&k, x, a);
    const bool step = a[10] == Py_True;
    return launch(step ? ggrn_recur_step : ggrn_recur, k, *x, out,
                  step ? "ggrn_recur_step" : "ggrn_recur");
  });
}
PyObject* py_recur_call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_recur_call k;
    const at::Tensor* x;
    fill_recur(&k, x, a);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&k), sizeof(k));
  });
}

// dout, x, input_gate, decay_gate, a, cu_seqlens, state, slots, resume, dstate, saved, dx,
// dinput_gate, ddecay_gate
PyObject* py_recur_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_recur_backward_call k;
    std::memset(&k, 0, sizeof(k));
    const at::Tensor& x = needed(a[1], "x");
    if (!x.is_cuda()) refuse("the recurrence runs on CUDA tensors only (no CPU path)");
    k.dtype = dtype_code(x);
    if (x.dim() < 2) refuse("x must be [rows, width] or [batch, length, width]");
    const int64_t width = x.size(-1);
    rows_of(x, width, "x", &k.rows, &k.x_row_stride);
    k.x = x.const_data_ptr();
    k.width = width;
    k.dout = alike(a[0], x, "dout", &k.dout_row_stride);
    k.input_gate = alike(a[2], x, "input_gate", &k.input_gate_row_stride);
    k.decay_gate = alike(a[3], x, "decay_gate", &k.decay_gate_row_stride);
    needed(a[4], "a");
    k.a = vector<float>(a[4], width, at::kFloat, x, "a");
    const int64_t held[1] = {width};
    fill_seqs(&k, x, a[5], a[6], a[7], a[8], held, at::kFloat, false);
    k.dstate = vector<float>(a[9], k.seqs * width, at::kFloat, x, "dstate");
    const int64_t kept = (k.rows + GGRN_RECUR_SAVED_ROWS - 1) / GGRN_RECUR_SAVED_ROWS;
    k.saved = vector<float>(a[10], kept * width, at::kFloat, x, "saved");
    const at::Tensor dx = output_rows(a[11], x, "dx", &k.dx, &k.dx_row_stride),
                     di = output_rows(a[12], x, "dinput_gate", &k.dinput_gate,
                                      &k.dinput_gate_row_stride),
                     dr = output_rows(a[13], x, "ddecay_gate", &k.ddecay_gate,
                                      &k.ddecay_gate_row_stride);
    const at::Tensor da = new_floats({width}, x);
    k.da = static_cast<float*>(da.data_ptr());
    at::Tensor dh;
    if (k.state) {
      dh = new_floats({k.seqs, width}, x);
      k.dinitial = static_cast<float*>(dh.data_ptr());
    }
    const at::Tensor ws = workspace_for(&k, ggrn_recur_backward_workspace_bytes, x);
    if (!made(ggrn_recur_backward, k, x, "ggrn_recur_backward")) return nullptr;
    return tuple_of({dx, di, dr, da, dh});
  });
}

PyObject* py_layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_layer_norm_call k;
    const at::Tensor* x;
    const at::Tensor out = fill_layer_norm(&k, x, a);
    return launch(ggrn_layer_norm, k, *x, out, "ggrn_layer_norm");
  });
}
PyObject* py_layer_norm_call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_layer_norm_call k;
    const at::Tensor* x;
    fill_layer_norm(&k, x, a);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&k), sizeof(k));
  });
}

// dout, x, w, eps, bias, dx
PyObject* py_layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_layer_norm_backward_call k;
    std::memset(&k, 0, sizeof(k));
    const at::Tensor& x = needed(a[1], "x");
    if (!x.is_cuda()) refuse("layer_norm_backward runs on CUDA tensors only (no CPU path)");
    k.dtype = dtype_code(x);
    if (x.dim() < 1) refuse("x must have rank >= 1");
    k.width = x.size(-1);
    rows_of(x, k.width, "x", &k.rows, &k.x_row_stride);
    k.x = x.const_data_ptr();
    k.dout = alike(a[0], x, "dout", &k.dout_row_stride);
    needed(a[2], "w");
    k.w = vector<float>(a[2], k.width, at::kFloat, x, "w");
    k.eps = static_cast<float>(PyFloat_AsDouble(a[3]));
    if (PyErr_Occurred()) throw python_error();
    const at::Tensor dx = output_rows(a[5], x, "dx", &k.dx, &k.dx_row_stride);
    const at::Tensor dw = new_floats({k.width}, x);
    k.dw = static_cast<float*>(dw.data_ptr());
    at::Tensor db;
    if (PyObject_IsTrue(a[4]) == 1) {
      db = new_floats({k.width}, x);
      k.db = static_cast<float*>(db.data_ptr());
    }
    const at::Tensor ws = workspace_for(&k, ggrn_layer_norm_backward_workspace_bytes, x);
    if (!made(ggrn_layer_norm_backward, k, x, "ggrn_layer_norm_backward")) return nullptr;
    return tuple_of({dx, dw, db});
  });
}

// dout, y, gate, w, group_size, eps, mode, dy, dgate
PyObject* py_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    ggrn_backward_call k;
    std::memset(&k, 0, sizeof(k));
    const at::Tensor& y = needed(a[1], "y");
    if (!y.is_cuda()) refuse("backward runs on CUDA tensors only (no CPU path)");
    k.dtype = dtype_code(y);
    if (y.dim() < 1) refuse("y must have rank >= 1");
    k.width = y.size(-1);
    k.group_size = PyLong_AsLongLong(a[4]);
    k.eps = static_cast<float>(PyFloat_AsDouble(a[5]));
    k.mode = static_cast<int32_t>(PyLong_AsLong(a[6]));
    if (PyErr_Occurred()) throw python_error();
    rows_of(y, k.width, "y", &k.rows, &k.y_row_stride);
    k.y = y.const_data_ptr();
    k.dout = alike(a[0], y, "dout", &k.dout_row_stride, "y");
    k.gate = alike(a[2], y, "gate", &k.gate_row_stride, "y");
    const bool onnx = k.mode == GGRN_MODE_ONNX;
    const at::Tensor& w0 = needed(a[3], "w");
    const int64_t columns = onnx ? k.group_size : k.width;
    const at::ScalarType wt = onnx ? y.scalar_type() : at::kFloat;
    if (w0.scalar_type() != wt || w0.numel() != columns || w0.device() != y.device())
      refuse(onnx ? "ONNX scale has the dtype of X and group_size elements"
                  : "MAMBA2 weight is float32 with `width` elements");
    const at::Tensor w = w0.contiguous();
    k.w = w.const_data_ptr();
    const at::Tensor dy = output_rows(a[7], y, "dy", &k.dy, &k.dy_row_stride, "y"),
                     dgate = output_rows(a[8], y, "dgate", &k.dgate, &k.dgate_row_stride, "y");
    const at::Tensor dw = new_floats(w0.sizes(), y);
    k.dw = static_cast<float*>(dw.data_ptr());
    const at::Tensor ws = workspace_for(&k, ggrn_backward_workspace_bytes, y);
    if (!made(ggrn_backward, k, y, "ggrn_backward")) return nullptr;
    return tuple_of({dy, dgate, dw});
  });
}

PyObject* py_rows_of(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 3)) return nullptr;
  return guarded([&]() -> PyObject* {
    int64_t rows, stride;
    rows_of(needed(a[0], "tensor"), PyLong_AsLongLong(a[1]), PyUnicode_AsUTF8(a[2]), &rows, &stride);
    return Py_BuildValue("LL", static_cast<long long>(rows), static_cast<long long>(stride));
  });
}

PyObject* py_on_error(PyObject*, PyObject* f) {
  Py_XDECREF(g_error);
  Py_INCREF(f);
  g_error = f;
  Py_RETURN_NONE;
}

#define FAST(name) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL
PyMethodDef kMethods[] = {{"conv", FAST(py_conv), nullptr},
                          {"scan", FAST(py_scan), nullptr},
                          {"scan_workspace_bytes", FAST(py_scan_workspace), nullptr},
                          {"conv_call", FAST(py_conv_call), nullptr},
                          {"scan_call", FAST(py_scan_call), nullptr},
                          {"recur", FAST(py_recur), nullptr},
                          {"recur_call", FAST(py_recur_call), nullptr},
                          {"recur_backward", FAST(py_recur_backward), nullptr},
                          {"layer_norm", FAST(py_layer_norm), nullptr},
                          {"layer_norm_call", FAST(py_layer_norm_call), nullptr},
                          {"layer_norm_backward", FAST(py_layer_norm_backward), nullptr},
                          {"norm_backward", FAST(py_norm_backward), nullptr},
                          {"rows_of", FAST(py_rows_of), nullptr},
                          {"on_error", py_on_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }

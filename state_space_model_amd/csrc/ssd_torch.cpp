// The operators between two scans, and the gated delta rule, as Python calls on
// torch tensors: checks of the arguments, outputs and workspace from torch's
// allocator, the C ABI on the current stream.  Host code only; _ssd_torch.so,
// next to libssd.so.
//
// It exists for the calls that a token makes one at a time, which the host
// bounds: a norm of one token needs the GPU for 2 us and 3.1 us of the host for
// its launch.  Per call, against the same checks and allocations made from
// Python: one-token add norm 4.7-5.6 us (8.2), add norm and 8-bit product 11.0 us
// (19.7), gradients of the gated norm 10.4 us (15.8).
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "ssd.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
using Shape = c10::SmallVector<int64_t, 6>;

PyObject* g_error = nullptr;           // SSDError(status, where)
PyObject* g_stream = nullptr;          // device index -> the current stream's handle
PyObject* g_current_device = nullptr;  // () -> the current device's index
PyObject* g_set_device = nullptr;      // device index -> None: made current

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------
std::string text(IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// NULL for None
const Tensor* maybe(PyObject* o, const char* name) {
  return !o || o == Py_None ? nullptr : &tensor(o, name);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

int32_t io_code(ScalarType t, const char* name) {
  if (t == at::kFloat) return SSD_F32;
  TORCH_CHECK_TYPE(t == at::kBFloat16, name, " must be float32 or bfloat16, got ", t);
  return SSD_BF16;
}

// The ABI receives bare pointers and cannot see a buffer's extent, so every
// tensor's shape is checked here.
void shape(const Tensor* t, const char* name, IntArrayRef want) {
  TORCH_CHECK_VALUE(!t || t->sizes() == want, name, " must have shape ", text(want), ", got ",
                    text(t->sizes()));
}

void device(const Tensor& t, const char* name, const Tensor& first) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a device tensor (got ", t.device(),
                    "); there is no CPU path");
  TORCH_CHECK_VALUE(t.get_device() == first.get_device(), name, " must be on ", first.device(),
                    " with the first argument, got ", t.device());
}

void dtype(const Tensor& t, const char* name, ScalarType want) {
  TORCH_CHECK_TYPE(t.scalar_type() == want, name, " must be ", want, ", got ", t.scalar_type());
}

void dense(const Tensor* t, const char* name, ScalarType want, const Tensor& first) {
  if (!t) return;
  device(*t, name, first);
  TORCH_CHECK_VALUE(t->is_contiguous(), name, " must be contiguous");
  dtype(*t, name, want);
}

// Elements between the rows of t [..., D], whose rows must be dense and evenly
// spaced (a slice of a projection's columns is).  One dimension is one row.
int64_t row_stride(const Tensor& t, const char* name) {
  const int64_t n = t.dim();
  const int64_t D = n ? t.size(n - 1) : 1;
  if (t.numel() == 0) return n < 2 ? D : std::max(t.stride(n - 2), D);
  bool ok = n == 0 || t.stride(n - 1) == 1 || D == 1;
  int64_t rows = 1, step = -1;
  for (int64_t d = n - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (step < 0) step = t.stride(d);
    ok = ok && t.stride(d) == step * rows;
    rows *= t.size(d);
  }
  if (step < 0) step = D;
  TORCH_CHECK_VALUE(ok && step >= D, name, " must have dense, evenly spaced rows (shape ",
                    text(t.sizes()), ", strides ", text(t.strides()), ")");
  return step;
}

int64_t spaced(const Tensor& t, const char* name, ScalarType want, const Tensor& first) {
  device(t, name, first);
  dtype(t, name, want);
  return row_stride(t, name);
}

// ---------------------------------------------------------------------------
// outputs
// ---------------------------------------------------------------------------
// the caller's buffer, checked (its shape was), or a new one
Tensor output(const Tensor* t, const char* name, IntArrayRef sizes, ScalarType type,
              const Tensor& first) {
  if (!t) return at::empty(sizes, first.options().dtype(type));
  dense(t, name, type, first);
  return *t;
}

Shape rows_of(const Tensor& x) { return Shape(x.sizes().begin(), x.sizes().end() - 1); }

Shape with_cols(const Tensor& x, int64_t cols) {
  Shape s(x.sizes().begin(), x.sizes().end());
  s.back() = cols;
  return s;
}

int64_t q8_cols(int64_t cols) { return (cols + SSD_Q8_PAD - 1) / SSD_Q8_PAD * SSD_Q8_PAD; }

int64_t rows(const Tensor& x) { return x.numel() / std::max<int64_t>(x.size(-1), 1); }

// the caller's gradient buffers, by name
struct Grads {
  PyObject* dict;
  Grads(PyObject* o, std::initializer_list<const char*> names)
      : dict(o == Py_None ? nullptr : o) {
    if (!dict) return;
    TORCH_CHECK_TYPE(PyDict_Check(dict), "grads must be a dict, got ", Py_TYPE(dict)->tp_name);
    PyObject *key, *value;
    for (Py_ssize_t at = 0; PyDict_Next(dict, &at, &key, &value);) {
      const char* k = PyUnicode_Check(key) ? PyUnicode_AsUTF8(key) : nullptr;
      if (!k) PyErr_Clear();
      bool known = false;
      for (const char* n : names) known = known || (k && std::string(k) == n);
      TORCH_CHECK_VALUE(known, "unknown gradient name ", k ? k : "that is no text");
    }
  }
  const Tensor* get(const char* name, IntArrayRef sizes) const {
    const Tensor* t = dict ? maybe(PyDict_GetItemString(dict, name), name) : nullptr;
    shape(t, name, sizes);
    return t;
  }
};

Tensor workspace(const Tensor* given, size_t bytes, const Tensor& first) {
  if (!given) {
    return at::empty({std::max<int64_t>((int64_t)bytes, 1)}, first.options().dtype(at::kByte));
  }
  dense(given, "workspace", given->scalar_type(), first);
  return *given;
}

void* ptr(const Tensor& t) { return t.data_ptr(); }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
float* f32(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }
float* f32(const Tensor* t) { return t ? f32(*t) : nullptr; }
int8_t* i8(const Tensor& t) { return static_cast<int8_t*>(t.data_ptr()); }

// a call's result as a number (None: 0)
int64_t number_of(PyObject* r) {
  if (!r) throw python_error();
  const int64_t v = r == Py_None ? 0 : (int64_t)PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  if (PyErr_Occurred()) throw python_error();
  return v;
}
int64_t ask(PyObject* f) { return number_of(PyObject_CallNoArgs(f)); }
int64_t ask(PyObject* f, int64_t index) {
  PyObject* i = PyLong_FromLongLong(index);
  if (!i) throw python_error();
  PyObject* r = PyObject_CallOneArg(f, i);
  Py_DECREF(i);
  return number_of(r);
}

// The device of a call's tensors, current while the call launches: the handle
// of the default stream is the same for every device and means the current
// one's.
class OnDevice {
 public:
  explicit OnDevice(int64_t index)
      : previous_(ask(g_current_device)), moved_(index != previous_) {
    if (moved_) ask(g_set_device, index);
  }
  ~OnDevice() {
    if (!moved_) return;
    try {
      ask(g_set_device, previous_);
    } catch (python_error&) {
      PyErr_WriteUnraisable(g_set_device);
    }
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;

 private:
  int64_t previous_;
  bool moved_;
};

// f(stream) -> status on the current stream of the first argument's device
template <typename F>
void launch(const Tensor& first, const char* where, F&& f) {
  const int64_t index = first.get_device();
  ssd_status st;
  {
    const auto s = reinterpret_cast<hipStream_t>((uintptr_t)ask(g_stream, index));
    const OnDevice on(index);
    st = f(s);
  }
  if (st == SSD_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, where);
  if (e) PyErr_SetObject(g_error, e);
  Py_XDECREF(e);
  throw python_error();
}

// ---------------------------------------------------------------------------
// results
// ---------------------------------------------------------------------------
PyObject* wrap(const Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw python_error();
  return o;
}

PyObject* tuple(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = THPVariable_Wrap(*t);
    if (!o) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

PyObject* dict(std::initializer_list<std::pair<const char*, const Tensor*>> ts) {
  PyObject* r = PyDict_New();
  if (!r) throw python_error();
  for (const auto& [name, t] : ts) {
    PyObject* o = THPVariable_Wrap(*t);
    const bool bad = !o || PyDict_SetItemString(r, name, o) < 0;
    Py_XDECREF(o);
    if (bad) {
      Py_DECREF(r);
      throw python_error();
    }
  }
  return r;
}

// ---------------------------------------------------------------------------
// the operators: positional arguments, as the Python functions pass them
// ---------------------------------------------------------------------------
void vectors(const Tensor& x, const Tensor& weight, const char* what) {
  TORCH_CHECK_VALUE(x.dim() >= 1 && weight.dim() == 1, what);
}

// x, weight, residual, scale, eps, y, residual_out
PyObject* add_norm(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
  const Tensor *residual = maybe(a[2], "residual"), *y_ = maybe(a[5], "y"),
               *r_ = maybe(a[6], "residual_out");
  vectors(x, weight, "x [..., D], weight [D]");
  const int64_t D = x.size(-1);
  shape(y_, "y", x.sizes());
  shape(&weight, "weight", D);
  shape(residual, "residual", x.sizes());
  shape(r_, "residual_out", x.sizes());
  const ScalarType io = x.scalar_type();
  const ssd_add_norm_desc desc{rows(x), D, io_code(io, "x"), (float)number(a[3]),
                               (float)number(a[4])};
  dense(&x, "x", io, x);
  dense(&weight, "weight", at::kFloat, x);
  dense(residual, "residual", at::kFloat, x);
  const Tensor r = output(r_, "residual_out", x.sizes(), at::kFloat, x);
  const Tensor y = output(y_, "y", x.sizes(), io, x);
  launch(x, "ssd_add_norm", [&](hipStream_t stream) {
    return ssd_add_norm(&desc, ptr(x), f32(residual), f32(weight), ptr(y), f32(r), stream);
  });
  return tuple({&y, &r});
}

// x, weight, residual, scale, eps, q, qscale, residual_out
PyObject* add_norm_q8(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
  const Tensor *residual = maybe(a[2], "residual"), *q_ = maybe(a[5], "q"),
               *s_ = maybe(a[6], "qscale"), *r_ = maybe(a[7], "residual_out");
  vectors(x, weight, "x [..., D], weight [D]");
  const int64_t D = x.size(-1);
  const Shape qshape = with_cols(x, q8_cols(D)), lead = rows_of(x);
  shape(q_, "q", qshape);
  shape(s_, "qscale", lead);
  shape(&weight, "weight", D);
  shape(residual, "residual", x.sizes());
  shape(r_, "residual_out", x.sizes());
  const ScalarType io = x.scalar_type();
  const ssd_add_norm_desc desc{rows(x), D, io_code(io, "x"), (float)number(a[3]),
                               (float)number(a[4])};
  dense(&x, "x", io, x);
  dense(&weight, "weight", at::kFloat, x);
  dense(residual, "residual", at::kFloat, x);
  const Tensor r = output(r_, "residual_out", x.sizes(), at::kFloat, x);
  const Tensor q = output(q_, "q", qshape, at::kChar, x);
  const Tensor s = output(s_, "qscale", lead, at::kFloat, x);
  launch(x, "ssd_add_norm_q8", [&](hipStream_t stream) {
    return ssd_add_norm_q8(&desc, ptr(x), f32(residual), f32(weight), i8(q), f32(s), f32(r),
                           stream);
  });
  return tuple({&q, &s, &r});
}

// residual_out, weight, dy, dresidual_out, scale, eps, workspace, grads
PyObject* add_norm_backward(PyObject* const* a) {
  const Tensor &r = tensor(a[0], "residual_out"), &weight = tensor(a[1], "weight"),
               &dy = tensor(a[2], "dy");
  const Tensor *dr = maybe(a[3], "dresidual_out"), *w_ = maybe(a[6], "workspace");
  vectors(r, weight, "residual_out [..., D], weight [D]");
  const int64_t D = r.size(-1);
  shape(&weight, "weight", D);
  shape(&dy, "dy", r.sizes());
  shape(dr, "dresidual_out", r.sizes());
  const ScalarType io = dy.scalar_type();
  const ssd_add_norm_desc desc{rows(r), D, io_code(io, "dy"), (float)number(a[4]),
                               (float)number(a[5])};
  const Grads g(a[7], {"dx", "dresidual", "dweight"});
  const Tensor *dx_ = g.get("dx", r.sizes()), *dr_ = g.get("dresidual", r.sizes()),
               *dw_ = g.get("dweight", D);
  dense(&r, "residual_out", at::kFloat, r);
  dense(&weight, "weight", at::kFloat, r);
  dense(&dy, "dy", io, r);
  dense(dr, "dresidual_out", at::kFloat, r);
  const Tensor dx = output(dx_, "dx", r.sizes(), io, r);
  const Tensor dresidual = output(dr_, "dresidual", r.sizes(), at::kFloat, r);
  const Tensor dweight = output(dw_, "dweight", D, at::kFloat, r);
  const Tensor ws = workspace(w_, ssd_add_norm_backward_workspace_bytes(&desc), r);
  launch(r, "ssd_add_norm_backward", [&](hipStream_t stream) {
    return ssd_add_norm_backward(&desc, f32(r), f32(weight), ptr(dy), f32(dr), ptr(dx),
                                 f32(dresidual), f32(dweight), ptr(ws), ws.nbytes(), stream);
  });
  return dict({{"dx", &dx}, {"dresidual", &dresidual}, {"dweight", &dweight}});
}

// seed and offset of the dropout's generator
const int64_t* generator(const Tensor& rng, const Tensor& first) {
  shape(&rng, "rng", 2);
  dense(&rng, "rng", at::kLong, first);
  return static_cast<const int64_t*>(rng.data_ptr());
}

// x, weight, residual, p, rng, scale, eps, y, residual_out
PyObject* dropout_add_norm(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight"), &rng = tensor(a[4], "rng");
  const Tensor *residual = maybe(a[2], "residual"), *y_ = maybe(a[7], "y"),
               *r_ = maybe(a[8], "residual_out");
  vectors(x, weight, "x [..., D], weight [D]");
  const int64_t D = x.size(-1);
  shape(y_, "y", x.sizes());
  shape(&weight, "weight", D);
  shape(residual, "residual", x.sizes());
  shape(r_, "residual_out", x.sizes());
  const ScalarType io = x.scalar_type();
  const ssd_dropout_add_norm_desc desc{rows(x), D, io_code(io, "x"), (float)number(a[5]),
                                       (float)number(a[6]), number(a[3])};
  dense(&x, "x", io, x);
  dense(&weight, "weight", at::kFloat, x);
  dense(residual, "residual", at::kFloat, x);
  const int64_t* state = generator(rng, x);
  const Tensor r = output(r_, "residual_out", x.sizes(), at::kFloat, x);
  const Tensor y = output(y_, "y", x.sizes(), io, x);
  launch(x, "ssd_dropout_add_norm", [&](hipStream_t stream) {
    return ssd_dropout_add_norm(&desc, ptr(x), f32(residual), f32(weight), state, ptr(y), f32(r), stream);
  });
  return tuple({&y, &r});
}

// residual_out, weight, dy, dresidual_out, p, rng, scale, eps, workspace, grads
PyObject* dropout_add_norm_backward(PyObject* const* a) {
  const Tensor &r = tensor(a[0], "residual_out"), &weight = tensor(a[1], "weight"),
               &dy = tensor(a[2], "dy"), &rng = tensor(a[5], "rng");
  const Tensor *dr = maybe(a[3], "dresidual_out"), *w_ = maybe(a[8], "workspace");
  vectors(r, weight, "residual_out [..., D], weight [D]");
  const int64_t D = r.size(-1);
  shape(&weight, "weight", D);
  shape(&dy, "dy", r.sizes());
  shape(dr, "dresidual_out", r.sizes());
  const ScalarType io = dy.scalar_type();
  const ssd_dropout_add_norm_desc desc{rows(r), D, io_code(io, "dy"), (float)number(a[6]),
                                       (float)number(a[7]), number(a[4])};
  const Grads g(a[9], {"dx", "dresidual", "dweight"});
  const Tensor *dx_ = g.get("dx", r.sizes()), *dr_ = g.get("dresidual", r.sizes()),
               *dw_ = g.get("dweight", D);
  dense(&r, "residual_out", at::kFloat, r);
  dense(&weight, "weight", at::kFloat, r);
  dense(&dy, "dy", io, r);
  dense(dr, "dresidual_out", at::kFloat, r);
  const int64_t* state = generator(rng, r);
  const Tensor dx = output(dx_, "dx", r.sizes(), io, r);
  const Tensor dresidual = output(dr_, "dresidual", r.sizes(), at::kFloat, r);
  const Tensor dweight = output(dw_, "dweight", D, at::kFloat, r);
  const Tensor ws = workspace(w_, ssd_dropout_add_norm_backward_workspace_bytes(&desc), r);
  launch(r, "ssd_dropout_add_norm_backward", [&](hipStream_t stream) {
    return ssd_dropout_add_norm_backward(&desc, f32(r), f32(weight), ptr(dy), f32(dr), state, ptr(dx),
                                         f32(dresidual), f32(dweight), ptr(ws), ws.nbytes(), stream);
  });
  return dict({{"dx", &dx}, {"dresidual", &dresidual}, {"dweight", &dweight}});
}

ssd_gated_norm_desc gated_desc(const Tensor& y, const Tensor& z, const Tensor& weight,
                               PyObject* groups, PyObject* eps) {
  const ScalarType io = y.scalar_type();
  const int32_t code = io_code(io, "y");
  dense(&y, "y", io, y);
  dense(&weight, "weight", at::kFloat, y);
  const int64_t stride = spaced(z, "z", io, y);
  return {rows(y), y.size(-1), integer(groups), stride, 0, code, (float)number(eps)};
}

// y, z, weight, groups, eps, out
PyObject* gated_norm(PyObject* const* a) {
  const Tensor &y = tensor(a[0], "y"), &z = tensor(a[1], "z"), &weight = tensor(a[2], "weight");
  const Tensor* o_ = maybe(a[5], "out");
  vectors(y, weight, "y [..., D], z [..., D], weight [D]");
  shape(o_, "out", y.sizes());
  shape(&z, "z", y.sizes());
  shape(&weight, "weight", y.size(-1));
  const ssd_gated_norm_desc desc = gated_desc(y, z, weight, a[3], a[4]);
  const Tensor out = output(o_, "out", y.sizes(), y.scalar_type(), y);
  launch(y, "ssd_gated_norm", [&](hipStream_t stream) {
    return ssd_gated_norm(&desc, ptr(y), ptr(z), f32(weight), ptr(out), stream);
  });
  return wrap(out);
}

// y, z, weight, groups, eps, q, qscale
PyObject* gated_norm_q8(PyObject* const* a) {
  const Tensor &y = tensor(a[0], "y"), &z = tensor(a[1], "z"), &weight = tensor(a[2], "weight");
  const Tensor *q_ = maybe(a[5], "q"), *s_ = maybe(a[6], "qscale");
  vectors(y, weight, "y [..., D], z [..., D], weight [D]");
  const Shape qshape = with_cols(y, q8_cols(y.size(-1))), lead = rows_of(y);
  shape(q_, "q", qshape);
  shape(s_, "qscale", lead);
  shape(&z, "z", y.sizes());
  shape(&weight, "weight", y.size(-1));
  const ssd_gated_norm_desc desc = gated_desc(y, z, weight, a[3], a[4]);
  const Tensor q = output(q_, "q", qshape, at::kChar, y);
  const Tensor s = output(s_, "qscale", lead, at::kFloat, y);
  launch(y, "ssd_gated_norm_q8", [&](hipStream_t stream) {
    return ssd_gated_norm_q8(&desc, ptr(y), ptr(z), f32(weight), i8(q), f32(s), stream);
  });
  return tuple({&q, &s});
}

// y, z, weight, dout, groups, eps, workspace, grads
PyObject* gated_norm_backward(PyObject* const* a) {
  const Tensor &y = tensor(a[0], "y"), &z = tensor(a[1], "z"), &weight = tensor(a[2], "weight"),
               &dout = tensor(a[3], "dout");
  const Tensor* w_ = maybe(a[6], "workspace");
  vectors(y, weight, "y [..., D], z [..., D], weight [D]");
  const int64_t D = y.size(-1);
  shape(&z, "z", y.sizes());
  shape(&weight, "weight", D);
  shape(&dout, "dout", y.sizes());
  const Grads g(a[7], {"dy", "dz", "dweight"});
  const Tensor *dy_ = g.get("dy", y.sizes()), *dz_ = g.get("dz", y.sizes()),
               *dw_ = g.get("dweight", D);
  const ScalarType io = y.scalar_type();
  ssd_gated_norm_desc desc = gated_desc(y, z, weight, a[4], a[5]);
  dense(&dout, "dout", io, y);
  desc.dz_stride = dz_ ? spaced(*dz_, "dz", io, y) : D;
  const Tensor dz = dz_ ? *dz_ : output(nullptr, "dz", y.sizes(), io, y);
  const Tensor dy = output(dy_, "dy", y.sizes(), io, y);
  const Tensor dweight = output(dw_, "dweight", D, at::kFloat, y);
  const Tensor ws = workspace(w_, ssd_gated_norm_backward_workspace_bytes(&desc), y);
  launch(y, "ssd_gated_norm_backward", [&](hipStream_t stream) {
    return ssd_gated_norm_backward(&desc, ptr(y), ptr(z), f32(weight), ptr(dout), ptr(dy), ptr(dz),
                                   f32(dweight), ptr(ws), ws.nbytes(), stream);
  });
  return dict({{"dy", &dy}, {"dz", &dz}, {"dweight", &dweight}});
}

// v, q, qscale
PyObject* quantize_q8(PyObject* const* a) {
  const Tensor& v = tensor(a[0], "v");
  const Tensor *q_ = maybe(a[1], "q"), *s_ = maybe(a[2], "qscale");
  TORCH_CHECK_VALUE(v.dim() >= 1, "v [..., K]");
  const int64_t K = v.size(-1);
  const Shape qshape = with_cols(v, q8_cols(K)), lead = rows_of(v);
  shape(q_, "q", qshape);
  shape(s_, "qscale", lead);
  const int32_t code = io_code(v.scalar_type(), "v");
  dense(&v, "v", v.scalar_type(), v);
  const Tensor q = output(q_, "q", qshape, at::kChar, v);
  const Tensor s = output(s_, "qscale", lead, at::kFloat, v);
  launch(v, "ssd_quantize_q8", [&](hipStream_t stream) {
    return ssd_quantize_q8(rows(v), K, code, ptr(v), i8(q), f32(s), stream);
  });
  return tuple({&q, &s});
}

// q, qscale, wq, wscale, bfloat16, out
PyObject* linear_q8(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &qscale = tensor(a[1], "qscale"), &wq = tensor(a[2], "wq"),
               &wscale = tensor(a[3], "wscale");
  const Tensor* o_ = maybe(a[5], "out");
  TORCH_CHECK_VALUE(q.dim() >= 1 && wq.dim() == 2, "q [..., Kp], wq [N, Kp]");
  const int64_t Kp = q.size(-1), N = wq.size(0);
  const ScalarType io = o_ ? o_->scalar_type() : a[4] == Py_True ? at::kBFloat16 : at::kFloat;
  const Shape oshape = with_cols(q, N);
  shape(&wq, "wq", {N, Kp});
  shape(&qscale, "qscale", rows_of(q));
  shape(&wscale, "wscale", N);
  shape(o_, "out", oshape);
  const ssd_linear_q8_desc desc{rows(q), Kp, N, io_code(io, "out")};
  dense(&q, "q", at::kChar, q);
  dense(&qscale, "qscale", at::kFloat, q);
  dense(&wq, "wq", at::kChar, q);
  dense(&wscale, "wscale", at::kFloat, q);
  const Tensor out = output(o_, "out", oshape, io, q);
  launch(q, "ssd_linear_q8", [&](hipStream_t stream) {
    return ssd_linear_q8(&desc, i8(q), f32(qscale), i8(wq), f32(wscale), ptr(out), stream);
  });
  return wrap(out);
}

// x, weight, bias, dy, state, dstate_out, silu, workspace, grads
PyObject* conv1d_backward(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight"), &dy = tensor(a[3], "dy");
  const Tensor *bias = maybe(a[2], "bias"), *state = maybe(a[4], "state"),
               *ds = maybe(a[5], "dstate_out"), *w_ = maybe(a[7], "workspace");
  TORCH_CHECK_VALUE(x.dim() == 3 && weight.dim() == 2 && weight.size(0) == x.size(2),
                    "x [Bt,T,D], weight [D,k]");
  const int64_t Bt = x.size(0), T = x.size(1), D = x.size(2), K = weight.size(1);
  TORCH_CHECK_VALUE(K >= 1, "weight [D,k] with k >= 1");
  const int64_t window[3] = {Bt, D, K - 1};
  shape(&dy, "dy", x.sizes());
  shape(bias, "bias", D);
  shape(state, "state", window);
  shape(ds, "dstate_out", window);
  const Grads g(a[8], {"dx", "dweight", "dbias", "dstate"});
  const Tensor *dx_ = g.get("dx", x.sizes()), *dw_ = g.get("dweight", weight.sizes()),
               *db_ = g.get("dbias", D), *dst_ = g.get("dstate", window);
  const ScalarType io = x.scalar_type();
  const int32_t code = io_code(io, "x");
  const ScalarType cot = dy.scalar_type() == at::kFloat ? at::kFloat : io;
  dense(&x, "x", io, x);
  dense(&weight, "weight", at::kFloat, x);
  dense(bias, "bias", at::kFloat, x);
  dense(state, "state", io, x);
  dense(&dy, "dy", cot, x);
  dense(ds, "dstate_out", io, x);
  const Tensor dx = output(dx_, "dx", x.sizes(), io, x);
  const Tensor dweight = output(dw_, "dweight", weight.sizes(), at::kFloat, x);
  const Tensor dbias = output(db_, "dbias", D, at::kFloat, x);
  const Tensor dstate = output(dst_, "dstate", window, io, x);
  const int silu = PyObject_IsTrue(a[6]);
  if (silu < 0) throw python_error();
  const ssd_conv_desc desc{Bt, T, D, K, code, silu};
  const Tensor ws = workspace(w_, ssd_conv1d_backward_workspace_bytes(&desc), x);
  launch(x, "ssd_conv1d_backward", [&](hipStream_t stream) {
    return ssd_conv1d_backward(&desc, io_code(cot, "dy"), ptr(x), f32(weight), f32(bias),
                               ptr(state), ptr(dy), ptr(ds), ptr(dx), f32(dweight), f32(dbias),
                               ptr(dstate), ptr(ws), ws.nbytes(), stream);
  });
  return dict({{"dx", &dx}, {"dweight", &dweight}, {"dbias", &dbias}, {"dstate", &dstate}});
}

// Elements between the tokens of t [..., heads, size], whose heads must be
// dense and whose tokens evenly spaced (a slice of the convolution's output is).
int64_t token_stride(const Tensor& t, const char* name, ScalarType want, const Tensor& first) {
  device(t, name, first);
  dtype(t, name, want);
  const int64_t n = t.dim(), size = t.size(n - 1), heads = t.size(n - 2), D = heads * size;
  if (t.numel() == 0) return D;
  bool ok = (t.stride(n - 1) == 1 || size == 1) && (t.stride(n - 2) == size || heads == 1);
  int64_t rows = 1, step = -1;
  for (int64_t d = n - 3; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (step < 0) step = t.stride(d);
    ok = ok && t.stride(d) == step * rows;
    rows *= t.size(d);
  }
  if (step < 0) step = D;
  TORCH_CHECK_VALUE(ok && step >= D, name, " must have dense heads and evenly spaced tokens (shape ",
                    text(t.sizes()), ", strides ", text(t.strides()), ")");
  return step;
}

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}

// The inputs of the gated delta rule: q, k, v, dt, A, beta, dt_bias, then
// dt_softplus, dt_min, dt_max, beta_sigmoid, qk_norm, norm_eps, scale (None:
// 1/sqrt(N)).  q and k [.., G, N], v [.., H, P], with one leading dimension for
// a token and two for a sequence.
constexpr int kDeltaInputs = 14;
struct Delta {
  const Tensor &q, &k, &v, &dt, &A, &beta;
  const Tensor* bias;
  ssd_delta_desc d;
  Shape yshape, state;
  ScalarType io;
  Delta(PyObject* const* a, bool step)
      : q(tensor(a[0], "q")), k(tensor(a[1], "k")), v(tensor(a[2], "v")), dt(tensor(a[3], "dt")),
        A(tensor(a[4], "A")), beta(tensor(a[5], "beta")), bias(maybe(a[6], "dt_bias")), d() {
    const int64_t lead = step ? 1 : 2;
    TORCH_CHECK_VALUE(v.dim() == lead + 2 && q.dim() == lead + 2,
                      step ? "q_t, k_t [Bt,G,N], v_t [Bt,H,P]" : "q, k [Bt,T,G,N], v [Bt,T,H,P]");
    d.batch = v.size(0);
    d.seqlen = step ? 1 : v.size(1);
    d.nheads = v.size(lead);
    d.headdim = v.size(lead + 1);
    d.ngroups = q.size(lead);
    d.dstate = q.size(lead + 1);
    Shape qk(v.sizes().begin(), v.sizes().begin() + lead), gate(qk);
    qk.push_back(d.ngroups);
    qk.push_back(d.dstate);
    gate.push_back(d.nheads);
    shape(&q, "q", qk);
    shape(&k, "k", qk);
    shape(&dt, "dt", gate);
    shape(&beta, "beta", gate);
    shape(&A, "A", d.nheads);
    shape(bias, "dt_bias", d.nheads);
    yshape = Shape(v.sizes().begin(), v.sizes().end());
    state = Shape{d.batch, d.nheads, d.headdim, d.dstate};
    io = v.scalar_type();
    d.io_dtype = io_code(io, "v");
    d.v_stride = token_stride(v, "v", io, v);
    d.q_stride = token_stride(q, "q", io, v);
    d.k_stride = token_stride(k, "k", io, v);
    dense(&dt, "dt", at::kFloat, v);
    dense(&A, "A", at::kFloat, v);
    dense(&beta, "beta", at::kFloat, v);
    dense(bias, "dt_bias", at::kFloat, v);
    d.dt_softplus = flag(a[7]);
    d.dt_min = (float)number(a[8]);
    d.dt_max = (float)number(a[9]);
    d.beta_sigmoid = flag(a[10]);
    d.qk_norm = flag(a[11]);
    d.norm_eps = (float)number(a[12]);
    d.scale = a[13] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(d.dstate, 1)))
                               : (float)number(a[13]);
  }
};

// the inputs, initial_state, return_final_state, y, final_state, workspace
PyObject* delta_scan(PyObject* const* a) {
  const Delta in(a, false);
  const Tensor *h0 = maybe(a[kDeltaInputs], "initial_state"),
               *y_ = maybe(a[kDeltaInputs + 2], "y"),
               *f_ = maybe(a[kDeltaInputs + 3], "final_state"),
               *w_ = maybe(a[kDeltaInputs + 4], "workspace");
  shape(h0, "initial_state", in.state);
  shape(y_, "y", in.yshape);
  shape(f_, "final_state", in.state);
  dense(h0, "initial_state", at::kFloat, in.v);
  const bool keep = f_ || flag(a[kDeltaInputs + 1]);
  const Tensor y = output(y_, "y", in.yshape, in.io, in.v);
  const Tensor f = keep ? output(f_, "final_state", in.state, at::kFloat, in.v) : Tensor();
  const Tensor ws = workspace(w_, ssd_delta_scan_workspace_bytes(&in.d), in.v);
  launch(in.v, "ssd_delta_scan", [&](hipStream_t stream) {
    return ssd_delta_scan(&in.d, ptr(in.q), ptr(in.k), ptr(in.v), f32(in.dt), f32(in.bias),
                          f32(in.A), f32(in.beta), f32(h0), ptr(y), keep ? f32(f) : nullptr, ptr(ws),
                          ws.nbytes(), stream);
  });
  PyObject* r = tuple({&y, keep ? &f : &y});
  if (!keep) {
    Py_INCREF(Py_None);
    PyTuple_SetItem(r, 1, Py_None);
  }
  return r;
}

// the inputs, dy, dfinal_state, initial_state, workspace, grads
PyObject* delta_scan_backward(PyObject* const* a) {
  Delta in(a, false);
  a += kDeltaInputs;
  const Tensor& dy = tensor(a[0], "dy");
  const Tensor *df = maybe(a[1], "dfinal_state"), *h0 = maybe(a[2], "initial_state"),
               *w_ = maybe(a[3], "workspace");
  const int64_t H = in.d.nheads;
  const IntArrayRef qk = in.q.sizes(), gate = in.dt.sizes();
  shape(&dy, "dy", in.yshape);
  shape(df, "dfinal_state", in.state);
  shape(h0, "initial_state", in.state);
  const Grads g(a[4], {"dq", "dk", "dv", "ddt", "dbeta", "dA", "ddt_bias", "dinitial_state"});
  const Tensor *dq_ = g.get("dq", qk), *dk_ = g.get("dk", qk), *dv_ = g.get("dv", in.yshape),
               *dt_ = g.get("ddt", gate), *db_ = g.get("dbeta", gate), *dA_ = g.get("dA", H),
               *dbias_ = g.get("ddt_bias", H), *dh_ = g.get("dinitial_state", in.state);
  dense(&dy, "dy", in.io, in.v);
  dense(df, "dfinal_state", at::kFloat, in.v);
  dense(h0, "initial_state", at::kFloat, in.v);
  // strided buffers, or new dense ones
  in.d.dq_stride = dq_ ? token_stride(*dq_, "dq", in.io, in.v) : in.d.ngroups * in.d.dstate;
  in.d.dk_stride = dk_ ? token_stride(*dk_, "dk", in.io, in.v) : in.d.ngroups * in.d.dstate;
  in.d.dv_stride = dv_ ? token_stride(*dv_, "dv", in.io, in.v) : H * in.d.headdim;
  const Tensor dq = dq_ ? *dq_ : output(nullptr, "dq", qk, in.io, in.v);
  const Tensor dk = dk_ ? *dk_ : output(nullptr, "dk", qk, in.io, in.v);
  const Tensor dv = dv_ ? *dv_ : output(nullptr, "dv", in.yshape, in.io, in.v);
  const Tensor ddt = output(dt_, "ddt", gate, at::kFloat, in.v);
  const Tensor dbeta = output(db_, "dbeta", gate, at::kFloat, in.v);
  const Tensor dA = output(dA_, "dA", H, at::kFloat, in.v);
  const Tensor dbias = output(dbias_, "ddt_bias", H, at::kFloat, in.v);
  const Tensor dh = output(dh_, "dinitial_state", in.state, at::kFloat, in.v);
  const Tensor ws = workspace(w_, ssd_delta_scan_backward_workspace_bytes(&in.d), in.v);
  launch(in.v, "ssd_delta_scan_backward", [&](hipStream_t stream) {
    return ssd_delta_scan_backward(&in.d, ptr(in.q), ptr(in.k), ptr(in.v), f32(in.dt), f32(in.bias),
                                   f32(in.A), f32(in.beta), f32(h0), ptr(dy), f32(df), ptr(dq), ptr(dk),
                                   ptr(dv), f32(ddt), f32(dbeta), f32(dA), f32(dbias), f32(dh), ptr(ws),
                                   ws.nbytes(), stream);
  });
  return dict({{"dq", &dq}, {"dk", &dk}, {"dv", &dv}, {"ddt", &ddt}, {"dbeta", &dbeta}, {"dA", &dA},
               {"ddt_bias", &dbias}, {"dinitial_state", &dh}});
}

// the inputs, state, y_t
PyObject* delta_step(PyObject* const* a) {
  const Delta in(a, true);
  const Tensor &state = tensor(a[kDeltaInputs], "state");
  const Tensor* y_ = maybe(a[kDeltaInputs + 1], "y_t");
  shape(&state, "state", in.state);
  shape(y_, "y_t", in.yshape);
  dense(&state, "state", at::kFloat, in.v);
  const Tensor y = output(y_, "y_t", in.yshape, in.io, in.v);
  launch(in.v, "ssd_delta_step", [&](hipStream_t stream) {
    return ssd_delta_step(&in.d, f32(state), ptr(in.q), ptr(in.k), ptr(in.v), f32(in.dt),
                          f32(in.bias), f32(in.A), f32(in.beta), ptr(y), stream);
  });
  return wrap(y);
}

// ---------------------------------------------------------------------------
// the module
// ---------------------------------------------------------------------------
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == N, "expected ", N, " arguments, got ", n);
  TORCH_CHECK(g_error, "connect() comes first");
  return F(args);
  END_HANDLE_TH_ERRORS
}

// SSDError, the current stream of a device, the current device, setting it
PyObject* connect(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  PyObject** const kept[] = {&g_error, &g_stream, &g_current_device, &g_set_device};
  TORCH_CHECK_TYPE(n == 4, "expected 4 arguments, got ", n);
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(args[i]);
    Py_XDECREF(*kept[i]);
    *kept[i] = args[i];
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// t, name
PyObject* row_stride_of(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 2, "expected 2 arguments, got ", n);
  const char* name = PyUnicode_AsUTF8(args[1]);
  if (!name) throw python_error();
  return PyLong_FromLongLong(row_stride(tensor(args[0], name), name));
  END_HANDLE_TH_ERRORS
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"connect", FAST(connect), nullptr},
    {"row_stride", FAST(row_stride_of), nullptr},
    {"add_norm", FAST((entry<add_norm, 7>)), nullptr},
    {"add_norm_q8", FAST((entry<add_norm_q8, 8>)), nullptr},
    {"add_norm_backward", FAST((entry<add_norm_backward, 8>)), nullptr},
    {"dropout_add_norm", FAST((entry<dropout_add_norm, 9>)), nullptr},
    {"dropout_add_norm_backward", FAST((entry<dropout_add_norm_backward, 10>)), nullptr},
    {"gated_norm", FAST((entry<gated_norm, 6>)), nullptr},
    {"gated_norm_q8", FAST((entry<gated_norm_q8, 7>)), nullptr},
    {"gated_norm_backward", FAST((entry<gated_norm_backward, 8>)), nullptr},
    {"quantize_q8", FAST((entry<quantize_q8, 3>)), nullptr},
    {"linear_q8", FAST((entry<linear_q8, 6>)), nullptr},
    {"conv1d_backward", FAST((entry<conv1d_backward, 9>)), nullptr},
    {"delta_scan", FAST((entry<delta_scan, kDeltaInputs + 5>)), nullptr},
    {"delta_scan_backward", FAST((entry<delta_scan_backward, kDeltaInputs + 5>)), nullptr},
    {"delta_step", FAST((entry<delta_step, kDeltaInputs + 2>)), nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ssd_torch",
                      "The operators between two scans, and the gated delta rule, on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__ssd_torch() { return PyModule_Create(&module); }

// Native marshalling of the calls that a decoding loop makes one after the other:
// torch tensors -> the C ABI of fq.h, on the current device's current stream. A call with
// its launch takes 3.5 to 4 us of host time here (0.2 us where nothing is enqueued) and 8
// through ctypes, more than the small kernels themselves.
//
// Every function takes the arguments of its C entry point without the stream and
// with (ws, ws_bytes) as one tensor or None, positionally, and returns the status.
// Tensors must be contiguous device tensors on the current device, of the C type's
// elements (uint16_t: bf16, or 16-bit integers as raw storage); a shape is a tuple
// (E, N, K), weights are StoredW, activation quantizers ActQ or None.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <type_traits>

#include "fq.h"

namespace {

struct Error {};  // a Python exception is set

// What a pointer of fq.h may be given as: a float16 or an int32 of the right size would
// only give wrong numbers.
template <class T>
constexpr const char *kWanted = "";
template <>
constexpr const char *kWanted<uint8_t> = "8-bit";
template <>
constexpr const char *kWanted<uint16_t> = "bfloat16";
template <>
constexpr const char *kWanted<int32_t> = "int32";
template <>
constexpr const char *kWanted<float> = "float32";
template <class T>
bool holds(const at::Tensor &t) {
  const at::ScalarType s = t.scalar_type();
  if (std::is_same<T, uint8_t>::value) return t.element_size() == 1 && s != at::kBool;
  if (std::is_same<T, uint16_t>::value)
    return s == at::kBFloat16 || s == at::kShort || s == at::kUInt16;
  if (std::is_same<T, int32_t>::value) return s == at::kInt || s == at::kUInt32;
  return s == at::kFloat;
}

PyObject *n_fmt, *n_group, *n_codes, *n_scale;

// The arguments of one call, taken from left to right.
class Args {
 public:
  Args(const char *fn, PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, not %zd", fn, want, n);
      throw Error{};
    }
    dev_ = c10::hip::current_device();
  }
  template <class T>
  T *ptr() {
    return tensor<T>(*a_++);
  }
  int32_t i32() {
    const long v = PyLong_AsLong(*a_++);
    if (v == -1 && PyErr_Occurred()) throw Error{};
    if (v != (int32_t)v) {
      PyErr_Format(PyExc_OverflowError, "%ld does not fit an int32", v);
      throw Error{};
    }
    return (int32_t)v;
  }
  float f32() {
    const double v = PyFloat_AsDouble(*a_++);
    if (v == -1.0 && PyErr_Occurred()) throw Error{};
    return (float)v;
  }
  fq_shape shape() {
    PyObject *s = *a_++;
    if (!PyTuple_Check(s) || PyTuple_GET_SIZE(s) != 3) {
      PyErr_SetString(PyExc_TypeError, "a shape is a tuple (E, N, K)");
      throw Error{};
    }
    PyObject *const *keep = a_;
    PyObject *v[3] = {PyTuple_GET_ITEM(s, 0), PyTuple_GET_ITEM(s, 1), PyTuple_GET_ITEM(s, 2)};
    a_ = v;
    fq_shape r;
    r.E = i32();
    r.N = i32();
    r.K = i32();
    a_ = keep;
    return r;
  }
  // a StoredW's fields that the int8 products read
  fq_stored_w stored() {
    PyObject *w = *a_++;
    fq_stored_w r{};
    r.fmt = (int32_t)number(w, n_fmt);
    r.group = (int32_t)number(w, n_group);
    r.codes = field<uint8_t>(w, n_codes);
    r.scale = field<float>(w, n_scale);
    return r;
  }
  // an ActQ or None
  const fq_act_q *actq(fq_act_q &q) {
    PyObject *a = *a_++;
    if (a == Py_None) return nullptr;
    q.fmt = (int32_t)number(a, n_fmt);
    q.scale = field<float>(a, n_scale);
    return &q;
  }
  // a workspace: pointer and size
  void *ws(size_t &bytes) {
    PyObject *o = *a_++;
    void *p = data(o);
    bytes = p ? THPVariable_Unpack(o).nbytes() : 0;
    return p;
  }
  fq_stream stream() { return c10::hip::getCurrentHIPStream(dev_).stream(); }

 private:
  PyObject *const *a_;
  c10::DeviceIndex dev_;

  template <class T>
  T *tensor(PyObject *o) {
    void *p = data(o);
    if (o != Py_None && !holds<T>(THPVariable_Unpack(o))) {
      PyErr_Format(PyExc_ValueError, "a tensor of %s elements is wanted, not of %s", kWanted<T>,
                   c10::toString(THPVariable_Unpack(o).scalar_type()));
      throw Error{};
    }
    return static_cast<T *>(p);
  }
  void *data(PyObject *o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "a tensor or None is wanted, not %s", Py_TYPE(o)->tp_name);
      throw Error{};
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
      PyErr_SetString(PyExc_ValueError, "libfq takes device tensors");
      throw Error{};
    }
    if (t.get_device() != dev_) {
      PyErr_Format(PyExc_ValueError, "tensor on cuda:%d, but the current device is cuda:%d",
                   (int)t.get_device(), (int)dev_);
      throw Error{};
    }
    if (!t.is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "libfq takes contiguous tensors");
      throw Error{};
    }
    return t.data_ptr();
  }
  PyObject *get(PyObject *o, PyObject *name) {
    PyObject *v = PyObject_GetAttr(o, name);
    if (!v) throw Error{};
    return v;
  }
  long number(PyObject *o, PyObject *name) {
    PyObject *v = get(o, name);
    const long r = PyLong_AsLong(v);
    Py_DECREF(v);
    if (r == -1 && PyErr_Occurred()) throw Error{};
    return r;
  }
  template <class T>
  T *field(PyObject *o, PyObject *name) {
    PyObject *v = get(o, name);
    // the object keeps its tensor alive; v is only this look at it
    struct Drop {
      PyObject *p;
      ~Drop() { Py_DECREF(p); }
    } drop{v};
    return tensor<T>(v);
  }
};

// The C call itself without the interpreter lock: a launch may wait for room in the queue,
// and other threads (a host function of the same stream among them) go on meanwhile.
struct Unlocked {
  PyThreadState *t = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(t); }
};

template <class F>
PyObject *guarded(F f) {
  try {
    return PyLong_FromLong((long)f());
  } catch (const Error &) {
    return nullptr;
  } catch (const c10::Error &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define FN(name) PyObject *name(PyObject *, PyObject *const *argv, Py_ssize_t n)

FN(quantize_tokens) {
  return guarded([&] {
    Args a("fq_quantize_tokens", argv, n, 6);
    const auto *x = a.ptr<uint16_t>();
    const int32_t rows = a.i32(), K = a.i32();
    const auto *n_rows = a.ptr<int32_t>();
    auto *codes = a.ptr<uint8_t>();
    auto *scale = a.ptr<float>();
    const fq_stream st = a.stream();
    Unlocked u;
    return fq_quantize_tokens(x, rows, K, n_rows, codes, scale, st);
  });
}

template <class Call>
PyObject *int8_call(const char *fn, Call call, PyObject *const *argv, Py_ssize_t n) {
  return guarded([&] {
    Args a(fn, argv, n, 11);
    const auto *xc = a.ptr<uint8_t>();
    const auto *sx = a.ptr<float>();
    const int32_t x_rows = a.i32();
    const auto *perm = a.ptr<int32_t>();
    const int32_t topk = a.i32(), R = a.i32();
    const auto *seg = a.ptr<int32_t>();
    const fq_shape s = a.shape();
    const fq_stored_w w = a.stored();
    auto *out = a.ptr<uint16_t>();
    size_t bytes;
    void *ws = a.ws(bytes);
    const fq_stream st = a.stream();
    Unlocked u;
    return call(xc, sx, x_rows, perm, topk, R, seg, s, &w, out, ws, bytes, st);
  });
}
FN(grouped_gemm_int8) { return int8_call("fq_grouped_gemm_int8", fq_grouped_gemm_int8, argv, n); }
FN(grouped_gated_int8) { return int8_call("fq_grouped_gated_int8", fq_grouped_gated_int8, argv, n); }

FN(grouped_gated_fwd) {
  return guarded([&] {
    Args a("fq_grouped_gated_fwd", argv, n, 11);
    const auto *x = a.ptr<uint16_t>();
    const int32_t x_rows = a.i32();
    const auto *perm = a.ptr<int32_t>();
    const int32_t topk = a.i32(), R = a.i32();
    const auto *seg = a.ptr<int32_t>();
    const fq_shape s = a.shape();
    const auto *w = a.ptr<uint16_t>();
    fq_act_q q;
    const fq_act_q *aq = a.actq(q);
    auto *out = a.ptr<uint16_t>();
    size_t bytes;
    void *ws = a.ws(bytes);
    const fq_stream st = a.stream();
    Unlocked u;
    return fq_grouped_gated_fwd(x, x_rows, perm, topk, R, seg, s, w, aq, out, ws, bytes, st);
  });
}

FN(grouped_gated_bwd) {
  return guarded([&] {
    Args a("fq_grouped_gated_bwd", argv, n, 13);
    const auto *daq = a.ptr<uint16_t>();
    const auto *x = a.ptr<uint16_t>();
    const int32_t x_rows = a.i32();
    const auto *perm = a.ptr<int32_t>();
    const int32_t topk = a.i32(), R = a.i32();
    const auto *seg = a.ptr<int32_t>();
    const fq_shape s = a.shape();
    const auto *w = a.ptr<uint16_t>();
    fq_act_q q;
    const fq_act_q *aq = a.actq(q);
    auto *dh = a.ptr<uint16_t>();
    auto *aqo = a.ptr<uint16_t>();
    size_t bytes;
    void *ws = a.ws(bytes);
    const fq_stream st = a.stream();
    Unlocked u;
    return fq_grouped_gated_bwd(daq, x, x_rows, perm, topk, R, seg, s, w, aq, dh, aqo, ws, bytes, st);
  });
}

FN(norm_residual_fwd) {
  return guarded([&] {
    Args a("fq_norm_residual_fwd", argv, n, 13);
    const auto *x = a.ptr<uint16_t>();
    const auto *b = a.ptr<uint16_t>();
    const auto *gate = a.ptr<float>();
    const float alpha = a.f32();
    const auto *w_post = a.ptr<uint16_t>();
    const auto *w_pre = a.ptr<uint16_t>();
    const float eps = a.f32();
    const int32_t T = a.i32(), H = a.i32();
    auto *y = a.ptr<uint16_t>();
    auto *nn = a.ptr<uint16_t>();
    auto *codes = a.ptr<uint8_t>();
    auto *scale = a.ptr<float>();
    const fq_stream st = a.stream();
    Unlocked u;
    return fq_norm_residual_fwd(x, b, gate, alpha, w_post, w_pre, eps, T, H, y, nn, codes, scale, st);
  });
}

FN(norm_residual_bwd) {
  return guarded([&] {
    Args a("fq_norm_residual_bwd", argv, n, 17);
    const auto *dy = a.ptr<uint16_t>();
    const auto *dn = a.ptr<uint16_t>();
    const auto *y = a.ptr<uint16_t>();
    const auto *b = a.ptr<uint16_t>();
    const auto *gate = a.ptr<float>();
    const float alpha = a.f32();
    const auto *w_post = a.ptr<uint16_t>();
    const auto *w_pre = a.ptr<uint16_t>();
    const float eps = a.f32();
    const int32_t T = a.i32(), H = a.i32();
    auto *dx = a.ptr<uint16_t>();
    auto *db = a.ptr<uint16_t>();
    auto *dgate = a.ptr<float>();
    auto *dw_post = a.ptr<float>();
    auto *dw_pre = a.ptr<float>();
    size_t bytes;
    void *ws = a.ws(bytes);
    const fq_stream st = a.stream();
    Unlocked u;
    return fq_norm_residual_bwd(dy, dn, y, b, gate, alpha, w_post, w_pre, eps, T, H, dx, db, dgate,
                                dw_post, dw_pre, ws, bytes, st);
  });
}

#define ENTRY(name) {"fq_" #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(quantize_tokens),   ENTRY(grouped_gemm_int8), ENTRY(grouped_gated_int8),
                         ENTRY(grouped_gated_fwd), ENTRY(grouped_gated_bwd), ENTRY(norm_residual_fwd),
                         ENTRY(norm_residual_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fqbind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fqbind(void) {
  n_fmt = PyUnicode_InternFromString("fmt");
  n_group = PyUnicode_InternFromString("group");
  n_codes = PyUnicode_InternFromString("codes");
  n_scale = PyUnicode_InternFromString("scale");
  if (!n_fmt || !n_group || !n_codes || !n_scale) return nullptr;
  return PyModule_Create(&module);
}

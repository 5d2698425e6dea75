// Python module _marshal: checks the tensors of the calls around the caches and hands them to libdsa.
//
// These calls take tensors whose types, shapes and strides the C ABI cannot see, and a decode step makes
// several of them.  Checked and passed from Python a call took 8 to 11 us, of which 3 are the launch;
// here the checks are a few hundred nanoseconds.  Python's lock is released for the call itself.  Every
// function takes its arguments by position and returns the library's status, or raises ValueError for a
// tensor that it cannot pass on: of another type, shape or layout, or on another device than the current
// one (whose stream the work goes to).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/dsa.h"

#ifndef DSA_MARSHAL_TARGET
#error "build.py says which torch and Python this module is compiled for"
#endif
// Read from the file by build.py and the package, which do not load a module made for another torch or Python.
extern "C" __attribute__((used, visibility("default"))) const char dsa_marshal_target[] = DSA_MARSHAL_TARGET;

namespace {

// A message for ValueError.
struct Refusal : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// A Python error that is already set.
struct Raised {};

// The positional arguments of one call.
class Args {
 public:
  Args(const char* where, PyObject* const* v, Py_ssize_t n, Py_ssize_t want) : where_(where), v_(v) {
    if (n != want) throw Refusal(std::string(where) + ": takes " + std::to_string(want) + " arguments, got " + std::to_string(n));
  }
  const char* where() const { return where_; }
  int64_t integer(int i) const {
    const int64_t x = PyLong_AsLongLong(v_[i]);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    return x;
  }
  // An int32_t argument; what does not fit is refused rather than cut.
  int32_t int32(int i, const char* name) const {
    const int64_t x = integer(i);
    if (x < INT32_MIN || x > INT32_MAX) throw Refusal(std::string(where_) + ": " + name + " does not fit 32 bits");
    return static_cast<int32_t>(x);
  }
  double real(int i) const {
    const double x = PyFloat_AsDouble(v_[i]);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return x;
  }
  bool truth(int i) const {
    const int x = PyObject_IsTrue(v_[i]);
    if (x < 0) throw Raised{};
    return x != 0;
  }
  // A tensor, or nullptr for None.
  const at::Tensor* tensor(int i, const char* name) const {
    if (v_[i] == Py_None) return nullptr;
    if (!THPVariable_Check(v_[i])) throw Refusal(std::string(where_) + ": " + name + " must be a tensor");
    return &THPVariable_Unpack(v_[i]);
  }
  const at::Tensor& required(int i, const char* name) const {
    const at::Tensor* t = tensor(i, name);
    if (t == nullptr) throw Refusal(std::string(where_) + ": " + name + " must be a tensor");
    return *t;
  }
  // The address of a dsa_kv_desc, or nullptr for None.
  const dsa_kv_desc* desc(int i) const {
    return v_[i] == Py_None ? nullptr : reinterpret_cast<const dsa_kv_desc*>(integer(i));
  }
  // The stream's handle: an address, or for None the current stream of the call's device.
  void* stream(int i, int dev) const {
    if (v_[i] != Py_None) return reinterpret_cast<void*>(integer(i));
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }

 private:
  const char* where_;
  PyObject* const* v_;
};

std::string shape_text(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

[[noreturn]] void refuse(const Args& a, const char* name, const at::Tensor& t, at::ScalarType type, c10::IntArrayRef shape,
                         const char* layout) {
  throw Refusal(std::string(a.where()) + ": " + name + " must be a " + c10::toString(type) + " tensor of shape " +
                shape_text(shape) + ", " + layout + ", on the current device, got " + c10::toString(t.scalar_type()) + " " +
                shape_text(t.sizes()) + " strides " + shape_text(t.strides()) + " on " + t.device().str());
}

// The current device, for a call whose first tensor is t: all of a call's tensors are on it.
int device_of(const Args& a, const at::Tensor& t) {
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    throw Refusal(std::string(a.where()) + ": tensors must be on the current CUDA device, got " + t.device().str());
  return static_cast<int>(t.get_device());
}

bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided; }

// The address of a contiguous tensor of this type and shape (nullptr for None).
void* dense(const Args& a, int i, const char* name, at::ScalarType type, c10::IntArrayRef shape, int dev) {
  const at::Tensor* t = a.tensor(i, name);
  if (t == nullptr) return nullptr;
  if (!on(*t, dev) || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous())
    refuse(a, name, *t, type, shape, "contiguous");
  return t->data_ptr();
}

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};

// Address and row stride of a tensor of this type and shape whose last dimension is dense.
Rows strided(const Args& a, int i, const char* name, at::ScalarType type, c10::IntArrayRef shape, int dev) {
  const at::Tensor* t = a.tensor(i, name);
  if (t == nullptr) return {};
  if (!on(*t, dev) || t->scalar_type() != type || t->sizes() != shape || (t->stride(-1) != 1 && shape.back() > 1))
    refuse(a, name, *t, type, shape, "dense in its last dimension");
  return {t->data_ptr(), shape[0] > 1 ? t->stride(0) : std::max(t->stride(0), shape.back())};
}

// The library's code of a floating type.
int32_t type_code(const Args& a, const at::Tensor& t, int64_t dims) {
  if (t.dim() == dims) {
    if (t.scalar_type() == at::kBFloat16) return DSA_BF16;
    if (t.scalar_type() == at::kHalf) return DSA_F16;
    if (t.scalar_type() == at::kFloat) return DSA_F32;
  }
  throw Refusal(std::string(a.where()) + ": expected a bf16, fp16 or fp32 tensor of " + std::to_string(dims) + " dimensions, got " +
                c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
}

int32_t columns(const Args& a, int64_t n) {
  if (n > INT32_MAX) throw Refusal(std::string(a.where()) + ": a dimension does not fit 32 bits");
  return static_cast<int32_t>(n);
}

// Calls the library without Python's lock, which the launch does not need: with a full launch queue it waits, and
// what it waits for may itself need a Python thread.  The arguments are read before.
template <typename... P, typename... A>
dsa_status unlocked(dsa_status (*f)(P...), A... a) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f(a...);
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return PyLong_FromLong(f());
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {  // a refusal, or an error of torch
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

// x, weight, eps, y, residual, residual_out, codes, scale, rstd, stream
PyObject* rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    const Args a("dsa_rmsnorm", v, n, 10);
    const at::Tensor& x = a.required(0, "x");
    const int dev = device_of(a, x);
    const int32_t code = type_code(a, x, 2);
    const at::ScalarType type = x.scalar_type();
    const auto shape = x.sizes();
    const int64_t rows = shape[0], cols = shape[1];
    const Rows xr = strided(a, 0, "x", type, shape, dev), y = strided(a, 3, "y", type, shape, dev);
    const Rows res = strided(a, 4, "residual", type, shape, dev), out = strided(a, 5, "residual_out", type, shape, dev);
    const at::Tensor* scale = a.tensor(7, "scale");
    const bool grouped = scale != nullptr && scale->dim() == 2;
    const int64_t groups = (cols + DSA_QUANT_GROUP - 1) / DSA_QUANT_GROUP;
    float* sp = static_cast<float*>(grouped ? dense(a, 7, "scale", at::kFloat, {rows, groups}, dev)
                                            : dense(a, 7, "scale", at::kFloat, {rows}, dev));
    return unlocked(dsa_rmsnorm, xr.p, xr.ld, res.p, res.ld, dense(a, 1, "weight", type, {cols}, dev), rows, columns(a, cols), code,
                    static_cast<float>(a.real(2)), y.p, y.ld, out.p, out.ld,
                    static_cast<uint8_t*>(dense(a, 6, "codes", at::kByte, shape, dev)), sp, grouped ? DSA_QUANT_GROUP : 0,
                    static_cast<float*>(dense(a, 8, "rstd", at::kFloat, {rows}, dev)), a.stream(9, dev));
  });
}

// A workspace tensor: its address and size in bytes (None: none).
void* workspace_of(const Args& a, int i, int dev, size_t* bytes) {
  const at::Tensor* t = a.tensor(i, "workspace");
  *bytes = t == nullptr ? 0 : static_cast<size_t>(t->nbytes());
  return t == nullptr ? nullptr : dense(a, i, "workspace", t->scalar_type(), t->sizes(), dev);
}

// dy, h, weight, rstd, dh, dw, workspace, dresidual, stream
PyObject* rmsnorm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    const Args a("dsa_rmsnorm_backward", v, n, 9);
    const at::Tensor& dy = a.required(0, "dy");
    const int dev = device_of(a, dy);
    const int32_t code = type_code(a, dy, 2);
    const at::ScalarType type = dy.scalar_type();
    const auto shape = dy.sizes();
    const int64_t rows = shape[0], cols = shape[1];
    const Rows g = strided(a, 0, "dy", type, shape, dev), h = strided(a, 1, "h", type, shape, dev);
    const Rows res = strided(a, 7, "dresidual", type, shape, dev), dh = strided(a, 4, "dh", type, shape, dev);
    size_t bytes;
    void* ws = workspace_of(a, 6, dev, &bytes);
    return unlocked(dsa_rmsnorm_backward, g.p, g.ld, h.p, h.ld, dense(a, 2, "weight", type, {cols}, dev),
                    static_cast<float*>(dense(a, 3, "rstd", at::kFloat, {rows}, dev)), res.p, res.ld, rows,
                    columns(a, cols), code, dh.p, dh.ld, static_cast<float*>(dense(a, 5, "dw", at::kFloat, {cols}, dev)),
                    ws, bytes, a.stream(8, dev));
  });
}

// x, positions, freqs, out, rot_offset, rot_dim, layout, mscale, transpose, stream
PyObject* rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    const Args a("dsa_rope", v, n, 10);
    const at::Tensor& x = a.required(0, "x");
    const int dev = device_of(a, x);
    const int32_t code = type_code(a, x, 3);
    const auto shape = x.sizes();
    const Rows xr = strided(a, 0, "x", x.scalar_type(), shape, dev);
    const at::Tensor& out = a.required(3, "out");
    const Rows o = strided(a, 3, "out", x.scalar_type(), shape, dev);
    const int32_t rot = a.int32(5, "rot_dim");
    return unlocked(dsa_rope, xr.p, xr.ld, x.stride(1), o.p, o.ld, out.stride(1), shape[0], columns(a, shape[1]), columns(a, shape[2]),
                    a.int32(4, "rot_offset"), rot, a.int32(6, "layout"), code,
                    static_cast<int32_t*>(dense(a, 1, "positions", at::kInt, {shape[0]}, dev)),
                    static_cast<double*>(dense(a, 2, "freqs", at::kDouble, {std::max<int64_t>(rot / 2, 0)}, dev)),
                    static_cast<float>(a.real(7)), a.truth(8), a.stream(9, dev));
  });
}

// kv, kv_weight, eps, key, seq, positions, freqs, latent, keys, batch, layout, key_layout, key_rot_offset, mscale, stream
PyObject* cache_append(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    const Args a("dsa_cache_append", v, n, 15);
    const at::Tensor& pos = a.required(5, "positions");
    const int dev = device_of(a, pos);
    if (pos.dim() != 1) throw Refusal("dsa_cache_append: positions must have one dimension");
    const int64_t rows = pos.size(0);
    const at::Tensor* key = a.tensor(3, "key");
    if (key != nullptr && key->dim() != 2) throw Refusal("dsa_cache_append: key must have two dimensions");
    const int64_t d_I = key != nullptr ? key->size(1) : 128;
    const Rows kv = strided(a, 0, "kv", at::kBFloat16, {rows, 576}, dev);
    const Rows k = strided(a, 3, "key", at::kBFloat16, {rows, d_I}, dev);
    return unlocked(dsa_cache_append, kv.p, kv.ld, dense(a, 1, "kv_weight", at::kBFloat16, {512}, dev), static_cast<float>(a.real(2)), k.p, k.ld,
                    columns(a, d_I), static_cast<int32_t*>(dense(a, 4, "seq", at::kInt, {rows}, dev)),
                    static_cast<int32_t*>(dense(a, 5, "positions", at::kInt, {rows}, dev)), rows, a.int32(9, "batch"),
                    static_cast<double*>(dense(a, 6, "freqs", at::kDouble, {32}, dev)), static_cast<float>(a.real(13)),
                    a.int32(10, "layout"), a.int32(11, "key_layout"), a.int32(12, "key_rot_offset"), a.desc(7), a.desc(8),
                    a.stream(14, dev));
  });
}

struct Window {
  const at::Tensor& q;
  int dev;
  int32_t B, H;
  void *qp, *out;
  float* lse;
};

// Arguments q (0), latent (1), B (2), H (3), ..., out (7), lse (8) of either window call.
Window window_of(const Args& a) {
  const at::Tensor& q = a.required(0, "q");
  const int dev = device_of(a, q);
  const int32_t B = a.int32(2, "B"), H = a.int32(3, "H");
  if (q.dim() != 3) throw Refusal(std::string(a.where()) + ": q must have three dimensions");
  const int64_t rows = q.size(0);
  a.required(7, "out");
  return {q, dev, B, H, dense(a, 0, "q", at::kBFloat16, {rows, H, 576}, dev), dense(a, 7, "out", at::kBFloat16, {rows, H, 512}, dev),
          static_cast<float*>(dense(a, 8, "lse", at::kFloat, {rows, H}, dev))};
}

// q, latent, B, H, window, sinks, sm_scale, out, lse, stream
PyObject* window_prefill(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    const Args a("dsa_window_mla_prefill", v, n, 10);
    const Window w = window_of(a);
    const dsa_kv_desc* latent = a.desc(1);
    if (latent != nullptr && latent->kind == DSA_KV_CONTIGUOUS && w.q.size(0) != latent->total_tokens)
      throw Refusal("dsa_window_mla_prefill: q has " + std::to_string(w.q.size(0)) + " rows, latent " +
                    std::to_string(latent->total_tokens) + " tokens");
    return unlocked(dsa_window_mla_prefill, w.qp, latent, w.B, w.H, a.int32(4, "window"), a.int32(5, "sinks"), static_cast<float>(a.real(6)),
                    w.out, w.lse, a.stream(9, w.dev));
  });
}

// q, latent, B, H, window, sinks, sm_scale, out, lse, workspace, stream
PyObject* window_decode(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    const Args a("dsa_window_mla_decode", v, n, 11);
    const Window w = window_of(a);
    if (w.q.size(0) != w.B)
      throw Refusal("dsa_window_mla_decode: q has " + std::to_string(w.q.size(0)) + " rows, B = " + std::to_string(w.B));
    size_t bytes;
    void* ws = workspace_of(a, 9, w.dev, &bytes);
    return unlocked(dsa_window_mla_decode, w.qp, a.desc(1), w.B, w.H, a.int32(4, "window"), a.int32(5, "sinks"), static_cast<float>(a.real(6)),
                    w.out, w.lse, ws, bytes, a.stream(10, w.dev));
  });
}

#define DSA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DSA_METHOD(rmsnorm),        DSA_METHOD(rmsnorm_backward), DSA_METHOD(rope),
                         DSA_METHOD(cache_append),   DSA_METHOD(window_prefill),   DSA_METHOD(window_decode),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Checked calls of libdsa on tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }

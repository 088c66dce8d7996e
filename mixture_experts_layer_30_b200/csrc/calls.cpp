// Short path of the binding's calls that take a few microseconds on the device: the
// arguments are checked and handed to the C ABI in one native call (about 1 us where the
// same checks in Python take 5).  A function returns the C ABI's status, or -1 when it
// does not understand an argument or a check fails: nothing has been launched then, and
// the binding's own path, which checks the same things, names what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>

#include "moe.h"

namespace {

struct Refused {};  // this path does not take the call

// Arguments of one call, for tensors on the current device.
struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  int at = 0;
  c10::DeviceIndex dev;

  Args(PyObject* const* v, Py_ssize_t n, Py_ssize_t expected) : v(v), n(n) {
    if (n != expected) throw Refused();
    dev = c10::cuda::current_device();
  }
  PyObject* next() { return v[at++]; }

  const at::Tensor& tensor(PyObject* o, at::ScalarType type) const {
    if (!THPVariable_Check(o)) throw Refused();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || !t.is_contiguous())
      throw Refused();
    return t;
  }
  // Device pointer of the next argument, a tensor of numel elements.
  void* ptr(at::ScalarType type, int64_t numel) {
    const at::Tensor& t = tensor(next(), type);
    if (t.numel() != numel) throw Refused();
    return t.data_ptr();
  }
  // Whether the next argument is None, which is passed over then.
  bool none() {
    if (v[at] != Py_None) return false;
    ++at;
    return true;
  }
  void* opt(at::ScalarType type, int64_t numel) { return none() ? nullptr : ptr(type, numel); }
  // Of a tensor of at least `least` elements.
  void* holding(at::ScalarType type, int64_t least) {
    const at::Tensor& t = tensor(next(), type);
    if (t.numel() < least) throw Refused();
    return t.data_ptr();
  }
  // Of a tensor with the shape of x.
  void* like(const at::Tensor& x, bool none_ok) {
    PyObject* o = next();
    if (o == Py_None && none_ok) return nullptr;
    const at::Tensor& t = tensor(o, x.scalar_type());
    if (!t.sizes().equals(x.sizes())) throw Refused();
    return t.data_ptr();
  }
  // The next argument as rows [T, d] of a layer dtype.
  const at::Tensor& rows(int32_t* code) {
    PyObject* o = next();
    if (!THPVariable_Check(o)) throw Refused();
    const auto type = THPVariable_Unpack(o).scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) throw Refused();
    *code = type == at::kBFloat16 ? MOE_BF16 : MOE_F32;
    const at::Tensor& t = tensor(o, type);
    if (t.dim() != 2 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) throw Refused();
    return t;
  }
  double number() {
    const double d = PyFloat_AsDouble(next());
    if (d == -1.0 && PyErr_Occurred()) throw Refused();
    return d;
  }
  int32_t integer() {
    const long d = PyLong_AsLong(next());
    if (PyErr_Occurred() || d < INT32_MIN || d > INT32_MAX) throw Refused();
    return (int32_t)d;
  }
  // A copy of the ctypes structure that the next argument is.
  moe_shape shape() {
    Py_buffer b;
    moe_shape s;
    if (PyObject_GetBuffer(next(), &b, PyBUF_SIMPLE) != 0) throw Refused();
    const bool ok = b.len == (Py_ssize_t)sizeof(s);
    if (ok) std::memcpy(&s, b.buf, sizeof(s));
    PyBuffer_Release(&b);
    if (!ok) throw Refused();
    return s;
  }
  // The workspace: a tensor of bytes.
  void* workspace(size_t* bytes) {
    const at::Tensor& t = tensor(next(), at::kByte);
    *bytes = (size_t)t.numel();
    return t.data_ptr();
  }
  // The last argument: None for torch's current stream, or a torch.cuda.Stream.
  void* stream() {
    PyObject* o = next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Refused();
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Refused();
    return p;
  }
};

struct W4 {
  const void *q, *s;
};
// The next argument as a (codes, scales) pair of n matrices [rows, cols].
W4 w4(Args& a, int64_t n, int64_t rows, int64_t cols, int32_t group) {
  PyObject* o = a.next();
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) throw Refused();
  if (group != 32 && group != 64 && group != 128) throw Refused();
  const int64_t blocks = n * ((rows + 15) / 16) * ((cols + 127) / 128);
  const at::Tensor& q = a.tensor(PyTuple_GET_ITEM(o, 0), at::kByte);
  const at::Tensor& s = a.tensor(PyTuple_GET_ITEM(o, 1), at::kBFloat16);
  if (q.numel() != blocks * 1024 || s.numel() != blocks * 2048 / group) throw Refused();
  return {q.data_ptr(), s.data_ptr()};
}

// Routed rows T * K of a shape whose sizes fit 64 bits when multiplied by a row's length.
int64_t routed_rows(const moe_shape& s) {
  if (s.T < 0 || s.K < 0 || s.N < 0 || s.Z < 0 || s.d < 0 || s.I < 0) throw Refused();
  const int64_t rows = (int64_t)s.T * s.K;
  if (rows > INT32_MAX) throw Refused();
  return rows;
}

at::ScalarType layer_type(const moe_shape& s) {
  return s.dtype == MOE_BF16 ? at::kBFloat16 : at::kFloat;
}

// Runs `body`, which checks its arguments and returns the launch as a function.
template <typename Body>
PyObject* run(Body body) {
  try {
    auto launch = body();
    long status;
    Py_BEGIN_ALLOW_THREADS
    status = (long)launch();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
  } catch (...) {
    PyErr_Clear();
    return PyLong_FromLong(-1);
  }
}

PyObject* rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run([&] {
    Args a(v, n, 10);
    int32_t code;
    const at::Tensor& x = a.rows(&code);
    const int32_t T = (int32_t)x.size(0), d = (int32_t)x.size(1);
    void* w = a.ptr(x.scalar_type(), d);
    const float eps = (float)a.number();
    void* y = a.like(x, true);
    void* res = a.like(x, true);
    void* sum = a.like(x, true);
    void* inv = a.opt(at::kFloat, T);
    void* q = a.opt(at::kByte, (int64_t)T * d);
    void* sf = a.opt(at::kByte, (int64_t)T * (d / 32));
    void* st = a.stream();
    const void* xp = x.data_ptr();
    return [=] { return moe_rmsnorm(T, d, code, xp, res, w, eps, sum, y, (float*)inv, q, sf, st); };
  });
}

PyObject* rmsnorm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run([&] {
    Args a(v, n, 9);
    int32_t code;
    size_t bytes;
    const at::Tensor& s = a.rows(&code);
    const int32_t T = (int32_t)s.size(0), d = (int32_t)s.size(1);
    void* w = a.ptr(s.scalar_type(), d);
    void* inv = a.ptr(at::kFloat, T);
    void* dy = a.like(s, false);
    void* dx = a.like(s, false);
    void* dw = a.ptr(s.scalar_type(), d);
    void* ws = a.workspace(&bytes);
    void* dsum = a.like(s, true);
    void* st = a.stream();
    const void* sp = s.data_ptr();
    return [=] {
      return moe_rmsnorm_backward(T, d, code, sp, w, (const float*)inv, dy, dsum, dx, dw, ws, bytes,
                                  st);
    };
  });
}

PyObject* permute_mxfp8_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run([&] {
    Args a(v, n, 12);
    size_t bytes;
    const moe_shape s = a.shape();
    const int64_t rows = routed_rows(s), codes = (int64_t)s.T * s.d;
    void* q = a.holding(at::kByte, codes);
    void* sf = a.holding(at::kByte, codes / 32);
    auto idx = (const int32_t*)a.holding(at::kInt, rows);
    auto counts = (const int32_t*)(a.none() ? nullptr : a.holding(at::kInt, (int64_t)s.N + s.Z));
    auto offsets = (int32_t*)a.holding(at::kInt, (int64_t)s.N + 1);
    auto row_token = (int32_t*)a.holding(at::kInt, rows);
    auto slot_pos = (int32_t*)a.holding(at::kInt, rows);
    void* oq = a.holding(at::kByte, rows * s.d);
    void* osf = a.holding(at::kByte, rows * s.d / 32);
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return [=] {
      return moe_permute_mxfp8_rows(&s, q, sf, idx, counts, offsets, row_token, slot_pos, oq, osf,
                                    ws, bytes, st);
    };
  });
}

PyObject* expert_gate_up_w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run([&] {
    Args a(v, n, 10);
    size_t bytes;
    const moe_shape s = a.shape();
    const int32_t group = a.integer();
    const int64_t rows = routed_rows(s);
    const bool in_place = v[3] == Py_None;  // x is x_perm
    void* x = a.holding(layer_type(s), (in_place ? rows : s.T) * s.d);
    const int32_t* row_token = nullptr;
    int32_t n_rows = (int32_t)rows;
    if (!a.none()) {
      const at::Tensor& t = a.tensor(a.next(), at::kInt);
      row_token = (const int32_t*)t.data_ptr();
      n_rows = (int32_t)std::min(rows, t.numel());
    }
    const W4 w1 = w4(a, s.N, s.I, s.d, group), w3 = w4(a, s.N, s.I, s.d, group);
    auto offsets = (const int32_t*)a.holding(at::kInt, (int64_t)s.N + 1);
    void* h = a.holding(layer_type(s), rows * s.I);
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return [=] {
      return moe_expert_gate_up_w4_rows(&s, group, n_rows, x, row_token, w1.q, w1.s, w3.q, w3.s,
                                        offsets, h, ws, bytes, st);
    };
  });
}

PyObject* expert_down_w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run([&] {
    Args a(v, n, 8);
    size_t bytes;
    const moe_shape s = a.shape();
    const int32_t group = a.integer();
    const int64_t rows = routed_rows(s);
    void* h = a.holding(layer_type(s), rows * s.I);
    const W4 w2 = w4(a, s.N, s.d, s.I, group);
    auto offsets = (const int32_t*)a.holding(at::kInt, (int64_t)s.N + 1);
    void* y = a.holding(layer_type(s), rows * s.d);
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return [=] { return moe_expert_down_w4(&s, group, h, w2.q, w2.s, offsets, y, ws, bytes, st); };
  });
}

// (number of tensors, table, max_norm or None for the norm alone, norm, workspace, stream)
PyObject* clip_gradients(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return run([&] {
    Args a(v, n, 6);
    size_t bytes;
    const int32_t count = a.integer();
    Py_buffer b;
    if (PyObject_GetBuffer(a.next(), &b, PyBUF_SIMPLE) != 0) throw Refused();
    // the caller's arguments keep the table alive through the call
    auto table = static_cast<const moe_grad*>(b.buf);
    const bool fits = count >= 0 && b.len >= (Py_ssize_t)(sizeof(moe_grad) * (size_t)count);
    PyBuffer_Release(&b);
    if (!fits) throw Refused();
    const bool clip = a.v[a.at] != Py_None;
    float most = 0.f;
    if (clip) most = (float)a.number();
    else ++a.at;
    auto norm = (float*)a.ptr(at::kFloat, 1);
    void* ws = a.workspace(&bytes);
    void* st = a.stream();
    return [=] {
      const moe_status s = moe_grad_norm(count, table, norm, ws, bytes, st);
      return s != MOE_OK || !clip ? s : moe_grad_clip(count, table, most, norm, st);
    };
  });
}

#define MOE_CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {MOE_CALL(rmsnorm),
                          MOE_CALL(rmsnorm_backward),
                          MOE_CALL(permute_mxfp8_rows),
                          MOE_CALL(expert_gate_up_w4),
                          MOE_CALL(expert_down_w4),
                          MOE_CALL(clip_gradients),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", "Short path of the binding's small calls.",
                       -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }

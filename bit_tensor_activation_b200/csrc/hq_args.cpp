// hq_args.cpp -- the binding's calls as a Python module: the arguments' checks and the call of libhq.so.
//
// A kernel of the library for a few tokens runs for some microseconds, and asking ten tensors for their
// type, sizes, strides, device and address from Python took as long again.  Here the same questions take
// a twentieth of a microsecond each.  Nothing is raised for an argument that does not fit: the call then
// returns None with nothing enqueued, and the binding finds out in Python what to say (or that it fits
// after all: a tensor of a kind that is not looked for here).  Otherwise a call returns the library's status.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstring>

#include "hq.h"

namespace {

using Sizes = std::initializer_list<int64_t>;
using Mask = unsigned long long;

constexpr Mask bit(at::ScalarType t) { return 1ull << static_cast<int>(t); }
constexpr Mask kBf16 = bit(at::kBFloat16) | bit(at::kShort) | bit(at::kUInt16);
constexpr Mask kF32 = bit(at::kFloat), kI32 = bit(at::kInt), kU8 = bit(at::kByte), kI8 = bit(at::kChar);
constexpr Mask kCodes = bit(at::kInt) | bit(at::kUInt32);

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool fits(const at::Tensor& t, int64_t dev, Mask mask, const int64_t* shape, size_t dims) {
  if (!t.is_cuda() || !((mask >> static_cast<int>(t.scalar_type())) & 1) || (dev >= 0 && t.get_device() != dev)) return false;
  const auto sizes = t.sizes();
  if (sizes.size() != dims) return false;
  for (size_t i = 0; i < dims; ++i)
    if (sizes[i] != shape[i]) return false;
  return true;
}

// One call's arguments, looked at in turn; `ok` falls with the first that does not fit.
struct Args {
  PyObject* const* at;
  int64_t dev = -1;
  bool ok = true;

  // the first tensor, whose device is the call's
  const at::Tensor* first(int i, int64_t dims) {
    const at::Tensor* t = tensor(at[i]);
    if (!t || !t->is_cuda() || (dims && t->dim() != dims)) {
      ok = false;
      return nullptr;
    }
    dev = t->get_device();
    return t;
  }
  void* dense(int i, Mask mask, const int64_t* shape, size_t dims, bool optional = false) {
    if (optional && at[i] == Py_None) return nullptr;
    const at::Tensor* t = ok ? tensor(at[i]) : nullptr;
    if (!t || !fits(*t, dev, mask, shape, dims) || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->numel() ? t->data_ptr() : nullptr;
  }
  void* dense(int i, Mask mask, Sizes shape, bool optional = false) {
    return dense(i, mask, shape.begin(), shape.size(), optional);
  }
  // rows that are dense and one pitch apart; of a tensor of at most one row, the width rounded up
  void* pitched(int i, Mask mask, const int64_t* shape, size_t dims, int64_t multiple, int* ld) {
    const at::Tensor* t = ok ? tensor(at[i]) : nullptr;
    if (!t || !fits(*t, dev, mask, shape, dims) || dims == 0) {
      ok = false;
      return nullptr;
    }
    const int64_t n = shape[dims - 1];
    int64_t pitch = -1, rows = 1;
    if (t->numel()) {
      const auto st = t->strides();
      if (st[dims - 1] != 1 && n > 1) ok = false;
      for (size_t d = dims - 1; d-- > 0;) {
        if (shape[d] <= 1) continue;
        if (pitch < 0) pitch = st[d];
        else if (st[d] != rows * pitch) ok = false;
        rows *= shape[d];
      }
    }
    if (pitch < 0) pitch = (n + multiple - 1) / multiple * multiple;
    if (pitch > INT_MAX) ok = false;
    *ld = static_cast<int>(pitch);
    return t->numel() ? t->data_ptr() : nullptr;
  }
  void* pitched(int i, Mask mask, Sizes shape, int64_t multiple, int* ld) {
    return pitched(i, mask, shape.begin(), shape.size(), multiple, ld);
  }
  int size(int64_t n) {
    if (n > INT_MAX) ok = false;
    return static_cast<int>(n);
  }
  bool f32(int i) {
    const at::Tensor* t = tensor(at[i]);
    return t && t->scalar_type() == at::kFloat;
  }
  // the stream given as a number, or the device's current one
  void* stream(int i) {
    if (!ok) return nullptr;
    if (at[i] == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void* s = PyLong_Check(at[i]) ? PyLong_AsVoidPtr(at[i]) : nullptr;
    if (!PyLong_Check(at[i]) || PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return s;
  }
  float number(int i) {
    const double v = PyFloat_AsDouble(at[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
  int integer(int i) {
    const long v = PyLong_AsLong(at[i]);
    if (PyErr_Occurred() || v < INT_MIN || v > INT_MAX) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<int>(v);
  }
};

// The library's call on the arguments' device.  Python's lock is not held meanwhile (a tenth of a microsecond):
// a launch waits where the stream's queue is full, and what it waits for may be a thread that needs the lock.
// `call` touches no Python object.
template <typename Call>
PyObject* run(Args& a, Call call) {
  if (!a.ok) Py_RETURN_NONE;
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(a.dev)));
  hq_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// A method as Python calls it.  A tensor without storage or with symbolic sizes throws when it is asked for
// them: such a one does not fit.
template <PyObject* (*kMethod)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* caught(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return kMethod(self, args, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// quantize_tokens(x, q, scale, stream)
PyObject* quantize_tokens(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args};
  const at::Tensor* x = n == 4 ? a.first(0, 0) : nullptr;
  if (!x || x->dim() < 1) Py_RETURN_NONE;
  const auto shape = x->sizes();
  const size_t dims = shape.size();
  int64_t rows = 1;
  for (size_t i = 0; i + 1 < dims; ++i) rows *= shape[i];
  int ldx, ldq;
  const auto* px = static_cast<const uint16_t*>(a.pitched(0, kBf16, shape.data(), dims, 8, &ldx));
  auto* pq = static_cast<int8_t*>(a.pitched(1, kI8, shape.data(), dims, 16, &ldq));
  auto* ps = static_cast<float*>(a.dense(2, kF32, shape.data(), dims - 1));
  const int K = a.size(shape[dims - 1]);
  void* st = a.stream(3);
  return run(a, [&] { return hq_quantize_tokens(px, ldx, rows, K, pq, ldq, ps, st); });
}

// int8_matmul(a, a_scale, w, w_scale, out, bias, stream)
PyObject* int8_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args};
  const at::Tensor* x = n == 7 ? a.first(0, 3) : nullptr;
  const at::Tensor* w = x ? tensor(args[2]) : nullptr;
  if (!w || w->dim() != 3) Py_RETURN_NONE;
  const int64_t P = x->size(0), T = x->size(1), K = x->size(2), H = w->size(1);
  int lda, ldw, ldo;
  const auto* pa = static_cast<const int8_t*>(a.pitched(0, kI8, {P, T, K}, 16, &lda));
  const auto* ps = static_cast<const float*>(a.dense(1, kF32, {P, T}));
  const auto* pw = static_cast<const int8_t*>(a.pitched(2, kI8, {P, H, K}, 16, &ldw));
  const auto* pws = static_cast<const float*>(a.dense(3, kF32, {P, H}));
  void* po = a.pitched(4, kBf16 | kF32, {P, T, H}, 8, &ldo);
  const auto* pb = static_cast<const uint16_t*>(a.dense(5, kBf16, {P, H}, true));
  void* st = a.stream(6);
  const int iP = a.size(P), iT = a.size(T), iH = a.size(H), iK = a.size(K);
  const hq_out_dtype odt = a.f32(4) ? HQ_OUT_F32 : HQ_OUT_BF16;
  return run(a, [&] { return hq_int8_matmul(pa, lda, ps, pw, ldw, pws, pb, iP, iT, iH, iK, po, ldo, odt, st); });
}

// int8_matmul_pack(a, a_scale, w, w_scale, keep_idx, rest_idx, inv_scale, zero, codes, side, stream)
PyObject* int8_matmul_pack(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args};
  const at::Tensor* x = n == 11 ? a.first(0, 3) : nullptr;
  const at::Tensor* w = x ? tensor(args[2]) : nullptr;
  const at::Tensor* keep = w ? tensor(args[4]) : nullptr;
  if (!keep || w->dim() != 3 || keep->dim() != 1) Py_RETURN_NONE;
  const int64_t P = x->size(0), T = x->size(1), K = x->size(2), H = w->size(1), k = keep->size(0);
  int lda, ldw;
  const auto* pa = static_cast<const int8_t*>(a.pitched(0, kI8, {P, T, K}, 16, &lda));
  const auto* ps = static_cast<const float*>(a.dense(1, kF32, {P, T}));
  const auto* pw = static_cast<const int8_t*>(a.pitched(2, kI8, {P, H, K}, 16, &ldw));
  const auto* pws = static_cast<const float*>(a.dense(3, kF32, {P, H}));
  const auto* pk = static_cast<const int32_t*>(a.dense(4, kI32, {k}));
  const auto* pr = static_cast<const int32_t*>(a.dense(5, kI32, {H - k}));
  const auto* pi = static_cast<const float*>(a.dense(6, kF32, {P, H}));
  const auto* pz = static_cast<const uint8_t*>(a.dense(7, kU8, {P, H}));
  auto* pc = static_cast<uint32_t*>(a.dense(8, kCodes, {P, T, (H - k) / 8}));
  auto* pd = static_cast<uint16_t*>(a.dense(9, kBf16, {P, k, T}));
  void* st = a.stream(10);
  const int iP = a.size(P), iT = a.size(T), iH = a.size(H), iK = a.size(K), ik = a.size(k);
  return run(a, [&] {
    return hq_int8_matmul_pack(pa, lda, ps, pw, ldw, pws, iP, iT, iH, iK, ik, pk, pr, pi, pz, pc, pd, st);
  });
}

// dequant_reduce(codes, side, keep_idx, rest_idx, scale, zero, out, stream)
PyObject* dequant_reduce(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args};
  const at::Tensor* c = n == 8 ? a.first(0, 3) : nullptr;
  const at::Tensor* keep = c ? tensor(args[2]) : nullptr;
  const at::Tensor* out = keep ? tensor(args[6]) : nullptr;
  if (!out || keep->dim() != 1 || out->dim() != 2) Py_RETURN_NONE;
  const int64_t P = c->size(0), T = c->size(1), k = keep->size(0), H = out->size(1);
  const auto* pc = static_cast<const uint32_t*>(a.dense(0, kCodes, {P, T, (H - k) / 8}));
  const auto* pd = static_cast<const uint16_t*>(a.dense(1, kBf16, {P, k, T}));
  const auto* pk = static_cast<const int32_t*>(a.dense(2, kI32, {k}));
  const auto* pr = static_cast<const int32_t*>(a.dense(3, kI32, {H - k}));
  const auto* ps = static_cast<const float*>(a.dense(4, kF32, {P, H}));
  const auto* pz = static_cast<const uint8_t*>(a.dense(5, kU8, {P, H}));
  void* po = a.dense(6, kBf16 | kF32, {T, H});
  void* st = a.stream(7);
  const int iP = a.size(P), iT = a.size(T), iH = a.size(H), ik = a.size(k);
  const hq_out_dtype odt = a.f32(6) ? HQ_OUT_F32 : HQ_OUT_BF16;
  return run(a, [&] { return hq_dequant_reduce(pc, pd, iP, iT, iH, ik, pk, pr, ps, pz, po, odt, st); });
}

// residual_norm(y, res, res_out, h, q, q_scale, post, post_w, post_b, gate, alpha, beta, pre, pre_w, pre_b, eps, stream)
PyObject* residual_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args};
  const at::Tensor* y = n == 17 ? a.first(0, 2) : nullptr;
  if (!y) Py_RETURN_NONE;
  const int64_t T = y->size(0), H = y->size(1);
  const void* py = a.dense(0, kBf16 | kF32, {T, H});
  const bool f32 = a.f32(1);
  const void* pr = a.dense(1, f32 ? kF32 : kBf16, {T, H});
  void* po = a.dense(2, f32 ? kF32 : kBf16, {T, H});
  auto* ph = static_cast<uint16_t*>(a.dense(3, kBf16, {T, H}, true));
  int ldq = 0;
  auto* pq = args[4] == Py_None ? nullptr : static_cast<int8_t*>(a.pitched(4, kI8, {T, H}, 16, &ldq));
  auto* pqs = static_cast<float*>(a.dense(5, kF32, {T}, true));
  const int post = a.integer(6), pre = a.integer(12);
  const auto* post_w = static_cast<const float*>(a.dense(7, kF32, {H}, true));
  const auto* post_b = static_cast<const float*>(a.dense(8, kF32, {H}, true));
  const uint16_t* gate = nullptr;
  int64_t gate_rows = 0;
  if (args[9] != Py_None) {
    const at::Tensor* g = tensor(args[9]);
    const int64_t G = g && g->dim() == 2 ? g->size(0) : 0;
    if (G < 1 || T % G) Py_RETURN_NONE;
    gate = static_cast<const uint16_t*>(a.dense(9, kBf16, {G, H}));
    gate_rows = T / G > 0 ? T / G : 1;
  }
  const float alpha = a.number(10), beta = a.number(11), eps = a.number(15);
  const auto* pre_w = static_cast<const float*>(a.dense(13, kF32, {H}, true));
  const auto* pre_b = static_cast<const float*>(a.dense(14, kF32, {H}, true));
  void* st = a.stream(16);
  const int iT = a.size(T), iH = a.size(H), ig = a.size(gate_rows);
  const hq_out_dtype ydt = a.f32(0) ? HQ_OUT_F32 : HQ_OUT_BF16;
  return run(a, [&] {
    return hq_residual_norm(py, ydt, pr, po, f32 ? HQ_OUT_F32 : HQ_OUT_BF16, iT, iH,
                            static_cast<hq_norm_kind>(post), post_w, post_b, gate, ig, alpha, beta,
                            static_cast<hq_norm_kind>(pre), pre_w, pre_b, eps, ph, pq, ldq, pqs, st);
  });
}

#define HQ_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(caught<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {HQ_METHOD(quantize_tokens), HQ_METHOD(int8_matmul),   HQ_METHOD(int8_matmul_pack),
                         HQ_METHOD(dequant_reduce),  HQ_METHOD(residual_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hqargs", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

// The module reads tensors by torch's C++ layout: it is for the Python and torch that it was built with.
bool built_for_this() {
  if ((Py_Version >> 16) != (PY_VERSION_HEX >> 16)) {
    PyErr_SetString(PyExc_ImportError, "_hqargs.so was built for Python " PY_VERSION);
    return false;
  }
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  const char* v = version && PyUnicode_Check(version) ? PyUnicode_AsUTF8(version) : nullptr;
  const size_t n = sizeof(TORCH_VERSION) - 1;
  const bool same = v && strncmp(v, TORCH_VERSION, n) == 0 && (v[n] == 0 || v[n] == '+');
  Py_XDECREF(version);
  Py_XDECREF(torch);
  if (!same && !PyErr_Occurred()) PyErr_SetString(PyExc_ImportError, "_hqargs.so was built for torch " TORCH_VERSION);
  return same;
}

}  // namespace

PyMODINIT_FUNC PyInit__hqargs() { return built_for_this() ? PyModule_Create(&module) : nullptr; }

// binding.cpp -- Python entry points of the mixture-of-experts operators: argument
// checks, output allocation and the call of the C ABI, on the current stream of
// the tensors' device.
//
// These calls take a few microseconds on the GPU at decode sizes, so their host
// side decides: from Python (attribute checks, torch.empty, ctypes) a residual
// norm took 13.3 us per call, of which the launch itself is 2.3.  Here the
// checks and allocations go through the C++ API directly: 5.2 us the norm, 4.1 the activation,
// 3.6 a grouped product.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/sqint8.h"

namespace {

PyObject* g_error_class = nullptr;   // SqError(function, status)
PyObject* g_memory_error = nullptr;  // torch.OutOfMemoryError

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor& tensor(PyObject* o, const char* fn, const char* name) {
  if (!THPVariable_Check(o)) throw Bad(std::string(fn) + ": " + name + " is not a tensor");
  return THPVariable_Unpack(o);
}

std::string list(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

// t has this type and shape, is contiguous and on CUDA device dev.
void fits(const char* fn, const char* name, const at::Tensor& t, int dev, at::ScalarType type,
          at::IntArrayRef shape) {
  if (t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.sizes() == shape &&
      t.is_contiguous())
    return;
  throw Bad(std::string(fn) + ": " + name + " is " + c10::toString(t.scalar_type()) + " " + list(t.sizes()) +
            " on " + t.device().str() + (t.is_contiguous() ? "" : " (not contiguous)") +
            ", expected contiguous " + c10::toString(type) + " " + list(shape) + " on cuda:" +
            std::to_string(dev));
}

int device_of(const char* fn, const char* name, const at::Tensor& t, int64_t dims) {
  if (!t.is_cuda() || t.dim() != dims)
    throw Bad(std::string(fn) + ": " + name + " is " + list(t.sizes()) + " on " + t.device().str() +
              ", expected a CUDA tensor of " + std::to_string(dims) + " dimensions");
  return t.get_device();
}

// Straight from the caching allocator (on the current device): at::empty's
// dispatch and guard cost as much again.  Every output has a storage of its own, as a torch
// caller expects: resizing, freeing or saving one touches no other.  (Parts of one allocation
// took 0.3 us less for each further output.)
at::Tensor make(at::IntArrayRef shape, at::ScalarType type) {
  const size_t bytes = static_cast<size_t>(c10::multiply_integers(shape)) * c10::elementSize(type);
  c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                         from->allocate(bytes), from, /*resizable=*/true)),
      c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

at::Tensor make_scales(int64_t rows, int64_t K, bool per_row) {
  return per_row ? make({rows}, at::kFloat) : make({rows, K / 128}, at::kFloat);
}

// The C entry points want 16-byte aligned operands.  Scales, factors, offsets and row indexes may
// be views that start at any element (a range of experts, a chunk of tokens): then they
// are copied, in stream order, to memory of their own, which is `t` from then on.
void align(at::Tensor& t) {
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0) return;
  at::AutoDispatchBelowADInplaceOrView plain;  // no gradient is recorded
  at::Tensor copy = make(t.sizes(), t.scalar_type());
  copy.copy_(t, /*non_blocking=*/true);
  t = std::move(copy);
}

PyObject* fail(const char* fn, sq_status rc) {
  PyObject* e = PyObject_CallFunction(g_error_class, "si", fn, static_cast<int>(rc));
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  return nullptr;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// Without the interpreter's lock while it lives, like torch's own calls: an allocation may wait
// for the device and a launch for room in its queue, and other host threads have to
// go on meanwhile (a host callback that the queue waits for may be one of theirs).
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory_error, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// (h, residual, gamma, eps, group, residual_out or None, fp8)
PyObject* add_rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  const double eps = PyFloat_AsDouble(a[3]);
  const long long group = PyLong_AsLongLong(a[4]);
  const int fp8 = PyObject_IsTrue(a[6]);
  if (PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* fn = fp8 ? "sq_add_rmsnorm_quant_fp8" : "sq_add_rmsnorm_quant";
    const at::Tensor &h = tensor(a[0], fn, "h"), &res = tensor(a[1], fn, "residual");
    at::Tensor gamma = tensor(a[2], fn, "gamma");
    const int dev = device_of(fn, "h", h, 2);
    const int64_t M = h.size(0), K = h.size(1);
    fits(fn, "h", h, dev, at::kBFloat16, {M, K});
    fits(fn, "residual", res, dev, at::kBFloat16, {M, K});
    fits(fn, "gamma", gamma, dev, at::kFloat, {K});
    at::Tensor out, q, sc, r;
    if (a[5] != Py_None) {
      out = tensor(a[5], fn, "residual_out");
      fits(fn, "residual_out", out, dev, at::kBFloat16, {M, K});
    }
    sq_status rc;
    {
      Unlocked unlocked;
      c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
      if (!out.defined()) out = make({M, K}, at::kBFloat16);
      q = make({M, K}, fp8 ? at::kByte : at::kChar);
      sc = make_scales(M, K, !fp8 && group != 128);
      r = make({M}, at::kFloat);
      align(gamma);
      rc = fp8 ? sq_add_rmsnorm_quant_fp8(h.data_ptr(), res.data_ptr(), static_cast<float*>(gamma.data_ptr()),
                                          static_cast<float>(eps), out.data_ptr(),
                                          static_cast<uint8_t*>(q.data_ptr()), static_cast<float*>(sc.data_ptr()),
                                          static_cast<float*>(r.data_ptr()), M, K, stream_of(dev))
               : sq_add_rmsnorm_quant(h.data_ptr(), res.data_ptr(), static_cast<float*>(gamma.data_ptr()),
                                      static_cast<float>(eps), group, out.data_ptr(),
                                      static_cast<int8_t*>(q.data_ptr()), static_cast<float*>(sc.data_ptr()),
                                      static_cast<float*>(r.data_ptr()), M, K, stream_of(dev));
    }
    if (rc != SQ_OK) return fail(fn, rc);
    PyObject* o = nullptr;
    if (a[5] == Py_None) {
      o = THPVariable_Wrap(std::move(out));
    } else {
      o = a[5];
      Py_INCREF(o);
    }
    return Py_BuildValue("(NNNN)", o, THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(sc)),
                         THPVariable_Wrap(std::move(r)));
  });
}

// (gate_up, inv_s or None, group, fp8)
PyObject* silu_mul_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 4)) return nullptr;
  const long long group = PyLong_AsLongLong(a[2]);
  const int fp8 = PyObject_IsTrue(a[3]);
  if (PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* fn = fp8 ? "sq_silu_mul_quant_fp8" : "sq_silu_mul_quant";
    const at::Tensor& gu = tensor(a[0], fn, "gate_up");
    const int dev = device_of(fn, "gate_up", gu, 2);
    const int64_t T = gu.size(0), K = gu.size(1) / 2;
    fits(fn, "gate_up", gu, dev, at::kBFloat16, {T, 2 * K});
    at::Tensor inv_s, q, sc;
    if (a[1] != Py_None) {
      inv_s = tensor(a[1], fn, "inv_s");
      fits(fn, "inv_s", inv_s, dev, at::kFloat, {K});
    }
    sq_status rc;
    {
      Unlocked unlocked;
      c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
      q = make({T, K}, fp8 ? at::kByte : at::kChar);
      sc = make_scales(T, K, !fp8 && group != 128);
      if (inv_s.defined()) align(inv_s);
      const float* inv = inv_s.defined() ? static_cast<const float*>(inv_s.data_ptr()) : nullptr;
      rc = fp8 ? sq_silu_mul_quant_fp8(gu.data_ptr(), inv, static_cast<uint8_t*>(q.data_ptr()),
                                       static_cast<float*>(sc.data_ptr()), T, K, stream_of(dev))
               : sq_silu_mul_quant(gu.data_ptr(), inv, group, static_cast<int8_t*>(q.data_ptr()),
                                   static_cast<float*>(sc.data_ptr()), T, K, stream_of(dev));
    }
    if (rc != SQ_OK) return fail(fn, rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(sc)));
  });
}

// (q_a, s_a, q_w, s_w, offsets, rows or None, out or None, fp8)
PyObject* grouped_mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 8)) return nullptr;
  const int fp8 = PyObject_IsTrue(a[7]);
  if (PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* fn = fp8 ? "fp8_block_grouped_mm" : "w8a8_grouped_mm";
    const at::Tensor &qa = tensor(a[0], fn, "q_a"), &qw = tensor(a[2], fn, "q_w");
    at::Tensor sa = tensor(a[1], fn, "s_a"), sw = tensor(a[3], fn, "s_w"), off = tensor(a[4], fn, "offsets"), row;
    const int dev = device_of(fn, "q_a", qa, 2);
    device_of(fn, "q_w", qw, 3);
    const int64_t M = qa.size(0), K = qa.size(1), E = qw.size(0), N = qw.size(1);
    const at::ScalarType code = fp8 ? at::kByte : at::kChar;
    fits(fn, "q_a", qa, dev, code, {M, K});
    if (fp8) fits(fn, "s_a", sa, dev, at::kFloat, {M, K / 128});
    else fits(fn, "s_a", sa, dev, at::kFloat, {M});
    fits(fn, "q_w", qw, dev, code, {E, N, K});
    if (fp8) fits(fn, "s_w", sw, dev, at::kFloat, {E, N / 128, K / 128});
    else fits(fn, "s_w", sw, dev, at::kFloat, {E, N});
    fits(fn, "offsets", off, dev, at::kInt, {E + 1});
    int64_t T = M;
    if (a[5] != Py_None) {
      row = tensor(a[5], fn, "rows");
      T = row.numel();
      fits(fn, "rows", row, dev, at::kInt, {T});
    }
    at::Tensor y;
    if (a[6] != Py_None) {
      y = tensor(a[6], fn, "out");
      fits(fn, "out", y, dev, at::kBFloat16, {T, N});
    }
    sq_status rc;
    {
      Unlocked unlocked;
      c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
      if (!y.defined()) y = make({T, N}, at::kBFloat16);
      for (at::Tensor* t : {&sa, &sw, &off}) align(*t);
      if (row.defined()) align(row);
      const float *psa = static_cast<const float*>(sa.data_ptr()), *psw = static_cast<const float*>(sw.data_ptr());
      const int32_t *poff = static_cast<const int32_t*>(off.data_ptr()),
                    *rows = row.defined() ? static_cast<const int32_t*>(row.data_ptr()) : nullptr;
      rc = fp8 ? fp8_block_grouped_mm(static_cast<const uint8_t*>(qa.data_ptr()), psa, rows,
                                      static_cast<const uint8_t*>(qw.data_ptr()), psw, poff, y.data_ptr(), T, M, E,
                                      N, K, stream_of(dev))
               : w8a8_grouped_mm(static_cast<const int8_t*>(qa.data_ptr()), psa, rows,
                                 static_cast<const int8_t*>(qw.data_ptr()), psw, poff, y.data_ptr(), T, M, E, N, K,
                                 stream_of(dev));
    }
    if (rc != SQ_OK) return fail(fn, rc);
    if (a[6] != Py_None) {
      Py_INCREF(a[6]);
      return a[6];
    }
    return THPVariable_Wrap(std::move(y));
  });
}

PyObject* set_errors(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 2)) return nullptr;
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XDECREF(g_error_class);
  Py_XDECREF(g_memory_error);
  g_error_class = a[0];
  g_memory_error = a[1];
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {{"add_rmsnorm_quant", FAST(add_rmsnorm_quant), nullptr},
                          {"silu_mul_quant", FAST(silu_mul_quant), nullptr},
                          {"grouped_mm", FAST(grouped_mm), nullptr},
                          {"set_errors", FAST(set_errors), nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&kModule);
  // what this file was compiled for (build.py), compared when it is loaded
  if (m && PyModule_AddStringConstant(m, "built_for", SQ_BINDING_KEY) != 0) Py_CLEAR(m);
  return m;
}

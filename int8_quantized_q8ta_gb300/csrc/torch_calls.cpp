// torch_calls.cpp -- the calls of tokens.py for the common case, from Python
// straight to the C functions of include/q8ta.h: tensors as they should be, on
// the current device, results and workspace from torch's allocator, nothing to
// record for autograd.  Such a call for a few rows takes the GPU some 3 to 15 us,
// and marshalling in Python took the host 18 (with two launches; 12 with one);
// here it takes 7.4 (5).  Allocations and launches run without the interpreter's
// lock.
//
// A function answers None where anything is not so, and the status, an int,
// where the C function refuses: tokens.py then goes its own way, which checks
// every argument by name.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "q8ta.h"

namespace {

using at::ScalarType;
using at::Tensor;

// -1: not a type of the library's
int code_of(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return Q8_F32;
    case ScalarType::Half: return Q8_F16;
    case ScalarType::BFloat16: return Q8_BF16;
    case ScalarType::Char: return Q8_I8;
    default: return -1;
  }
}
ScalarType type_of(int code) {
  return code == Q8_F32 ? ScalarType::Float : code == Q8_F16 ? ScalarType::Half : ScalarType::BFloat16;
}

// One call's tensors: all contiguous, on one device, which is the current one.
struct Call {
  c10::DeviceIndex device = -1;

  const Tensor* get(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) return nullptr;
    if (device < 0) device = t.get_device();
    return t.get_device() == device ? &t : nullptr;
  }
  // A matrix (rows and columns as they are), or a tensor of this type and shape.
  const Tensor* matrix(PyObject* o) {
    const Tensor* t = get(o);
    return t != nullptr && t->dim() == 2 && code_of(t->scalar_type()) >= 0 ? t : nullptr;
  }
  const Tensor* tensor(PyObject* o, ScalarType type, int64_t n) {
    const Tensor* t = get(o);
    return t != nullptr && t->scalar_type() == type && t->dim() == 1 && t->size(0) == n ? t : nullptr;
  }
  const Tensor* tensor(PyObject* o, ScalarType type, int64_t m, int64_t n) {
    const Tensor* t = get(o);
    return t != nullptr && t->scalar_type() == type && t->dim() == 2 && t->size(0) == m &&
                   t->size(1) == n
               ? t
               : nullptr;
  }
  // scales or biases: [n], or [2, n] of a gated pair
  const Tensor* vector(PyObject* o, bool pair, int64_t n) {
    return pair ? tensor(o, ScalarType::Float, 2, n) : tensor(o, ScalarType::Float, n);
  }
  bool current() const { return c10::cuda::current_device() == device; }
  q8_stream_t stream() const {
    return reinterpret_cast<q8_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
  }
  Tensor empty(at::IntArrayRef sizes, ScalarType type) const {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, device));
  }
  // Some sizes need none; freed to torch's allocator once the call is enqueued.
  Tensor workspace(size_t bytes) const {
    return bytes == 0 ? Tensor() : empty({static_cast<int64_t>(bytes)}, ScalarType::Byte);
  }
};

void* at_or_null(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
void* space_of(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T* as(const Tensor* t) {
  return static_cast<T*>(at_or_null(t));
}

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}
PyObject* answer(q8_status st, Tensor out) {
  return st == Q8_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(st);
}

// C++ exceptions (an allocation that fails) as Python's.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    at::AutoDispatchBelowADInplaceOrView below;   // nothing here is recorded
    return f();
  } catch (const std::bad_alloc&) {
    return PyErr_NoMemory();
  } catch (const std::exception&) {
    return none();   // the slow way says what is wrong, in torch's words
  }
}

// The interpreter's lock, let go of for as long as this lives: allocations and
// launches may wait for the GPU (a full launch queue), and other threads run on
// meanwhile.  The arguments' tensors live: the caller holds them.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// Whether autograd follows this tensor, backward or forward: tokens.py says then
// what is recorded and what is refused.
bool followed(const Tensor* t) {
  return t != nullptr && ((at::GradMode::is_enabled() && t->requires_grad()) ||
                          (c10::AutogradState::get_tls_state().get_fw_grad_mode() &&
                           t->_fw_grad(0).defined()));
}

// dtype argument: None (`otherwise`), or a float type of the library's; else -1
int out_code(PyObject* o, int otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) return -1;
  const int code = code_of(reinterpret_cast<THPDtype*>(o)->scalar_type);
  return code == Q8_I8 ? -1 : code;
}

// x -> (q, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    Call c;
    const Tensor* x = c.matrix(a[0]);
    if (x == nullptr || x->scalar_type() == ScalarType::Char || !c.current() || followed(x))
      return none();
    const int64_t M = x->size(0), K = x->size(1);
    Tensor q, s;
    q8_status st;
    {
      const Unlocked unlocked;
      q = c.empty({M, K}, ScalarType::Char);
      s = c.empty({M}, ScalarType::Float);
      st = q8_quantize_per_token(x->data_ptr(), static_cast<q8_dtype>(code_of(x->scalar_type())), M, K,
                                 as<int8_t>(&q), as<float>(&s), c.stream());
    }
    if (st != Q8_OK) return PyLong_FromLong(st);
    PyObject* both = PyTuple_New(2);
    if (both == nullptr) return nullptr;
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(std::move(q)));
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(std::move(s)));
    return both;
  });
}

// q, scales, dtype -> x
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Call c;
    const Tensor* q = c.matrix(a[0]);
    if (q == nullptr || q->scalar_type() != ScalarType::Char || !c.current()) return none();
    const int64_t M = q->size(0), K = q->size(1);
    const Tensor* s = c.tensor(a[1], ScalarType::Float, M);
    const int code = out_code(a[2], -1);
    if (s == nullptr || code < 0 || followed(s)) return none();
    Tensor out;
    q8_status st;
    {
      const Unlocked unlocked;
      out = c.empty({M, K}, type_of(code));
      st = q8_dequantize_per_token(as<int8_t>(q), as<float>(s), M, K, static_cast<q8_dtype>(code),
                                   out.data_ptr(), c.stream());
    }
    return answer(st, out);
  });
}

// The product or the gated pair: x, x_scales, packed, N, K, weight_scales, bias,
// activation, out_dtype -> y
template <bool GATED>
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call c;
    const Tensor* x = c.matrix(a[0]);
    if (x == nullptr || !c.current()) return none();
    const int64_t N = PyLong_AsLongLong(a[3]), K = PyLong_AsLongLong(a[4]);
    const int64_t M = x->size(0);
    const int code = code_of(x->scalar_type());
    if (x->size(1) != K || (code == Q8_I8) != (a[1] != Py_None)) return none();
    const Tensor* xs = a[1] == Py_None ? nullptr : c.tensor(a[1], ScalarType::Float, M);
    const Tensor* w = c.get(a[2]);
    const Tensor* ws = c.vector(a[5], GATED, N);
    const Tensor* b = a[6] == Py_None ? nullptr : c.vector(a[6], GATED, N);
    const char* act = PyUnicode_Check(a[7]) ? PyUnicode_AsUTF8(a[7]) : nullptr;
    const int out_type = out_code(a[8], code == Q8_I8 ? static_cast<int>(Q8_BF16) : code);
    if ((xs == nullptr) != (a[1] == Py_None) || w == nullptr || ws == nullptr ||
        (b == nullptr) != (a[6] == Py_None) || act == nullptr || out_type < 0)
      return none();
    if (followed(x) || followed(xs) || followed(ws) || followed(b)) return none();
    Tensor out;
    q8_status st;
    {
      const Unlocked unlocked;
      out = c.empty({M, N}, type_of(out_type));
      const size_t bytes = GATED ? q8_linear_gated_workspace_bytes(M, K, N)
                                 : q8_linear_per_token_workspace_bytes(M, K, N);
      const Tensor space = c.workspace(bytes);
      st = (GATED ? q8_linear_gated : q8_linear_per_token)(
          x->data_ptr(), static_cast<q8_dtype>(code), M, K, nullptr, as<float>(xs), w->data_ptr(), N,
          as<float>(ws), as<float>(b), act, static_cast<q8_dtype>(out_type), out.data_ptr(),
          space_of(space), bytes, c.stream());
    }
    return answer(st, out);
  });
}

// dy, packed_t, N, K, weight_scales, y -> dx
PyObject* product_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Call c;
    const Tensor* dy = c.matrix(a[0]);
    if (dy == nullptr || !c.current()) return none();
    const int64_t N = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]), M = dy->size(0);
    const ScalarType type = dy->scalar_type();
    const Tensor* w = c.get(a[1]);
    const Tensor* ws = c.vector(a[4], false, N);
    const Tensor* y = a[5] == Py_None ? nullptr : c.tensor(a[5], type, M, N);
    if (dy->size(1) != N || w == nullptr || ws == nullptr || (y == nullptr) != (a[5] == Py_None) ||
        (type != ScalarType::Half && type != ScalarType::BFloat16))
      return none();
    Tensor out;
    q8_status st;
    {
      const Unlocked unlocked;
      out = c.empty({M, K}, type);
      const size_t bytes = q8_linear_per_token_backward_workspace_bytes(M, N, K);
      const Tensor space = c.workspace(bytes);
      st = q8_linear_per_token_backward(dy->data_ptr(), static_cast<q8_dtype>(code_of(type)), M, N,
                                        at_or_null(y), w->data_ptr(), K, as<float>(ws),
                                        out.data_ptr(), space_of(space), bytes, c.stream());
    }
    return answer(st, out);
  });
}

// dh, x, x_scales, packed, packed_t, N, K, weight_scales, bias, activation -> dx
PyObject* gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c;
    const Tensor* dh = c.matrix(a[0]);
    if (dh == nullptr || !c.current()) return none();
    const int64_t N = PyLong_AsLongLong(a[5]), K = PyLong_AsLongLong(a[6]), M = dh->size(0);
    const ScalarType type = dh->scalar_type();
    const Tensor* x = c.tensor(a[1], ScalarType::Char, M, K);
    const Tensor* xs = c.tensor(a[2], ScalarType::Float, M);
    const Tensor *w = c.get(a[3]), *wt = c.get(a[4]);
    const Tensor* ws = c.vector(a[7], true, N);
    const Tensor* b = a[8] == Py_None ? nullptr : c.vector(a[8], true, N);
    const char* act = PyUnicode_Check(a[9]) ? PyUnicode_AsUTF8(a[9]) : nullptr;
    if (dh->size(1) != N || x == nullptr || xs == nullptr || w == nullptr || wt == nullptr ||
        ws == nullptr || (b == nullptr) != (a[8] == Py_None) || act == nullptr ||
        (type != ScalarType::Half && type != ScalarType::BFloat16))
      return none();
    Tensor out;
    q8_status st;
    {
      const Unlocked unlocked;
      out = c.empty({M, K}, type);
      const size_t bytes = q8_linear_gated_backward_workspace_bytes(M, K, N);
      const Tensor space = c.workspace(bytes);
      st = q8_linear_gated_backward(dh->data_ptr(), static_cast<q8_dtype>(code_of(type)), M, N,
                                    as<int8_t>(x), as<float>(xs), K, w->data_ptr(), wt->data_ptr(),
                                    as<float>(ws), as<float>(b), act, out.data_ptr(), space_of(space),
                                    bytes, c.stream());
    }
    return answer(st, out);
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() {
  static PyMethodDef methods[] = {
      {"quantize_per_token", fast(quantize), METH_FASTCALL, nullptr},
      {"dequantize_per_token", fast(dequantize), METH_FASTCALL, nullptr},
      {"linear_per_token", fast(product<false>), METH_FASTCALL, nullptr},
      {"linear_gated", fast(product<true>), METH_FASTCALL, nullptr},
      {"linear_per_token_backward", fast(product_backward), METH_FASTCALL, nullptr},
      {"linear_gated_backward", fast(gated_backward), METH_FASTCALL, nullptr},
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                               nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}

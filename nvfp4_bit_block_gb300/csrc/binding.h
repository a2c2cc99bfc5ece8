// binding.h -- what the Python bindings of the layer and attention operators share:
// argument checks, result tensors, errors.
#pragma once

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <string>

#include "nvfp4.h"

namespace {

struct Refused {
  PyObject* type;
  std::string what;
};
struct Status {
  int64_t status;
  const char* where;
};

[[noreturn]] void value_error(std::string s) { throw Refused{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void type_error(std::string s) { throw Refused{PyExc_TypeError, std::move(s)}; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor* tensor(PyObject* o, const char* name) {  // nullptr for None
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) type_error(std::string(name) + " must be a tensor");
  return *t;
}
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Refused{nullptr, ""};
  return r != 0;
}
// 1 for bfloat16, 0 for float32.
int is_bf16(at::ScalarType t, const char* name) {
  if (t == at::kBFloat16) return 1;
  if (t == at::kFloat) return 0;
  type_error(std::string(name) + " must be torch.bfloat16 or torch.float32 (got " + c10::toString(t) + ")");
}
at::ScalarType dtype_of(PyObject* o, at::ScalarType none) {
  if (o == Py_None) return none;
  if (!THPDtype_Check(o)) type_error("out_dtype must be a torch.dtype");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  is_bf16(t, "out_dtype");
  return t;
}

void on_device(const at::Tensor& t, const char* name, c10::Device dev) {
  if (!t.is_cuda() || t.device() != dev)
    value_error(std::string(name) + " must be a CUDA tensor on " + dev.str() + " (got " + t.device().str() + ")");
}

struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
};
void check_shape(const at::Tensor& t, const char* name, int64_t M, int64_t N) {
  if (t.size(0) != M || t.size(1) != N)
    value_error(std::string(name) + " must have shape (" + std::to_string(M) + ", " + std::to_string(N) + ") (got " +
                shape_of(t) + ")");
}
// A 2-D tensor on `dev` with unit column stride.
Matrix matrix(const at::Tensor& t, const char* name, c10::Device dev) {
  if (t.dim() != 2) type_error(std::string(name) + " must be a 2-D tensor");
  on_device(t, name, dev);
  if (t.size(1) > 1 && t.stride(1) != 1) value_error(std::string(name) + " must have unit stride along columns");
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), 1)};
}
Matrix matrix(const at::Tensor& t, const char* name, c10::Device dev, int64_t M, int64_t N, at::ScalarType type) {
  const Matrix m = matrix(t, name, dev);
  check_shape(t, name, M, N);
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + " (got " + c10::toString(t.scalar_type()) + ")");
  return m;
}
// A contiguous tensor of n elements; nullptr for None.
void* vector(const at::Tensor* t, const char* name, int64_t n, c10::Device dev) {
  if (!t) return nullptr;
  on_device(*t, name, dev);
  if (t->numel() != n || !t->is_contiguous())
    value_error(std::string(name) + " must be contiguous with " + std::to_string(n) + " elements (got " + shape_of(*t) +
                ")");
  return t->data_ptr();
}
void* vector(const at::Tensor* t, const char* name, int64_t n, c10::Device dev, at::ScalarType type) {
  void* p = vector(t, name, n, dev);
  if (t && t->scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + " (got " + c10::toString(t->scalar_type()) + ")");
  return p;
}

// A new tensor on `dev` (straight from the CUDA allocator, without the dispatcher's way there).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType t, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(sizes, t, dev, std::nullopt));
}
at::Tensor new_matrix(int64_t M, int64_t N, at::ScalarType t, c10::Device dev) { return fresh({M, N}, t, dev); }

// Small fp32 results of one call: each 16-byte aligned in one allocation that they share.
class Floats {
 public:
  explicit Floats(c10::Device dev) : dev_(dev) {}
  int64_t add(int64_t n) {
    const int64_t at = total_;
    total_ += (n + 3) / 4 * 4;
    return at;
  }
  void make() {
    if (total_ > 0) base_ = fresh({total_}, at::kFloat, dev_);
  }
  float* ptr(int64_t at) { return base_.defined() ? base_.data_ptr<float>() + at : nullptr; }
  at::Tensor view(int64_t at, int64_t n) {
    if (!base_.defined()) return fresh({n}, at::kFloat, dev_);
    auto t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base_.storage()), base_.key_set(), base_.dtype());
    c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    impl->set_sizes_contiguous({n});
    impl->set_storage_offset(at);
    return t;
  }

 private:
  c10::Device dev_;
  int64_t total_ = 0;
  at::Tensor base_;
};

// Scratch memory on the current stream, and its size; nothing where none is needed.
struct Workspace {
  at::Tensor t;
  void* p = nullptr;
  int64_t n = 0;
  Workspace() = default;
  Workspace(int64_t bytes, const char* where, c10::Device dev) : n(bytes) {
    if (n < 0) throw Status{n, where};
    if (n > 0) {
      t = fresh({n}, at::kByte, dev);
      p = t.data_ptr();
    }
  }
};

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
void check(int status, const char* where) {
  if (status != 0) throw Status{status, where};
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}
template <typename... P>
PyObject* tuple(P*... p) {
  PyObject* items[] = {p...};
  PyObject* t = PyTuple_New(sizeof...(p));
  for (size_t i = 0; i < sizeof...(p); ++i) PyTuple_SET_ITEM(t, (Py_ssize_t)i, items[i]);
  return t;
}

// Every C++ exception becomes a Python one here; none passes into the interpreter.
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != ARGS) type_error("wrong number of arguments");
    return F(args);
  } catch (const Refused& e) {
    if (e.type) PyErr_SetString(e.type, e.what.c_str());
  } catch (const Status& e) {
    PyObject* m = PyImport_ImportModule("nvfp4_bit_block_gb300");
    PyObject* c = m ? PyObject_GetAttrString(m, "Nvfp4Error") : nullptr;
    PyObject* v = c ? PyObject_CallFunction(c, "Ls", (long long)e.status, e.where) : nullptr;
    if (v) PyErr_SetObject(c, v);
    Py_XDECREF(v);
    Py_XDECREF(c);
    Py_XDECREF(m);
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* m = PyImport_ImportModule("torch");
    PyObject* c = m ? PyObject_GetAttrString(m, "OutOfMemoryError") : nullptr;
    if (c) PyErr_SetString(c, e.what_without_backtrace());
    Py_XDECREF(c);
    Py_XDECREF(m);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, ARGS>)), METH_FASTCALL, nullptr};
}

}  // namespace

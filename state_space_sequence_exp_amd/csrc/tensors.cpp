// tensors.cpp -- what a call of the short operators asks of its tensors, asked in
// one go, and the new ones it returns: a Python module of three functions.  A tensor's type, shape, device, strides
// and address cost about a microsecond from Python; a single-token call has a dozen
// tensors and runs for five.
//
//   dense(dtype, shape, device index, t, ...) -> (address, ...)
//   rows(dtype, shape, device index, t, ...)  -> (address, distance, ...)
//
// Every t is a tensor of this type, shape and device, contiguous (dense), or with a
// contiguous last axis and its rows at one distance (rows: 0 for a contiguous one,
// else elements from one row to the next), or None (address 0).  None is returned
// where one is not: the caller then finds out which, and says so.
//
//   empty(dtype, shape, t) -> a new tensor on t's device
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <utility>

namespace {

using Sizes = c10::SmallVector<int64_t, 8>;  // (more dimensions than that take an allocation)

struct Wanted {
  at::ScalarType type;
  Sizes sizes;
  long device;
};

// The numbers of a tuple; false with Python's error set.
bool sizes_of(PyObject* tuple, Sizes& sizes) {
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tuple); ++i) {
    sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i)));
    if (sizes.back() == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

// The first three arguments.
bool wanted(PyObject* const* args, Py_ssize_t n, Wanted& w) {
  if (n < 3 || !THPDtype_Check(args[0]) || !PyTuple_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "expected (dtype, shape, device index, tensors...)");
    return false;
  }
  w.type = reinterpret_cast<THPDtype*>(args[0])->scalar_type;
  if (!sizes_of(args[1], w.sizes)) return false;
  w.device = PyLong_AsLong(args[2]);
  return !(w.device == -1 && PyErr_Occurred());
}

bool matches(const at::Tensor& t, const Wanted& w) {
  if (t.scalar_type() != w.type || t.layout() != at::kStrided || t.sizes() != at::IntArrayRef(w.sizes)) return false;
  return (t.is_cuda() ? (long)t.get_device() : -1) == w.device;
}

// Elements from one row to the next (0: contiguous), or -1.
int64_t distance(const at::Tensor& t) {
  if (t.is_contiguous()) return 0;
  const at::IntArrayRef sizes = t.sizes(), strides = t.strides();
  const int64_t last = t.dim() - 1, row = last < 0 ? 1 : sizes[last];
  if (row > 1 && strides[last] != 1) return -1;
  int64_t ld = 0, step = 0;
  for (int64_t i = last - 1; i >= 0; --i) {
    if (sizes[i] == 1) continue;
    if (ld == 0) ld = step = strides[i];
    if (strides[i] != step || strides[i] < row) return -1;
    step *= sizes[i];
  }
  return ld;
}

// A reference to a new object, given up where it is not handed on.
class Held {
 public:
  explicit Held(PyObject* p) : p_(p) {}
  Held(const Held&) = delete;
  Held& operator=(const Held&) = delete;
  ~Held() { Py_XDECREF(p_); }
  PyObject* get() const { return p_; }
  PyObject* hand_on() { return std::exchange(p_, nullptr); }

 private:
  PyObject* p_;
};

template <bool kRows>
PyObject* check(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Wanted w;
  if (!wanted(args, n, w)) return nullptr;
  constexpr int kEach = kRows ? 2 : 1;
  Held out(PyTuple_New((n - 3) * kEach));
  if (!out.get()) return nullptr;
  for (Py_ssize_t i = 3; i < n; ++i) {
    int64_t ld = 0;
    uintptr_t at = 0;
    if (args[i] != Py_None) {
      if (!THPVariable_Check(args[i])) Py_RETURN_NONE;
      const at::Tensor& t = THPVariable_Unpack(args[i]);
      if (!matches(t, w)) Py_RETURN_NONE;
      if (kRows ? (ld = distance(t)) < 0 : !t.is_contiguous()) Py_RETURN_NONE;
      at = reinterpret_cast<uintptr_t>(t.data_ptr());
    }
    PyObject* address = PyLong_FromUnsignedLongLong(at);
    if (!address) return nullptr;
    PyTuple_SET_ITEM(out.get(), (i - 3) * kEach, address);
    if (kRows) {
      PyObject* between = PyLong_FromLongLong(ld);
      if (!between) return nullptr;
      PyTuple_SET_ITEM(out.get(), (i - 3) * kEach + 1, between);
    }
  }
  return out.hand_on();
}

PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != 3 || !THPDtype_Check(args[0]) || !PyTuple_Check(args[1]) || !THPVariable_Check(args[2])) {
      PyErr_SetString(PyExc_TypeError, "expected (dtype, shape, tensor)");
      return nullptr;
    }
    Sizes sizes;
    if (!sizes_of(args[1], sizes)) return nullptr;
    const auto like = THPVariable_Unpack(args[2]).options();
    return THPVariable_Wrap(at::empty(at::IntArrayRef(sizes),
                                      like.dtype(reinterpret_cast<THPDtype*>(args[0])->scalar_type).requires_grad(false)));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (no C++ exception reaches Python's frames: torch's own become its errors)
template <bool kRows>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return check<kRows>(self, args, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"dense", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<false>)), METH_FASTCALL,
     "Addresses of contiguous tensors of one type, shape and device; None where one is not."},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<true>)), METH_FASTCALL,
     "Addresses and row distances of tensors of one type, shape and device; None where one is not."},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&empty)), METH_FASTCALL,
     "A new tensor of this type and shape on a tensor's device."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }

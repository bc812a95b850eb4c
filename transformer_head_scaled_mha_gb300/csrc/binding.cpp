// The inner part of the Python binding of include/mha_paged.h: a tensor's checks, and the
// calls.  A step of generation makes some calls of a few microseconds each, with ten tensors
// to a call; in Python a tensor's checks take 0.35 us and a call through ctypes 2 us, here
// 0.07 and 0.2.
//
// Entry points come by address (bind), so that there is one libmha.so; what a function is
// given it takes from the header's declaration.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <tuple>
#include <type_traits>
#include <utility>

#include "mha_paged.h"

namespace {

PyObject *plain_at;  // the same check in Python, for what is no tensor and for the refusals

// at(name, tensor or None, shape, dtype, device number): the tensor's address, or None.
PyObject *at_checked(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n == 5 && args[1] == Py_None) Py_RETURN_NONE;
  if (n == 5 && THPVariable_Check(args[1]) && PyTuple_Check(args[2]) && THPDtype_Check(args[3]) &&
      PyLong_Check(args[4])) {
    try {
      const at::Tensor &t = THPVariable_Unpack(args[1]);
      const Py_ssize_t dims = PyTuple_GET_SIZE(args[2]);
      bool same = t.layout() == at::kStrided && t.dim() == dims &&
                  t.scalar_type() == reinterpret_cast<THPDtype *>(args[3])->scalar_type &&
                  t.get_device() == PyLong_AsLong(args[4]);
      for (Py_ssize_t i = 0; same && i < dims; ++i)
        same = t.size(i) == PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], i));
      if (same && t.is_contiguous() && !PyErr_Occurred()) return PyLong_FromVoidPtr(t.data_ptr());
    } catch (...) {  // (a tensor without memory, for instance)
    }
    PyErr_Clear();
  }
  return PyObject_Vectorcall(plain_at, args, n, nullptr);
}

// One argument of a C function; an error is left with Python.
template <typename T>
T from(PyObject *o) {
  if constexpr (std::is_pointer_v<T>) {
    return o == Py_None ? nullptr : reinterpret_cast<T>(PyLong_AsVoidPtr(o));
  } else if constexpr (std::is_floating_point_v<T>) {
    return static_cast<T>(PyFloat_AsDouble(o));
  } else if constexpr (std::is_same_v<T, size_t>) {
    return PyLong_AsSize_t(o);
  } else {
    static_assert(std::is_same_v<T, int>, "what the header's functions take");
    const long v = PyLong_AsLong(o);
    if (v > INT_MAX || v < INT_MIN) {
      PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
      return 0;
    }
    return static_cast<int>(v);
  }
}

// The call of entry point F, at `address` (F itself gives the types and tells entries apart;
// nothing here links to the library).
template <auto F>
struct Call;
template <typename R, typename... A, R (*F)(A...)>
struct Call<F> {
  static inline R (*address)(A...) = nullptr;
  template <size_t... I>
  static PyObject *with(PyObject *const *args, std::index_sequence<I...>) {
    const std::tuple<A...> values{from<A>(args[I])...};
    if (PyErr_Occurred()) return nullptr;
    R result;
    Py_BEGIN_ALLOW_THREADS;
    result = std::apply(address, values);
    Py_END_ALLOW_THREADS;
    if constexpr (std::is_same_v<R, int>) return PyLong_FromLong(result);
    else return PyLong_FromSize_t(result);
  }
  static PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != sizeof...(A) || address == nullptr)
      return PyErr_Format(PyExc_TypeError, "%d arguments expected, not %zd",
                          static_cast<int>(sizeof...(A)), n);
    return with(args, std::index_sequence_for<A...>{});
  }
  static void bind(void *to) { address = reinterpret_cast<R (*)(A...)>(to); }
};

struct Entry {
  const char *name;
  PyObject *(*call)(PyObject *, PyObject *const *, Py_ssize_t);
  void (*bind)(void *);
};
#define ENTRY(f) {#f, Call<&f>::call, Call<&f>::bind}
const Entry entries[] = {
    ENTRY(mha_qk_norm_rope_fwd),  ENTRY(mha_qk_norm_rope_bwd_workspace_size),
    ENTRY(mha_qk_norm_rope_bwd),  ENTRY(mha_paged_append),
    ENTRY(mha_paged_append_at),   ENTRY(mha_paged_workspace_size),
    ENTRY(mha_paged_fwd),         ENTRY(mha_paged_tree_fwd),
    ENTRY(mha_paged_path),        ENTRY(mha_paged_reserve_workspace_size),
    ENTRY(mha_paged_reserve),     ENTRY(mha_paged_copy),
    ENTRY(mha_paged_compact),
};
constexpr size_t kEntries = sizeof(entries) / sizeof(entries[0]);

// bind(name, address of that entry point)
PyObject *bind(PyObject *, PyObject *args) {
  const char *name;
  PyObject *address;
  if (!PyArg_ParseTuple(args, "sO", &name, &address)) return nullptr;
  void *to = PyLong_AsVoidPtr(address);
  if (PyErr_Occurred()) return nullptr;
  for (const Entry &e : entries)
    if (std::strcmp(e.name, name) == 0) {
      e.bind(to);
      Py_RETURN_NONE;
    }
  return PyErr_Format(PyExc_KeyError, "no entry point %s", name);
}

// refuse_with(at): the Python form of `at`
PyObject *refuse_with(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XSETREF(plain_at, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[kEntries + 4] = {
    {"at", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(at_checked)), METH_FASTCALL,
     "at(name, tensor, shape, dtype, device): the checked tensor's address"},
    {"bind", bind, METH_VARARGS, "bind(name, address) of an entry point"},
    {"refuse_with", refuse_with, METH_O, "the Python form of at()"},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mha_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mha_binding() {
  for (size_t i = 0; i < kEntries; ++i)
    methods[3 + i] = {entries[i].name,
                      reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entries[i].call)),
                      METH_FASTCALL, nullptr};
  return PyModule_Create(&module);
}

// The inner part of the Python binding of include/mha_paged.h: a tensor's checks, and the
// calls.  A step of generation makes some calls of a few microseconds each, with ten tensors
// to a call; in Python a tensor's checks take 0.35 us and a call through ctypes 2 us, here
// 0.07 and 0.2.
//
// The calls of a step whose results the caller brings along are made here from their
// tensors on (append, attend, copy, compact, reserve; an append 7.2 -> 3.8 us of the host's
// time, 2.7 of them the launch); what does not look right goes back to Python, which does the
// same and says what is wrong.
//
// Entry points come by address (bind), so that there is one libmha.so; what a function is
// given it takes from the header's declaration.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <initializer_list>
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

// ---- whole calls -------------------------------------------------------------------
PyObject *current_stream;  // handle of the current stream, by the device's number

// The arguments of one call; `ok` is false once one of them is not what the call takes.
struct Given {
  bool ok = true;
  int64_t dev = -1;
  at::ScalarType dtype = at::kFloat;

  const at::Tensor *tensor(PyObject *o, int64_t dims) {
    if (ok && THPVariable_Check(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      if (t.layout() == at::kStrided && t.dim() == dims) return &t;
    }
    ok = false;
    return nullptr;
  }
  // the tensor that tells the call's device and type
  void leads(const at::Tensor *t) {
    if (t == nullptr) return;
    dev = t->get_device();
    dtype = t->scalar_type();
    ok = ok && dev >= 0 && (dtype == at::kFloat || dtype == at::kBFloat16);
  }
  int type() const { return dtype == at::kBFloat16 ? MHA_DTYPE_BF16 : MHA_DTYPE_F32; }
  // the address of a contiguous tensor of that shape and type; nullptr of None
  void *at(PyObject *o, std::initializer_list<int64_t> shape, at::ScalarType type) {
    if (!ok || o == Py_None) return nullptr;
    const at::Tensor *t = tensor(o, static_cast<int64_t>(shape.size()));
    if (t == nullptr) return nullptr;
    ok = t->scalar_type() == type && t->get_device() == dev && t->is_contiguous();
    int64_t i = 0;
    for (const int64_t n : shape) ok = ok && t->size(i++) == n;
    return ok ? t->data_ptr() : nullptr;
  }
  int32_t *ints(PyObject *o, std::initializer_list<int64_t> shape) {
    return static_cast<int32_t *>(at(o, shape, at::kInt));
  }
  int count(int64_t n) {
    ok = ok && n <= INT_MAX;
    return static_cast<int>(n);
  }
  int number(PyObject *o) { return from<int>(o); }
  int layout(PyObject *o) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s != nullptr && std::strcmp(s, "bshd") == 0) return MHA_LAYOUT_BSHD;
    if (s == nullptr || std::strcmp(s, "bhsd") != 0) ok = false;
    return MHA_LAYOUT_BHSD;
  }
  // bytes of a workspace
  size_t scratch(PyObject *o, void **p) {
    if (!ok || !THPVariable_Check(o)) {
      ok = false;
      return 0;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    ok = t.layout() == at::kStrided && t.get_device() == dev && t.is_contiguous();
    if (!ok) return 0;
    *p = t.data_ptr();
    return static_cast<size_t>(t.nbytes());
  }
  void *stream(PyObject *o) {
    ok = ok && !PyErr_Occurred();
    if (!ok) return nullptr;
    PyObject *handle = nullptr;
    if (o == Py_None && current_stream != nullptr) {
      PyObject *number = PyLong_FromLongLong(dev);
      handle = number != nullptr ? PyObject_CallOneArg(current_stream, number) : nullptr;
      Py_XDECREF(number);
    } else if (PyLong_Check(o)) {
      handle = Py_NewRef(o);
    } else if (o != Py_None) {
      handle = PyObject_GetAttrString(o, "cuda_stream");
    }
    void *p = handle != nullptr ? PyLong_AsVoidPtr(handle) : nullptr;
    ok = handle != nullptr && !PyErr_Occurred();
    Py_XDECREF(handle);
    return p;
  }
};

// The status of the call that `make` returns, or None: it is to be made in Python.
template <typename Make>
PyObject *whole(Make make) {
  try {
    Given g;
    const auto call = make(g);
    if (g.ok && !PyErr_Occurred()) {
      int status;
      Py_BEGIN_ALLOW_THREADS;
      status = call();
      Py_END_ALLOW_THREADS;
      return PyLong_FromLong(status);
    }
  } catch (...) {  // (a tensor without memory, for instance)
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}
bool counted(Py_ssize_t n, Py_ssize_t want) {
  if (n != want)
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", want, n);
  return n == want;
}

// append(at, q, k, v, k_cache, v_cache, q_out, positions, q_starts, kv_lengths, block_table,
//        q_weight, k_weight, inv_freq, layout, interleaved, eps, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!counted(n, 18)) return nullptr;
  return whole([&](Given &g) {
    const bool at = a[0] == Py_True;
    const at::Tensor *k = g.tensor(a[2], 3), *cache = g.tensor(a[4], 4), *table = g.tensor(a[10], 2);
    const at::Tensor *q = a[1] == Py_None ? nullptr : g.tensor(a[1], 3);
    const at::Tensor *freq = a[13] == Py_None ? nullptr : g.tensor(a[13], 1);
    g.leads(k);
    const int lay = g.layout(a[14]);
    g.ok = g.ok && (a[1] == Py_None) == (a[6] == Py_None);
    int T = 0, Hkv = 0, d = 0, H = 0, pages = 0, page = 0, B = 0, width = 0, rotary = 0;
    if (g.ok) {
      T = g.count(k->size(0));
      Hkv = g.count(k->size(1));
      d = g.count(k->size(2));
      H = q != nullptr ? g.count(q->size(1)) : 0;
      pages = g.count(cache->size(0));
      page = g.count(cache->size(lay == MHA_LAYOUT_BSHD ? 1 : 2));
      B = g.count(table->size(0));
      width = g.count(table->size(1));
      rotary = freq != nullptr ? g.count(2 * freq->numel()) : 0;
    }
    const bool rows_first = lay == MHA_LAYOUT_BSHD;
    const auto cell = {int64_t{pages}, int64_t{rows_first ? page : Hkv}, int64_t{rows_first ? Hkv : page},
                       int64_t{d}};
    void *const qp = g.at(a[1], {T, H, d}, g.dtype), *const kp = g.at(a[2], {T, Hkv, d}, g.dtype),
               *const vp = g.at(a[3], {T, Hkv, d}, g.dtype),
               *const op = g.at(a[6], {T, H, d}, g.dtype), *const kc = g.at(a[4], cell, g.dtype),
               *const vc = g.at(a[5], cell, g.dtype), *const qw = g.at(a[11], {d}, g.dtype),
               *const kw = g.at(a[12], {d}, g.dtype);
    const float *fp = static_cast<float *>(g.at(a[13], {rotary / 2}, at::kFloat));
    const int32_t *pos = at ? g.ints(a[7], {T}) : nullptr, *qs = g.ints(a[8], {int64_t{B} + 1}),
                  *lens = g.ints(a[9], {B}), *tab = g.ints(a[10], {B, width});
    const int style = PyObject_IsTrue(a[15]) ? 1 : 0, type = g.type();
    const float eps = from<float>(a[16]);
    void *const stream = g.stream(a[17]);
    return [=]() {
      return at ? Call<&mha_paged_append_at>::address(qp, kp, vp, op, kc, vc, qw, kw, fp, pos, qs, lens,
                                                      tab, B, T, H, Hkv, d, pages, page, width, rotary,
                                                      lay, style, eps, type, stream)
                : Call<&mha_paged_append>::address(qp, kp, vp, op, kc, vc, qw, kw, fp, qs, lens, tab, B,
                                                   T, H, Hkv, d, pages, page, width, rotary, lay, style,
                                                   eps, type, stream);
    };
  });
}

// attend(q, k_cache, v_cache, out, tree_mask or None, q_starts, kv_lengths, block_table, max_q,
//        layout, mask_kind, scale, workspace, stream)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!counted(n, 14)) return nullptr;
  return whole([&](Given &g) {
    const at::Tensor *q = g.tensor(a[0], 3), *cache = g.tensor(a[1], 4), *table = g.tensor(a[7], 2);
    const at::Tensor *tree = a[4] == Py_None ? nullptr : g.tensor(a[4], 2);
    g.leads(q);
    const int lay = g.layout(a[9]);
    const bool rows_first = lay == MHA_LAYOUT_BSHD;
    int T = 0, H = 0, d = 0, Hkv = 0, pages = 0, page = 0, B = 0, width = 0, words = 0;
    if (g.ok) {
      T = g.count(q->size(0));
      H = g.count(q->size(1));
      d = g.count(q->size(2));
      pages = g.count(cache->size(0));
      page = g.count(cache->size(rows_first ? 1 : 2));
      Hkv = g.count(cache->size(rows_first ? 2 : 1));
      B = g.count(table->size(0));
      width = g.count(table->size(1));
      words = tree != nullptr ? g.count(tree->size(1)) : 1;
      g.ok = g.ok && words >= 1 && a[3] != Py_None;
    }
    const auto cell = {int64_t{pages}, int64_t{rows_first ? page : Hkv}, int64_t{rows_first ? Hkv : page},
                       int64_t{d}};
    void *const qp = g.at(a[0], {T, H, d}, g.dtype), *const kc = g.at(a[1], cell, g.dtype),
               *const vc = g.at(a[2], cell, g.dtype), *const op = g.at(a[3], {T, H, d}, g.dtype);
    const int32_t *mask = g.ints(a[4], {T, words}), *qs = g.ints(a[5], {int64_t{B} + 1}),
                  *lens = g.ints(a[6], {B}), *tab = g.ints(a[7], {B, width});
    const int max_q = g.number(a[8]), kind = g.number(a[10]), type = g.type();
    const float scale = a[11] == Py_None ? static_cast<float>(std::pow(static_cast<double>(d), -0.5))
                                         : from<float>(a[11]);
    void *ws = nullptr;
    const size_t bytes = g.scratch(a[12], &ws);
    void *const stream = g.stream(a[13]);
    const bool of_tree = a[4] != Py_None;
    return [=]() {
      return of_tree ? Call<&mha_paged_tree_fwd>::address(qp, kc, vc, op, mask, qs, lens, tab, B, T, H,
                                                          Hkv, d, max_q, pages, page, width, words, lay,
                                                          scale, type, ws, bytes, stream)
                     : Call<&mha_paged_fwd>::address(qp, kc, vc, op, qs, lens, tab, B, T, H, Hkv, d,
                                                     max_q, pages, page, width, lay, kind, scale, type,
                                                     ws, bytes, stream);
    };
  });
}

// Layers, and one layer's sizes, of caches with or without a dimension of layers in front.
struct Stack {
  int layers = 0, pages = 0, a = 0, b = 0, d = 0;
  Stack(Given &g, PyObject *o) {
    const bool stacked = THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 5;
    const at::Tensor *t = g.tensor(o, stacked ? 5 : 4);
    g.leads(t);
    if (!g.ok) return;
    const int first = stacked ? 1 : 0;
    layers = stacked ? g.count(t->size(0)) : 1;
    pages = g.count(t->size(first));
    a = g.count(t->size(first + 1));
    b = g.count(t->size(first + 2));
    d = g.count(t->size(first + 3));
  }
  void *at(Given &g, PyObject *o) const {
    if (THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 5)
      return g.at(o, {layers, pages, a, b, d}, g.dtype);
    return g.at(o, {pages, a, b, d}, g.dtype);
  }
};
// (both caches have the same number of dimensions)
bool alike(PyObject *k, PyObject *v) {
  return THPVariable_Check(k) && THPVariable_Check(v) &&
         THPVariable_Unpack(k).dim() == THPVariable_Unpack(v).dim();
}

// copy(k_cache, v_cache, moves, stream)
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!counted(n, 4)) return nullptr;
  return whole([&](Given &g) {
    g.ok = alike(a[0], a[1]);
    const Stack s(g, a[0]);
    const at::Tensor *moves = g.tensor(a[2], 2);
    const int pairs = g.ok ? g.count(moves->size(0)) : 0;
    void *const kc = s.at(g, a[0]), *const vc = s.at(g, a[1]);
    const int32_t *m = g.ints(a[2], {pairs, 2});
    const bool first = s.a >= 16 && (s.a & (s.a - 1)) == 0;
    const int page = first ? s.a : s.b, heads = first ? s.b : s.a, type = g.type();
    void *const stream = g.stream(a[3]);
    return [=]() {
      return Call<&mha_paged_copy>::address(kc, vc, m, pairs, s.layers, heads, s.d, s.pages, page, type,
                                            stream);
    };
  });
}

// compact(k_cache, v_cache, keep, keep_counts, lengths_out, starts, kv_lengths, block_table,
//         src_table, layout, stream)
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!counted(n, 11)) return nullptr;
  return whole([&](Given &g) {
    g.ok = alike(a[0], a[1]) && a[4] != Py_None;
    const Stack s(g, a[0]);
    const at::Tensor *keep = g.tensor(a[2], 2), *table = g.tensor(a[7], 2);
    const int lay = g.layout(a[9]);
    const int B = g.ok ? g.count(keep->size(0)) : 0, most = g.ok ? g.count(keep->size(1)) : 0;
    const int width = g.ok ? g.count(table->size(1)) : 0;
    void *const kc = s.at(g, a[0]), *const vc = s.at(g, a[1]);
    const int32_t *kp = g.ints(a[2], {B, most}), *counts = g.ints(a[3], {B}),
                  *starts = g.ints(a[5], {B}), *lens = g.ints(a[6], {B}),
                  *src = g.ints(a[8], {B, width}), *tab = g.ints(a[7], {B, width});
    int32_t *const out = g.ints(a[4], {B});
    const bool rows_first = lay == MHA_LAYOUT_BSHD;
    const int page = rows_first ? s.a : s.b, heads = rows_first ? s.b : s.a, type = g.type();
    void *const stream = g.stream(a[10]);
    return [=]() {
      return Call<&mha_paged_compact>::address(kc, vc, out, kp, counts, starts, lens, src, tab, B,
                                               s.layers, heads, s.d, s.pages, page, width, most, lay,
                                               type, stream);
    };
  });
}

// reserve(block_table, kv_lengths, new_lengths, parents, refs, table_out, lengths_out, refs_out,
//         moves, counts, page_size, workspace, stream)
PyObject *reserve(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (!counted(n, 13)) return nullptr;
  return whole([&](Given &g) {
    const at::Tensor *table = g.tensor(a[0], 2), *news = g.tensor(a[2], 1), *refs = g.tensor(a[4], 1);
    int B_old = 0, width = 0, B = 0, pages = 0;
    for (int i = 5; i < 10; ++i) g.ok = g.ok && a[i] != Py_None;
    if (g.ok) {
      g.dev = table->get_device();
      g.ok = g.dev >= 0;
      B_old = g.count(table->size(0));
      width = g.count(table->size(1));
      B = g.count(news->size(0));
      pages = g.count(refs->size(0));
    }
    const int32_t *tab = g.ints(a[0], {B_old, width}), *lens = g.ints(a[1], {B_old}),
                  *want = g.ints(a[2], {B}), *parents = g.ints(a[3], {B}), *held = g.ints(a[4], {pages});
    int32_t *const out = g.ints(a[5], {B, width}), *const lens_out = g.ints(a[6], {B}),
                  *const held_out = g.ints(a[7], {pages}), *const moves = g.ints(a[8], {B, 2}),
                  *const counts = g.ints(a[9], {2});
    const int page = g.number(a[10]);
    void *ws = nullptr;
    const size_t bytes = g.scratch(a[11], &ws);
    void *const stream = g.stream(a[12]);
    return [=]() {
      return Call<&mha_paged_reserve>::address(tab, lens, want, parents, held, out, lens_out, held_out,
                                               moves, counts, B_old, B, pages, page, width, ws, bytes,
                                               stream);
    };
  });
}

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

// stream_with(f): what tells the current stream's handle
PyObject *stream_with(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XSETREF(current_stream, f);
  Py_RETURN_NONE;
}

template <PyObject *(*kCall)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef fast(const char *name, const char *doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kCall)), METH_FASTCALL, doc};
}
constexpr size_t kOthers = 9;
PyMethodDef methods[kEntries + kOthers + 1] = {
    fast<at_checked>("at", "at(name, tensor, shape, dtype, device): the checked tensor's address"),
    {"bind", bind, METH_VARARGS, "bind(name, address) of an entry point"},
    {"refuse_with", refuse_with, METH_O, "the Python form of at()"},
    {"stream_with", stream_with, METH_O, "what tells a device's current stream"},
    fast<append>("append", "status of mha_paged_append or mha_paged_append_at, or None"),
    fast<attend>("attend", "status of mha_paged_fwd or mha_paged_tree_fwd, or None"),
    fast<copy>("copy", "status of mha_paged_copy, or None"),
    fast<compact>("compact", "status of mha_paged_compact, or None"),
    fast<reserve>("reserve", "status of mha_paged_reserve, or None"),
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mha_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mha_binding() {
  for (size_t i = 0; i < kEntries; ++i)
    methods[kOthers + i] = {entries[i].name,
                      reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entries[i].call)),
                      METH_FASTCALL, nullptr};
  return PyModule_Create(&module);
}

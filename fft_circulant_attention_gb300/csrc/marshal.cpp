// Native marshalling of the operator plans' Python calls (attention, layer
// norm, clipping): checks the tensors, allocates the outputs that were not
// given and calls the C interface.  In Python these steps take longer than
// the kernels of a small call (82 tokens in 3 sequences, 2 heads of 32, GB300:
// 16 us a call from Python, 7.2 us from here, of which the C call takes 5.2;
// layer norm of 256 short rows 15 us and, by the machine, 6.4 to 9; clipping 133
// tensors 97 us, all of it the host's, and 88 us, the kernels' time).
//
// make(...) -> a handle that holds a plan's shape and entry points; the calls
// return their outputs, or the status of a failed C call as an int.  Tensors
// that do not fit raise ValueError.
#include <Python.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

namespace {

// The C interface (include/cat.h), by address.
using AttnFwd = int (*)(void*, const void*, const void*, const void*, void*, float*, const int*,
                        int, int, long long, long long, long long);
using AttnBwd = int (*)(void*, const void*, const void*, const void*, const void*, const float*,
                        const void*, void*, void*, void*, const int*, int, int, long long,
                        long long, long long, long long, long long, long long);
using NormFwd = int (*)(void*, const void*, const void*, const void*, void*, float*, float*, int);
using NormBwd = int (*)(void*, const void*, const void*, const float*, const float*, const void*,
                        void*, void*, void*, int);
using ClipNorm = int (*)(void*, void* const*, float*);
using ClipScale = int (*)(void*, void* const*, void* const*, float, float*);

struct Handle {
  void* fn[2];
  void* plan;
  int64_t dims[3];
  at::ScalarType type;
  at::Device device{at::kCPU};
  std::vector<int64_t> sizes;
  std::vector<at::ScalarType> types;
};

const char* kName = "cat_operator_plan";

void free_handle(PyObject* o) { delete static_cast<Handle*>(PyCapsule_GetPointer(o, kName)); }

Handle* handle_of(PyObject* o) {
  if (!PyCapsule_IsValid(o, kName)) {
    PyErr_SetString(PyExc_ValueError, "the plan is closed");
    return nullptr;
  }
  return static_cast<Handle*>(PyCapsule_GetPointer(o, kName));
}

at::ScalarType type_of(long code) { return code == 1 ? at::kBFloat16 : at::kFloat; }

bool bad(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s %s", name, what);
  return false;
}

// The tensor behind `o`, on the plan's device and of `type`.
const at::Tensor* tensor(const Handle& p, PyObject* o, const char* name, at::ScalarType type) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.device() != p.device) {
    bad(name, "is not on the plan's device");
    return nullptr;
  }
  if (t.scalar_type() != type) {
    bad(name, "does not have the plan's dtype (statistics: float32, offsets: int32)");
    return nullptr;
  }
  return &t;
}

const at::Tensor* shaped(const Handle& p, PyObject* o, const char* name, at::ScalarType type,
                         at::IntArrayRef shape) {
  const at::Tensor* t = tensor(p, o, name, type);
  if (!t) return nullptr;
  if (t->sizes() != shape) {
    bad(name, "does not have the shape the plan and the other tensors give");
    return nullptr;
  }
  return t;
}

const at::Tensor* dense(const Handle& p, PyObject* o, const char* name, at::ScalarType type,
                        at::IntArrayRef shape) {
  const at::Tensor* t = shaped(p, o, name, type, shape);
  if (t && !t->is_contiguous()) {
    bad(name, "must be contiguous");
    return nullptr;
  }
  return t;
}

// A [T, heads, dh] operand with its row stride.
const at::Tensor* rows(const Handle& p, PyObject* o, const char* name, at::IntArrayRef shape,
                       long long* ld) {
  const at::Tensor* t = shaped(p, o, name, p.type, shape);
  if (!t) return nullptr;
  const auto st = t->strides();
  if (t->numel() && ((shape[2] > 1 && st[2] != 1) || (shape[1] > 1 && st[1] != shape[2]))) {
    bad(name, "must have its heads contiguous within each token row");
    return nullptr;
  }
  // A single row has no stride of its own (any may be reported).
  *ld = shape[0] > 1 ? st[0] : shape[1] * shape[2];
  return t;
}

// cu_seqlens [S + 1] over T rows, both within an int.
bool offsets(const at::Tensor& cu, int64_t T) {
  if (cu.dim() != 1 || cu.size(0) < 1 || !cu.is_contiguous())
    return bad("cu_seqlens", "must hold S + 1 contiguous entries");
  if (T > INT32_MAX || cu.size(0) > INT32_MAX) return bad("Q or cu_seqlens", "has too many rows");
  return true;
}

at::Tensor fresh(const Handle& p, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(p.device));
}

// The given output, or a new one.
bool output(const Handle& p, PyObject* o, const char* name, at::ScalarType type,
            at::IntArrayRef shape, at::Tensor* out) {
  if (o == Py_None) {
    *out = fresh(p, shape, type);
    return true;
  }
  const at::Tensor* t = dense(p, o, name, type, shape);
  if (t) *out = *t;
  return t != nullptr;
}
bool output_rows(const Handle& p, PyObject* o, const char* name, at::IntArrayRef shape,
                 at::Tensor* out, long long* ld) {
  if (o == Py_None) {
    *out = fresh(p, shape, p.type);
    *ld = shape[1] * shape[2];
    return true;
  }
  const at::Tensor* t = rows(p, o, name, shape, ld);
  if (t) *out = *t;
  return t != nullptr;
}

PyObject* result(int status, std::initializer_list<at::Tensor*> outs) {
  if (status) return PyLong_FromLong(status);
  PyObject* r = PyTuple_New((Py_ssize_t)outs.size());
  Py_ssize_t i = 0;
  for (at::Tensor* t : outs) {
    PyObject* w = r ? THPVariable_Wrap(*t) : nullptr;
    if (!w) {
      Py_XDECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, w);
  }
  return r;
}

// A call of the C interface, other Python threads running meanwhile (it waits
// where the launch queue is full).
template <typename F, typename... A>
int call(void* fn, A... args) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = reinterpret_cast<F>(fn)(args...);
  Py_END_ALLOW_THREADS
  return st;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// C++ exceptions (an allocation that failed) end as Python ones.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// make(fn0, fn1, plan, d0, d1, d2, dtype, device index)
PyObject* make(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    Handle* p = new Handle();
    for (int i = 0; i < 2; ++i) p->fn[i] = PyLong_AsVoidPtr(a[i]);
    p->plan = PyLong_AsVoidPtr(a[2]);
    for (int i = 0; i < 3; ++i) p->dims[i] = PyLong_AsLongLong(a[3 + i]);
    p->type = type_of(PyLong_AsLong(a[6]));
    p->device = at::Device(at::kCUDA, (c10::DeviceIndex)PyLong_AsLong(a[7]));
    if (PyErr_Occurred()) {
      delete p;
      return nullptr;
    }
    return PyCapsule_New(p, kName, free_handle);
  });
}

// set_list(handle, sizes, dtype codes): a clipping plan's tensors.
PyObject* set_list(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 3)) return nullptr;
  return guarded([&]() -> PyObject* {
    Handle* p = handle_of(a[0]);
    if (!p) return nullptr;
    const Py_ssize_t k = PyList_Size(a[1]);
    if (k < 0 || PyList_Size(a[2]) != k) {
      if (!PyErr_Occurred()) bad("sizes and dtypes", "differ in number");
      return nullptr;
    }
    for (Py_ssize_t i = 0; i < k; ++i) {
      p->sizes.push_back(PyLong_AsLongLong(PyList_GET_ITEM(a[1], i)));
      p->types.push_back(type_of(PyLong_AsLong(PyList_GET_ITEM(a[2], i))));
    }
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  });
}

// attn_forward(handle, Q, K, V, cu_seqlens, O, lse)
PyObject* attn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Handle* p = handle_of(a[0]);
    if (!p) return nullptr;
    const at::Tensor* q0 = tensor(*p, a[1], "Q", p->type);
    if (!q0) return nullptr;
    const int64_t T = q0->dim() ? q0->size(0) : 0, hq = p->dims[0], hkv = p->dims[1],
                  dh = p->dims[2];
    long long ld[3];
    const at::Tensor* q = rows(*p, a[1], "Q", {T, hq, dh}, ld);
    const at::Tensor* k = q ? rows(*p, a[2], "K", {T, hkv, dh}, ld + 1) : nullptr;
    const at::Tensor* v = k ? rows(*p, a[3], "V", {T, hkv, dh}, ld + 2) : nullptr;
    const at::Tensor* cu = v ? tensor(*p, a[4], "cu_seqlens", at::kInt) : nullptr;
    if (!cu) return nullptr;
    if (!offsets(*cu, T)) return nullptr;
    at::Tensor o, lse;
    if (!output(*p, a[5], "O", p->type, {T, hq, dh}, &o) ||
        !output(*p, a[6], "lse", at::kFloat, {hq, T}, &lse))
      return nullptr;
    const int st = call<AttnFwd>(
        p->fn[0], p->plan, q->data_ptr(), k->data_ptr(), v->data_ptr(), o.data_ptr(),
        static_cast<float*>(lse.data_ptr()), static_cast<const int*>(cu->data_ptr()), (int)T,
        (int)cu->size(0) - 1, ld[0], ld[1], ld[2]);
    return result(st, {&o, &lse});
  });
}

// attn_backward(handle, Q, K, V, O, lse, dO, cu_seqlens, dQ, dK, dV)
PyObject* attn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Handle* p = handle_of(a[0]);
    if (!p) return nullptr;
    const at::Tensor* q0 = tensor(*p, a[1], "Q", p->type);
    if (!q0) return nullptr;
    const int64_t T = q0->dim() ? q0->size(0) : 0, hq = p->dims[0], hkv = p->dims[1],
                  dh = p->dims[2];
    long long ld[6];
    const at::Tensor* q = rows(*p, a[1], "Q", {T, hq, dh}, ld);
    const at::Tensor* k = q ? rows(*p, a[2], "K", {T, hkv, dh}, ld + 1) : nullptr;
    const at::Tensor* v = k ? rows(*p, a[3], "V", {T, hkv, dh}, ld + 2) : nullptr;
    const at::Tensor* o = v ? dense(*p, a[4], "O", p->type, {T, hq, dh}) : nullptr;
    const at::Tensor* lse = o ? dense(*p, a[5], "lse", at::kFloat, {hq, T}) : nullptr;
    const at::Tensor* g = lse ? dense(*p, a[6], "dO", p->type, {T, hq, dh}) : nullptr;
    const at::Tensor* cu = g ? tensor(*p, a[7], "cu_seqlens", at::kInt) : nullptr;
    if (!cu) return nullptr;
    if (!offsets(*cu, T)) return nullptr;
    at::Tensor dq, dk, dv;
    if (!output_rows(*p, a[8], "dQ", {T, hq, dh}, &dq, ld + 3) ||
        !output_rows(*p, a[9], "dK", {T, hkv, dh}, &dk, ld + 4) ||
        !output_rows(*p, a[10], "dV", {T, hkv, dh}, &dv, ld + 5))
      return nullptr;
    const int st = call<AttnBwd>(
        p->fn[1], p->plan, q->data_ptr(), k->data_ptr(), v->data_ptr(), o->data_ptr(),
        static_cast<const float*>(lse->data_ptr()), g->data_ptr(), dq.data_ptr(), dk.data_ptr(),
        dv.data_ptr(), static_cast<const int*>(cu->data_ptr()), (int)T, (int)cu->size(0) - 1,
        ld[0], ld[1], ld[2], ld[3], ld[4], ld[5]);
    return result(st, {&dq, &dk, &dv});
  });
}

// X and its rows; gamma, beta or null pointers.
const at::Tensor* norm_input(const Handle& p, PyObject* o, int64_t* nrows) {
  const at::Tensor* x = tensor(p, o, "X", p.type);
  if (!x) return nullptr;
  if (x->dim() < 1 || x->size(-1) != p.dims[0]) {
    bad("X", "does not have the plan's width as its last dimension");
    return nullptr;
  }
  if (!x->is_contiguous()) {
    bad("X", "must be contiguous");
    return nullptr;
  }
  *nrows = x->numel() / p.dims[0];
  return x;
}
bool weight(const Handle& p, PyObject* o, const char* name, const void** ptr) {
  *ptr = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = dense(p, o, name, p.type, {p.dims[0]});
  if (t) *ptr = t->data_ptr();
  return t != nullptr;
}

// ln_forward(handle, X, gamma, beta, Y, mean, rstd)
PyObject* ln_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Handle* p = handle_of(a[0]);
    int64_t nrows = 0;
    const at::Tensor* x = p ? norm_input(*p, a[1], &nrows) : nullptr;
    const void *w, *b;
    if (!x || !weight(*p, a[2], "gamma", &w) || !weight(*p, a[3], "beta", &b)) return nullptr;
    const auto lead = x->sizes().slice(0, x->dim() - 1);
    at::Tensor y, mean, rstd;
    if (!output(*p, a[4], "Y", p->type, x->sizes(), &y) ||
        !output(*p, a[5], "mean", at::kFloat, lead, &mean) ||
        !output(*p, a[6], "rstd", at::kFloat, lead, &rstd))
      return nullptr;
    if (nrows > INT32_MAX) return bad("X", "has too many rows"), nullptr;
    const int st = call<NormFwd>(
        p->fn[0], p->plan, x->data_ptr(), w, b, y.data_ptr(), static_cast<float*>(mean.data_ptr()),
        static_cast<float*>(rstd.data_ptr()), (int)nrows);
    return result(st, {&y, &mean, &rstd});
  });
}

// ln_backward(handle, X, gamma, mean, rstd, dY, dX, dgamma, dbeta)
PyObject* ln_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Handle* p = handle_of(a[0]);
    int64_t nrows = 0;
    const at::Tensor* x = p ? norm_input(*p, a[1], &nrows) : nullptr;
    const void* w;
    if (!x || !weight(*p, a[2], "gamma", &w)) return nullptr;
    const auto lead = x->sizes().slice(0, x->dim() - 1);
    const at::Tensor* mean = dense(*p, a[3], "mean", at::kFloat, lead);
    const at::Tensor* rstd = mean ? dense(*p, a[4], "rstd", at::kFloat, lead) : nullptr;
    const at::Tensor* dy = rstd ? dense(*p, a[5], "dY", p->type, x->sizes()) : nullptr;
    at::Tensor dx, dg, db;
    if (!dy || !output(*p, a[6], "dX", p->type, x->sizes(), &dx) ||
        !output(*p, a[7], "dgamma", p->type, {p->dims[0]}, &dg) ||
        !output(*p, a[8], "dbeta", p->type, {p->dims[0]}, &db))
      return nullptr;
    if (nrows > INT32_MAX) return bad("X", "has too many rows"), nullptr;
    const int st = call<NormBwd>(
        p->fn[1], p->plan, x->data_ptr(), w, static_cast<const float*>(mean->data_ptr()),
        static_cast<const float*>(rstd->data_ptr()), dy->data_ptr(), dx.data_ptr(), dg.data_ptr(),
        db.data_ptr(), (int)nrows);
    return result(st, {&dx, &dg, &db});
  });
}

// A clipping plan's list of tensors: their addresses, and the tensors themselves
// for as long as it lives (the argument may be a generator that made them, or a
// list that another thread changes while the C call runs).
struct List {
  PyObject* seq = nullptr;
  std::vector<void*> ptrs;
  List() = default;
  List(const List&) = delete;
  List& operator=(const List&) = delete;
  ~List() { Py_XDECREF(seq); }
};
bool list_of(const Handle& p, PyObject* o, const char* name, List* list) {
  list->seq = PySequence_Tuple(o);
  if (!list->seq) return false;
  PyObject* seq = list->seq;
  std::vector<void*>* ptrs = &list->ptrs;
  const Py_ssize_t n = PyTuple_GET_SIZE(seq);
  bool ok = n == (Py_ssize_t)p.sizes.size();
  if (!ok) bad(name, "does not have as many tensors as the plan");
  ptrs->resize(p.sizes.size());
  for (Py_ssize_t i = 0; ok && i < n; ++i) {
    PyObject* e = PyTuple_GET_ITEM(seq, i);
    if (!THPVariable_Check(e)) {
      ok = bad(name, "must hold tensors");
      break;
    }
    const at::Tensor& t = THPVariable_Unpack(e);
    if (t.scalar_type() != p.types[i] || t.numel() != p.sizes[i] || !t.is_contiguous() ||
        t.device() != p.device)
      ok = bad(name, "must be contiguous, of the plan's sizes, dtypes and device");
    else
      (*ptrs)[i] = t.data_ptr();
  }
  return ok;
}

// clip(handle, grads, outs or None, max_norm or None, norm): max_norm None is
// the norm alone.
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Handle* p = handle_of(a[0]);
    if (!p) return nullptr;
    List in, out;
    if (!list_of(*p, a[1], "grads", &in)) return nullptr;
    const bool apart = a[2] != Py_None && a[2] != a[1];
    if (apart && !list_of(*p, a[2], "out", &out)) return nullptr;
    float most = 0.f;
    if (a[3] != Py_None) {
      most = (float)PyFloat_AsDouble(a[3]);
      if (PyErr_Occurred()) return nullptr;
    }
    at::Tensor norm;
    if (!output(*p, a[4], "norm", at::kFloat, {}, &norm)) return nullptr;
    float* to = static_cast<float*>(norm.data_ptr());
    const int st =
        a[3] == Py_None
            ? call<ClipNorm>(p->fn[0], p->plan, in.ptrs.data(), to)
            : call<ClipScale>(p->fn[1], p->plan, in.ptrs.data(), (apart ? out : in).ptrs.data(),
                              most, to);
    return st ? PyLong_FromLong(st) : THPVariable_Wrap(norm);
  });
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(make),       FAST(set_list),   FAST(attn_forward),
                          FAST(attn_backward), FAST(ln_forward), FAST(ln_backward),
                          FAST(clip),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }

// Call layer of the operators around the decode step: checks a call's tensors
// and hands their addresses to libseer's C entry points, without the
// interpreter in between (a call runs for a few microseconds; checking ten
// tensors in Python costs twice that).
//
// Each function takes the arguments of its namesake in seer.py, all of them, in
// order, and returns the C entry point's status, or -1 when an argument is
// not as it must be or not understood: the caller then runs its named checks, which say what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "seer.h"

namespace {

// C entry points of the library that seer.py has loaded (set by bind)
struct Entry {
  const char* name;
  void* fn;
};
Entry g_entries[] = {{"seer_page_plan", nullptr},
                     {"seer_page_release", nullptr},
                     {"seer_qk_norm_rope", nullptr},
                     {"seer_qk_norm_rope_backward", nullptr},
                     {"seer_dense_decode", nullptr}};
template <typename F>
F* entry(int i, F*) {
  return reinterpret_cast<F*>(g_entries[i].fn);
}

constexpr auto kI32 = at::ScalarType::Int;

// The tensors of one call.  `ok` turns false at the first that does not fit; the address is then not used.
struct Call {
  bool ok = true;
  int dev = -1;

  const at::Tensor* get(PyObject* o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) {
      ok = false;
      return nullptr;
    }
    if (dev < 0) {
      dev = t.get_device();
      if (dev != c10::cuda::current_device()) ok = false;
    } else if (t.get_device() != dev) {
      ok = false;
    }
    return &t;
  }
  // contiguous, of this shape and type
  void* dense(PyObject* o, at::IntArrayRef shape, at::ScalarType type) {
    const at::Tensor* t = get(o);
    if (!t || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* dense_or_null(PyObject* o, at::IntArrayRef shape, at::ScalarType type) {
    return o == Py_None ? nullptr : dense(o, shape, type);
  }
  int32_t* err(PyObject* o) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = get(o);
    if (!t || t->scalar_type() != kI32 || !t->is_contiguous() || t->numel() < 1) {
      ok = false;
      return nullptr;
    }
    return static_cast<int32_t*>(t->data_ptr());
  }
  // [T, heads, d] view with unit-stride d; None: absent
  const seer_rows_t* rows(PyObject* o, int64_t T, int64_t heads, int64_t d, at::ScalarType type, seer_rows_t* r) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = get(o);
    if (!t || t->scalar_type() != type || t->dim() != 3 || t->size(0) != T || t->size(1) != heads || t->size(2) != d ||
        t->stride(2) != 1) {
      ok = false;
      return nullptr;
    }
    r->data = t->data_ptr();
    r->stride_t = T > 1 ? t->stride(0) : heads * d;   // a stride that is never taken may be anything
    r->stride_h = heads > 1 ? t->stride(1) : d;
    return r;
  }
  // [pages, heads, page, d] view with unit-stride d; None: absent
  const seer_pool_t* pool(PyObject* o, int64_t heads, int64_t d, at::ScalarType type, seer_pool_t* p) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = get(o);
    if (!t || t->scalar_type() != type || t->dim() != 4 || t->size(1) != heads || t->size(3) != d || t->stride(3) != 1 ||
        t->size(2) > INT32_MAX) {
      ok = false;
      return nullptr;
    }
    const int64_t page = t->size(2);
    p->data = t->data_ptr();
    p->stride_t = page > 1 ? t->stride(2) : d;
    p->stride_h = heads > 1 ? t->stride(1) : p->stride_t * page;
    p->stride_page = t->size(0) > 1 ? t->stride(0) : p->stride_h * heads;
    p->num_pages = t->size(0);
    p->page_size = (int32_t)page;
    return p;
  }
  int32_t i32(PyObject* o) {
    const long v = PyLong_Check(o) ? PyLong_AsLong(o) : (ok = false, 0);
    if (v > INT32_MAX || v < INT32_MIN || (v == -1 && PyErr_Occurred())) ok = false;   // the error: beyond 64 bits
    return (int32_t)v;
  }
  float f32(PyObject* o) {
    if (!PyFloat_Check(o) && !PyLong_Check(o)) {
      ok = false;
      return 0.f;
    }
    return (float)PyFloat_AsDouble(o);
  }
  void* stream(PyObject* o) {
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
    void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
    Py_XDECREF(s);
    if (PyErr_Occurred()) ok = false;
    return p;
  }
};

// Runs `body` (which fills in a Call and makes the C call with the interpreter's lock released).
template <typename Body>
PyObject* run(Py_ssize_t n, Py_ssize_t want, Body body) {
  long st = -1;
  if (n == want) {
    try {
      st = body();
    } catch (...) {
      st = -1;
    }
  }
  if (PyErr_Occurred()) {   // the named checks raise their own
    PyErr_Clear();
    st = -1;
  }
  return PyLong_FromLong(st);
}

template <typename F>
long unlocked(F f) {
  long st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

struct Pages {
  int64_t B = 0, width = 0, pages = 0;
  int32_t *lens, *per_request, *table, *free_list, *count;
  bool read(Call& c, PyObject* const* a) {   // seqlens, per request, block_table, free_list, free_count
    const at::Tensor *l = c.get(a[0]), *t = c.get(a[2]), *f = c.get(a[3]);
    if (!c.ok || l->dim() != 1 || t->dim() != 2 || f->dim() != 1) return false;
    B = l->size(0);
    width = t->size(1);
    pages = f->size(0);
    if (B > INT32_MAX || width > INT32_MAX || pages > INT32_MAX) return false;
    lens = static_cast<int32_t*>(c.dense(a[0], {B}, kI32));
    per_request = static_cast<int32_t*>(c.dense(a[1], {B}, kI32));
    table = static_cast<int32_t*>(c.dense(a[2], {B, width}, kI32));
    free_list = static_cast<int32_t*>(c.dense(a[3], {pages}, kI32));
    count = static_cast<int32_t*>(c.dense(a[4], {1}, kI32));
    return c.ok;
  }
};

PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 13, [&]() -> long {
    Call c;
    Pages g;
    if (!g.read(c, a + 1)) return -1;
    const int32_t page = c.i32(a[0]);
    const at::Tensor* s = c.get(a[7]);
    if (!c.ok || s->dim() != 1 || s->size(0) < 1 || s->size(0) > INT32_MAX) return -1;
    const int64_t room = s->size(0);
    auto* cu = static_cast<int32_t*>(c.dense(a[6], {g.B + 1}, kI32));
    auto* slots = static_cast<int32_t*>(c.dense(a[7], {room}, kI32));
    auto* pos = static_cast<int32_t*>(c.dense(a[8], {room}, kI32));
    auto* lo = a[9] == Py_None ? g.lens : static_cast<int32_t*>(c.dense(a[9], {g.B}, kI32));
    auto* co = a[10] == Py_None ? g.count : static_cast<int32_t*>(c.dense(a[10], {1}, kI32));
    int32_t* err = c.err(a[11]);
    void* stream = c.stream(a[12]);
    if (!c.ok) return -1;
    auto* fn = entry(0, &seer_page_plan);
    return unlocked([&] {
      return fn((int32_t)g.B, page, (int32_t)g.pages, (int32_t)g.width, (int32_t)room, g.lens, g.per_request, g.table,
                g.free_list, g.count, lo, co, cu, slots, pos, err, stream);
    });
  });
}

PyObject* page_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 10, [&]() -> long {
    Call c;
    Pages g;
    if (!g.read(c, a + 1)) return -1;
    const int32_t page = c.i32(a[0]);
    auto* lo = a[6] == Py_None ? g.lens : static_cast<int32_t*>(c.dense(a[6], {g.B}, kI32));
    auto* co = a[7] == Py_None ? g.count : static_cast<int32_t*>(c.dense(a[7], {1}, kI32));
    int32_t* err = c.err(a[8]);
    void* stream = c.stream(a[9]);
    if (!c.ok) return -1;
    auto* fn = entry(1, &seer_page_release);
    return unlocked([&] {
      return fn((int32_t)g.B, page, (int32_t)g.pages, (int32_t)g.width, g.lens, g.per_request, g.table, g.free_list,
                g.count, lo, co, err, stream);
    });
  });
}

// Shape of a norm + rotation call from its query and / or key rows.
struct Qk {
  seer_qk_t s{};
  int64_t T = 0, Hq = 0, Hkv = 0, d = 0;
  at::ScalarType type = at::ScalarType::Undefined;
  bool read(Call& c, PyObject* q, PyObject* k, PyObject* base, PyObject* rope, PyObject* eps) {
    const at::Tensor *tq = q == Py_None ? nullptr : c.get(q), *tk = k == Py_None ? nullptr : c.get(k);
    if (!c.ok || (!tq && !tk) || (tq && tq->dim() != 3) || (tk && tk->dim() != 3)) return false;
    const at::Tensor* one = tq ? tq : tk;
    type = one->scalar_type();
    T = one->size(0);
    d = one->size(2);
    Hq = one->size(1);
    Hkv = tk ? tk->size(1) : Hq;
    if (T > INT32_MAX || Hq > INT32_MAX || Hkv > INT32_MAX || d > INT32_MAX) return false;
    s.num_tokens = (int32_t)T;
    s.num_q_heads = (int32_t)Hq;
    s.num_kv_heads = (int32_t)Hkv;
    s.head_dim = (int32_t)d;
    s.rope_dim = rope == Py_None ? s.head_dim : c.i32(rope);
    s.rope_base = c.f32(base);
    s.eps = c.f32(eps);
    if (type == at::ScalarType::BFloat16) s.dtype = SEER_BF16;
    else if (type == at::ScalarType::Half) s.dtype = SEER_FP16;
    else if (type == at::ScalarType::Float) s.dtype = SEER_FP32;
    else return false;
    return c.ok;
  }
};

// q, k, positions, q_out, k_out, q_weight, k_weight, rope_base, rope_dim, eps, q_nope, k_nope, v, k_cache, v_cache,
// slot_map, num_tokens, err, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 19, [&]() -> long {
    Call c;
    Qk g;
    if (!g.read(c, a[0], a[1], a[7], a[8], a[9])) return -1;
    seer_rows_t r[7];
    seer_pool_t p[2];
    const seer_rows_t* q = c.rows(a[0], g.T, g.Hq, g.d, g.type, r);
    const seer_rows_t* k = c.rows(a[1], g.T, g.Hkv, g.d, g.type, r + 1);
    const seer_rows_t* qo = c.rows(a[3], g.T, g.Hq, g.d, g.type, r + 2);
    const seer_rows_t* ko = c.rows(a[4], g.T, g.Hkv, g.d, g.type, r + 3);
    const seer_rows_t* qn = c.rows(a[10], g.T, g.Hq, g.d, g.type, r + 4);
    const seer_rows_t* kn = c.rows(a[11], g.T, g.Hkv, g.d, g.type, r + 5);
    const seer_rows_t* v = c.rows(a[12], g.T, g.Hkv, g.d, g.type, r + 6);
    const seer_pool_t* kc = c.pool(a[13], g.Hkv, g.d, g.type, p);
    const seer_pool_t* vc = c.pool(a[14], g.Hkv, g.d, g.type, p + 1);
    const auto* pos = static_cast<int32_t*>(c.dense_or_null(a[2], {g.T}, kI32));
    const void* wq = c.dense_or_null(a[5], {g.d}, g.type);
    const void* wk = c.dense_or_null(a[6], {g.d}, g.type);
    const auto* slots = static_cast<int32_t*>(c.dense_or_null(a[15], {g.T}, kI32));
    const auto* live = static_cast<int32_t*>(c.dense_or_null(a[16], {1}, kI32));
    int32_t* err = c.err(a[17]);
    void* stream = c.stream(a[18]);
    if (!c.ok || g.T == 0 || (g.s.rope_dim > 0 && a[2] == Py_None) || ((kc || vc) && a[15] == Py_None)) return -1;
    auto* fn = entry(2, &seer_qk_norm_rope);
    return unlocked([&] { return fn(&g.s, q, k, v, wq, wk, pos, qo, ko, qn, kn, kc, vc, slots, live, err, stream); });
  });
}

// dq_out, dk_out, q, k, positions, dq, dk, workspace, q_weight, k_weight, dq_weight, dk_weight, rope_base, rope_dim, eps,
// dq_nope, dk_nope, num_tokens, stream
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 19, [&]() -> long {
    Call c;
    Qk g;
    if (!g.read(c, a[2] != Py_None ? a[2] : a[5], a[3] != Py_None ? a[3] : a[6], a[12], a[13], a[14])) return -1;
    seer_rows_t r[8];
    const seer_rows_t* zq = c.rows(a[0], g.T, g.Hq, g.d, g.type, r);
    const seer_rows_t* zk = c.rows(a[1], g.T, g.Hkv, g.d, g.type, r + 1);
    const seer_rows_t* q = c.rows(a[2], g.T, g.Hq, g.d, g.type, r + 2);
    const seer_rows_t* k = c.rows(a[3], g.T, g.Hkv, g.d, g.type, r + 3);
    const seer_rows_t* dq = c.rows(a[5], g.T, g.Hq, g.d, g.type, r + 4);
    const seer_rows_t* dk = c.rows(a[6], g.T, g.Hkv, g.d, g.type, r + 5);
    const seer_rows_t* yq = c.rows(a[15], g.T, g.Hq, g.d, g.type, r + 6);
    const seer_rows_t* yk = c.rows(a[16], g.T, g.Hkv, g.d, g.type, r + 7);
    const auto* pos = static_cast<int32_t*>(c.dense_or_null(a[4], {g.T}, kI32));
    const void* wq = c.dense_or_null(a[8], {g.d}, g.type);
    const void* wk = c.dense_or_null(a[9], {g.d}, g.type);
    auto* gq = static_cast<float*>(c.dense_or_null(a[10], {g.d}, at::ScalarType::Float));
    auto* gk = static_cast<float*>(c.dense_or_null(a[11], {g.d}, at::ScalarType::Float));
    const auto* live = static_cast<int32_t*>(c.dense_or_null(a[17], {1}, kI32));
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[7] != Py_None) {
      const at::Tensor* w = c.get(a[7]);
      if (!c.ok || w->scalar_type() != at::ScalarType::Byte || !w->is_contiguous()) return -1;
      ws = w->data_ptr();
      bytes = (size_t)w->numel();
    }
    void* stream = c.stream(a[18]);
    if (!c.ok || g.T == 0 || (g.s.rope_dim > 0 && (zq || zk) && a[4] == Py_None)) return -1;
    auto* fn = entry(3, &seer_qk_norm_rope_backward);
    return unlocked([&] {
      return fn(&g.s, zq, zk, yq, yk, q, k, wq, wk, pos, dq, dk, gq, gk, live, ws, bytes, stream);
    });
  });
}

// One cache of a dense decode from KVCache's tensors: (cache,) or (pool, block table).
bool cache_of(Call& c, PyObject* keep, int64_t B, int64_t d, at::ScalarType type, int64_t* heads, int64_t* page, seer_kv_t* kv) {
  if (!PyTuple_Check(keep)) return false;
  const bool paged = PyTuple_GET_SIZE(keep) == 2;
  const at::Tensor* t = c.get(PyTuple_GET_ITEM(keep, 0));
  if (!c.ok || t->scalar_type() != type || t->dim() != 4 || t->size(3) != d || t->stride(3) != 1) return false;
  if (*heads && t->size(1) != *heads) return false;
  *heads = t->size(1);
  *kv = seer_kv_t{};
  kv->layout = paged ? SEER_KV_PAGED : SEER_KV_CONTIGUOUS;
  kv->data = t->data_ptr();
  kv->stride_b = t->stride(0);
  kv->stride_h = t->stride(1);
  kv->stride_t = t->stride(2);
  if (!paged) {
    kv->num_tokens = t->size(2);
    return t->size(0) >= B;
  }
  if (*page && t->size(2) != *page) return false;
  *page = t->size(2);
  const at::Tensor* table = c.get(PyTuple_GET_ITEM(keep, 1));
  if (!c.ok || table->scalar_type() != kI32 || table->dim() != 2 || table->size(0) < B || !table->is_contiguous() ||
      table->size(1) > INT32_MAX)
    return false;
  kv->num_pages = t->size(0);
  kv->block_table = static_cast<const int32_t*>(table->data_ptr());
  kv->max_pages_per_seq = (int32_t)table->size(1);
  return true;
}

// q, k's tensors, v's tensors, seqlens, out, workspace, window, softmax_scale, lse, err, stream
PyObject* dense_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 11, [&]() -> long {
    Call c;
    const at::Tensor* q = c.get(a[0]);
    if (!c.ok || q->dim() != 3) return -1;
    const int64_t B = q->size(0), Hq = q->size(1), d = q->size(2);
    const at::ScalarType type = q->scalar_type();
    if (type != at::ScalarType::BFloat16 && type != at::ScalarType::Half) return -1;
    int64_t heads = 0, page = 0;
    seer_kv_t k, v;
    if (!cache_of(c, a[1], B, d, type, &heads, &page, &k) || !cache_of(c, a[2], B, d, type, &heads, &page, &v)) return -1;
    if (B > INT32_MAX || Hq > INT32_MAX || d > INT32_MAX || heads > INT32_MAX || page > INT32_MAX) return -1;
    seer_dense_t s{};
    s.batch = (int32_t)B;
    s.num_q_heads = (int32_t)Hq;
    s.num_kv_heads = (int32_t)heads;
    s.head_dim = (int32_t)d;
    s.dtype = type == at::ScalarType::Half ? SEER_FP16 : SEER_BF16;
    s.page_size = page ? (int32_t)page : 1;
    s.window = c.i32(a[6]);
    s.softmax_scale = c.f32(a[7]);
    if (s.softmax_scale == 0.f && PyObject_IsTrue(a[7]) == 1) return -1;   // not 0 but for its rounding
    const void* qp = c.dense(a[0], {B, Hq, d}, type);
    const auto* lens = static_cast<int32_t*>(c.dense(a[3], {B}, kI32));
    void* out = c.dense(a[4], {B, Hq, d}, type);
    auto* lse = static_cast<float*>(c.dense_or_null(a[8], {B, Hq}, at::ScalarType::Float));
    int32_t* err = c.err(a[9]);
    const at::Tensor* w = c.get(a[5]);
    void* stream = c.stream(a[10]);
    if (!c.ok || w->scalar_type() != at::ScalarType::Byte || !w->is_contiguous()) return -1;
    void* ws = w->data_ptr();
    const size_t bytes = (size_t)w->numel();
    auto* fn = entry(4, &seer_dense_decode);
    return unlocked([&] { return fn(&s, qp, &k, &v, lens, out, lse, ws, bytes, err, stream); });
  });
}

// bind(name, address): a C entry point of the loaded library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* name = n == 2 ? PyUnicode_AsUTF8(a[0]) : nullptr;
  void* fn = name ? PyLong_AsVoidPtr(a[1]) : nullptr;
  if (PyErr_Occurred()) return nullptr;
  for (Entry& e : g_entries)
    if (name && !strcmp(e.name, name)) {
      e.fn = fn;
      Py_RETURN_NONE;
    }
  PyErr_SetString(PyExc_ValueError, "bind(name, address) of an entry point of this layer");
  return nullptr;
}

PyObject* entries(PyObject*, PyObject*) {
  PyObject* l = PyList_New(0);
  for (const Entry& e : g_entries) {
    PyObject* s = PyUnicode_FromString(e.name);
    PyList_Append(l, s);
    Py_DECREF(s);
  }
  return l;
}

#define SEER_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {SEER_METHOD(page_plan),
                           SEER_METHOD(page_release),
                           SEER_METHOD(qk_norm_rope),
                           SEER_METHOD(qk_norm_rope_backward),
                           SEER_METHOD(dense_decode),
                           SEER_METHOD(bind),
                           {"entries", entries, METH_NOARGS, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_seer_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seer_call() { return PyModule_Create(&g_module); }

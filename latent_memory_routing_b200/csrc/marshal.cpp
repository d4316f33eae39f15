// Argument marshalling of the generation calls (norms, append, tree attention)
// for CPython: what the ctypes binding does in Python -- element type, size,
// layout and device of every tensor, the token strides, the current stream --
// in one native call.  A decode step calls these operators once a layer with
// kernels of 3 to 15 us, and the checks in Python cost as much again.
//
// It only ever takes the case in which every check passes.  Anything else
// (another type, too few elements, a tensor elsewhere, a number that is none)
// makes it return None without having called the library, and the Python path
// then says what is wrong.  Returns the library's status otherwise.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/msa.h"

namespace {

PyObject *s_dtype, *s_shape, *s_stride, *s_numel, *s_contiguous, *s_device, *s_ptr, *s_stream;
PyObject* dtypes[5];  // float32, bfloat16, int32, int64, uint8
enum Kind { F32 = 0, BF16 = 1, I32 = 2, I64 = 3, U8 = 4 };
PyObject *get_device, *raw_stream;

decltype(&msa_qk_norm_rope) f_norm;
decltype(&msa_qk_norm_rope_backward) f_norm_back;
decltype(&msa_paged_append) f_append;
decltype(&msa_tree_attn) f_tree;

// The arguments of one call, read in order; `ok` falls once one does not pass.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  bool ok;
  long dev = -2;

  Args(PyObject* const* args, Py_ssize_t have, Py_ssize_t want)
      : a(args), n(have), ok(have == want) {
    if (!ok) return;
    PyObject* d = PyObject_CallNoArgs(get_device);
    if (!d) {
      ok = false;
      return;
    }
    dev = PyLong_AsLong(d);
    Py_DECREF(d);
  }
  long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  long long whole() { return ok ? integer(a[i++]) : 0; }
  int small() {
    const long long v = whole();
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return (int)v;
  }
  int peek(int at) {  // an argument ahead of its turn
    const long long v = ok ? integer(a[at]) : 0;
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return (int)v;
  }
  float real() {
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(a[i++]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return (float)v;
  }
  // t.name(), an integer
  long long ask(PyObject* t, PyObject* name) {
    if (!ok) return 0;
    PyObject* r = PyObject_CallMethodNoArgs(t, name);
    if (!r) {
      ok = false;
      return 0;
    }
    const long long v = r == Py_True ? 1 : r == Py_False ? 0 : integer(r);
    Py_DECREF(r);
    return v;
  }
  void typed(PyObject* t, int kind) {
    if (!ok) return;
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d || kind < 0 || d != dtypes[kind]) ok = false;
    Py_XDECREF(d);
    if (ok && ask(t, s_device) != dev) ok = false;
  }
  // A contiguous tensor of at least `need` elements, an address, or None.
  void* tensor(long long need, int kind) {
    if (!ok) return nullptr;
    PyObject* t = a[i++];
    if (t == Py_None) return nullptr;
    if (PyLong_Check(t)) return reinterpret_cast<void*>((intptr_t)integer(t));
    typed(t, kind);
    if (ok && (ask(t, s_numel) < need || !ask(t, s_contiguous))) ok = false;
    return reinterpret_cast<void*>((intptr_t)ask(t, s_ptr));
  }
  // [>= n_tok][heads][D] with tokens `stride` elements apart.
  void* rows(long long n_tok, long long heads, long long D, int kind, int64_t* stride) {
    *stride = heads * D;
    if (!ok) return nullptr;
    PyObject* t = a[i++];
    if (t == Py_None) return nullptr;
    if (PyLong_Check(t)) return reinterpret_cast<void*>((intptr_t)integer(t));
    typed(t, kind);
    long long sh[3] = {0, 0, 0}, st[3] = {0, 0, 0};
    PyObject* p = ok ? PyObject_GetAttr(t, s_shape) : nullptr;
    three(p, sh);
    p = ok ? PyObject_CallMethodNoArgs(t, s_stride) : nullptr;
    three(p, st);
    if (!ok || sh[0] < n_tok || sh[1] != heads || sh[2] != D) {
      ok = false;
      return nullptr;
    }
    if (sh[0] > 0 && heads > 0) {
      if (st[2] != 1 || (heads > 1 && st[1] != D)) ok = false;
      if (sh[0] > 1) {
        if (st[0] < *stride || st[0] * (kind == F32 ? 4 : 2) % 16) ok = false;
        *stride = st[0];
      }
    }
    return reinterpret_cast<void*>((intptr_t)ask(t, s_ptr));
  }
  void three(PyObject* p, long long (&v)[3]) {
    if (!p || !PyTuple_Check(p) || PyTuple_GET_SIZE(p) != 3)
      ok = false;
    else
      for (int x = 0; x < 3; ++x) v[x] = integer(PyTuple_GET_ITEM(p, x));
    Py_XDECREF(p);
  }
  msa_stream_t stream() {
    if (!ok) return nullptr;
    PyObject *o = a[i++], *r = nullptr;
    long long v = 0;
    if (PyLong_Check(o)) {
      v = integer(o);
    } else {
      if (o == Py_None) {
        PyObject* d = PyLong_FromLong(dev);
        r = d ? PyObject_CallOneArg(raw_stream, d) : nullptr;
        Py_XDECREF(d);
      } else {
        r = PyObject_GetAttr(o, s_stream);
      }
      if (r) v = integer(r);
      else ok = false;
      Py_XDECREF(r);
    }
    return reinterpret_cast<msa_stream_t>((intptr_t)v);
  }
  // Calls the library, or returns None where an argument did not pass.
  template <typename Call> PyObject* finish(Call call) {
    if (!ok) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = call();
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
  }
};

int float_kind(int dt) { return dt == MSA_F32 ? F32 : dt == MSA_BF16 ? BF16 : -1; }

// dt, n_tok, Hq, H, D, q, k, q_weight, k_weight, positions, eps, rope_base,
// q_out, k_out, stream
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args g(args, n, 15);
  const int dt = g.small();
  const long long n_tok = g.whole();
  const int Hq = g.small(), H = g.small(), D = g.small(), k = float_kind(dt);
  int64_t qs, ks;
  void *q = g.rows(n_tok, Hq, D, k, &qs), *kk = g.rows(n_tok, H, D, k, &ks);
  void *qw = g.tensor(D, k), *kw = g.tensor(D, k), *pos = g.tensor(n_tok, I32);
  const float eps = g.real(), base = g.real();
  void *qo = g.tensor(n_tok * Hq * D, k), *ko = g.tensor(n_tok * H * D, k);
  const msa_stream_t s = g.stream();
  return g.finish([&] {
    return f_norm((msa_dtype)dt, n_tok, Hq, H, D, q, qs, kk, ks, qw, kw,
                  static_cast<int32_t*>(pos), eps, base, qo, ko, s);
  });
}

// dt, grad_dt, n_tok, Hq, H, D, q, k, q_weight, k_weight, positions, eps,
// rope_base, dq_out, dk_out, dq, dk, dq_weight, dk_weight, ws, ws_bytes, stream
PyObject* norm_back(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args g(args, n, 22);
  const int dt = g.small(), gdt = g.small();
  const long long n_tok = g.whole();
  const int Hq = g.small(), H = g.small(), D = g.small();
  const int k = float_kind(dt), gk = float_kind(gdt);
  int64_t qs, ks, dqs, dks;
  void *q = g.rows(n_tok, Hq, D, k, &qs), *kk = g.rows(n_tok, H, D, k, &ks);
  void *qw = g.tensor(D, k), *kw = g.tensor(D, k), *pos = g.tensor(n_tok, I32);
  const float eps = g.real(), base = g.real();
  void *dqo = g.tensor(n_tok * Hq * D, gk), *dko = g.tensor(n_tok * H * D, gk);
  void *dq = g.rows(n_tok, Hq, D, gk, &dqs), *dk = g.rows(n_tok, H, D, gk, &dks);
  void *dqw = g.tensor(D, F32), *dkw = g.tensor(D, F32);
  const long long ws_bytes = g.ok ? g.integer(args[20]) : 0;
  void* ws = g.tensor(ws_bytes, U8);
  ++g.i;
  if (ws_bytes < 0) g.ok = false;
  const msa_stream_t s = g.stream();
  return g.finish([&] {
    return f_norm_back((msa_dtype)dt, (msa_dtype)gdt, n_tok, Hq, H, D, q, qs, kk, ks, qw, kw,
                       static_cast<int32_t*>(pos), eps, base, dqo, dko, dq, dqs, dk, dks,
                       static_cast<float*>(dqw), static_cast<float*>(dkw), ws, (size_t)ws_bytes,
                       s);
  });
}

// dt, B, n_tok, Hq, H, D, q, k, v, q_weight, k_weight, tok_offsets, positions,
// eps, rope_base, block_table, max_pages, cache_len, page_size, n_pages,
// k_pages, v_pages, q_out, stream
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args g(args, n, 24);
  const int dt = g.small(), B = g.small();
  const long long n_tok = g.whole();
  const int Hq = g.small(), H = g.small(), D = g.small(), k = float_kind(dt);
  int64_t qs, ks, vs;
  void *q = g.rows(n_tok, Hq, D, k, &qs), *kk = g.rows(n_tok, H, D, k, &ks),
       *v = g.rows(n_tok, H, D, k, &vs);
  void *qw = g.tensor(D, k), *kw = g.tensor(D, k);
  void *off = g.tensor((long long)B + 1, I64), *pos = g.tensor(n_tok, I32);
  const float eps = g.real(), base = g.real();
  const int max_pages = g.peek(16);
  void* table = g.tensor((long long)B * max_pages, I32);
  ++g.i;
  void* len = g.tensor(B, I32);
  const int page = g.small(), n_pages = g.small();
  const long long pool = (long long)n_pages * H * page * D;
  void *kp = g.tensor(pool, k), *vp = g.tensor(pool, k), *qo = g.tensor(n_tok * Hq * D, k);
  const msa_stream_t s = g.stream();
  return g.finish([&] {
    return f_append((msa_dtype)dt, B, n_tok, Hq, H, D, q, qs, kk, ks, v, vs, qw, kw,
                    static_cast<int64_t*>(off), static_cast<int32_t*>(pos), eps, base,
                    static_cast<int32_t*>(table), max_pages, static_cast<int32_t*>(len), page,
                    n_pages, kp, vp, qo, s);
  });
}

// dt, B, n_tok, n_max, Hq, H, D, q, tok_offsets, parents, k_mem, v_mem,
// mem_len, m_cap, k_pages, v_pages, n_pages, page_size, block_table,
// max_pages, cache_len, scale, out, ws, ws_bytes, stream
PyObject* tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args g(args, n, 26);
  const int dt = g.small(), B = g.small();
  const long long n_tok = g.whole();
  const int n_max = g.small(), Hq = g.small(), H = g.small(), D = g.small(), k = float_kind(dt);
  const long long rows = n_tok * Hq * D;
  void *q = g.tensor(rows, k), *off = g.tensor((long long)B + 1, I64),
       *par = g.tensor(n_tok, I32);
  const int m_cap = g.peek(13);
  const int n_pages = g.peek(16);
  const int page = g.peek(17);
  const long long mem = (long long)B * m_cap * H * D, pool = (long long)n_pages * H * page * D;
  void *km = g.tensor(mem, k), *vm = g.tensor(mem, k), *ml = g.tensor(m_cap ? B : 0, I32);
  ++g.i;
  void *kp = g.tensor(pool, k), *vp = g.tensor(pool, k);
  g.i += 2;
  const int max_pages = g.peek(19);
  void* table = g.tensor((long long)B * max_pages, I32);
  ++g.i;
  void* len = g.tensor(B, I32);
  const float scale = g.real();
  void* out = g.tensor(rows, k);
  const long long ws_bytes = g.ok ? g.integer(args[24]) : 0;
  void* ws = g.tensor(ws_bytes, U8);
  ++g.i;
  if (ws_bytes < 0) g.ok = false;
  const msa_stream_t s = g.stream();
  return g.finish([&] {
    return f_tree((msa_dtype)dt, B, n_tok, n_max, Hq, H, D, q, static_cast<int64_t*>(off),
                  static_cast<int32_t*>(par), km, vm, static_cast<int32_t*>(ml), m_cap, kp, vp,
                  n_pages, page, static_cast<int32_t*>(table), max_pages,
                  static_cast<int32_t*>(len), scale, out, ws, (size_t)ws_bytes, s);
  });
}

// bind((address of each function), (the five dtypes), current device,
// raw stream of a device)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[4];
  PyObject *d[5], *dev, *raw;
  if (!PyArg_ParseTuple(args, "(KKKK)(OOOOO)OO", &f[0], &f[1], &f[2], &f[3], &d[0], &d[1], &d[2],
                        &d[3], &d[4], &dev, &raw))
    return nullptr;
  f_norm = reinterpret_cast<decltype(f_norm)>(f[0]);
  f_norm_back = reinterpret_cast<decltype(f_norm_back)>(f[1]);
  f_append = reinterpret_cast<decltype(f_append)>(f[2]);
  f_tree = reinterpret_cast<decltype(f_tree)>(f[3]);
  for (int i = 0; i < 5; ++i) {
    Py_INCREF(d[i]);
    dtypes[i] = d[i];
  }
  Py_INCREF(dev);
  Py_INCREF(raw);
  get_device = dev;
  raw_stream = raw;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "Takes the library's addresses and torch's types."},
    {"msa_qk_norm_rope", (PyCFunction)(void*)norm, METH_FASTCALL, nullptr},
    {"msa_qk_norm_rope_backward", (PyCFunction)(void*)norm_back, METH_FASTCALL, nullptr},
    {"msa_paged_append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
    {"msa_tree_attn", (PyCFunction)(void*)tree, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_numel = PyUnicode_InternFromString("numel");
  s_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_device = PyUnicode_InternFromString("get_device");
  s_ptr = PyUnicode_InternFromString("data_ptr");
  s_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}

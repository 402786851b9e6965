/* aq_python.c -- marshalling of the serving calls from torch tensors to the C ABI, as a CPython module.
 *
 * A decode step makes these calls one after another on a few tokens, each a launch of a few
 * microseconds, and the marshalling of a call in Python (shapes, strides, pointers, then up to 23 converted
 * arguments) took longer than its kernel: 13 to 18 us a call against 5 to 8 us this way, launch included.
 * The module knows tensors by their Python attributes alone (dtype, shape, stride(), data_ptr()): it is
 * built against Python.h and aq.h, and is given the library's entry points by address, so that it serves
 * whichever build of the library the binding has loaded. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "aq.h"

static aq_status (*f_rope)(const aq_rope_spec*, const int32_t*, int64_t, int32_t, int32_t, const void*, int64_t, int64_t,
                           void*, int64_t, int64_t, int32_t, void*);
static aq_status (*f_kv_write)(const aq_kv_cache*, const int64_t*, int64_t, const void*, int64_t, int64_t, const void*,
                               int64_t, int64_t, const aq_rope_spec*, const int32_t*, const void*, int32_t, int64_t, int64_t,
                               void*, int64_t, int64_t, void*);
static aq_status (*f_kv_read)(const aq_kv_cache*, const int64_t*, int64_t, void*, int64_t, int64_t, void*, int64_t, int64_t,
                              void*);
static size_t (*f_attention_bytes)(const aq_kv_cache*, const aq_draft_batch*, int32_t);
static aq_status (*f_attention)(const aq_kv_cache*, const aq_draft_batch*, const void*, int32_t, int64_t, int64_t, float,
                                void*, int64_t, int64_t, float*, void*, size_t, void*);
static aq_status (*f_verify)(int32_t, int32_t, const int32_t*, const int32_t*, const int32_t*, int64_t, int32_t, const void*,
                             int64_t, const void*, int64_t, int64_t, int32_t, const float*, const float*, int64_t, int32_t*,
                             int32_t*, int64_t, int32_t, int32_t*, void*);

static PyObject *t_bf16, *t_f32, *t_i32, *t_i64, *t_u64, *t_u8;   /* torch dtypes: one object each */
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_freq, *s_layout, *s_magnitude, *s_k, *s_v, *s_k_scale, *s_v_scale;

typedef struct {
  int nd;
  int64_t shape[4], stride[4];
  uintptr_t ptr;
} tensor;

/* dtype (NULL: any of a and b), dimensions, pointer of a tensor; 0 on success, with a Python error otherwise. */
static int read_ints(PyObject* tuple, int64_t* out, int nd) {
  for (int i = 0; i < nd; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return 0;
}

static int read_tensor(PyObject* obj, const char* name, PyObject* a, PyObject* b, int nd, tensor* t, PyObject** dtype) {
  PyObject* d = PyObject_GetAttr(obj, s_dtype);
  if (!d) return -1;
  Py_DECREF(d);   /* torch keeps its dtype objects */
  if (d != a && d != b) {
    PyErr_Format(PyExc_TypeError, "%s: expected a %S tensor, got %S", name, a, d);
    return -1;
  }
  if (dtype) *dtype = d;
  PyObject* shape = PyObject_GetAttr(obj, s_shape);
  if (!shape) return -1;
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != nd) {
    PyErr_Format(PyExc_ValueError, "%s: expected %d dimensions, got shape %S", name, nd, shape);
    Py_DECREF(shape);
    return -1;
  }
  int bad = read_ints(shape, t->shape, nd);
  Py_DECREF(shape);
  if (bad) return -1;
  PyObject* stride = PyObject_CallMethodNoArgs(obj, s_stride);
  if (!stride) return -1;
  bad = !PyTuple_Check(stride) || PyTuple_GET_SIZE(stride) != nd || read_ints(stride, t->stride, nd);
  Py_DECREF(stride);
  if (bad) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: unexpected strides", name);
    return -1;
  }
  PyObject* ptr = PyObject_CallMethodNoArgs(obj, s_data_ptr);
  if (!ptr) return -1;
  t->ptr = (uintptr_t)PyLong_AsUnsignedLongLong(ptr);
  Py_DECREF(ptr);
  t->nd = nd;
  return PyErr_Occurred() ? -1 : 0;
}

static int contiguous(const tensor* t) {
  int64_t want = 1;
  for (int i = t->nd - 1; i >= 0; --i) {
    if (t->shape[i] == 0) return 1;
    if (t->shape[i] > 1 && t->stride[i] != want) return 0;
    want *= t->shape[i];
  }
  return 1;
}

/* A contiguous 1-D tensor of n elements (n < 0: any number). */
static int read_flat(PyObject* obj, const char* name, PyObject* dtype, int64_t n, tensor* t) {
  if (read_tensor(obj, name, dtype, dtype, 1, t, NULL)) return -1;
  if ((n >= 0 && t->shape[0] != n) || !contiguous(t)) {
    if (n >= 0) PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor of %lld elements, got %lld", name, (long long)n, (long long)t->shape[0]);
    else PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor", name);
    return -1;
  }
  return 0;
}

/* A bf16 [tokens, heads, head_dim] tensor or view, -1: any; strides as the ABI takes them. */
static int read_heads(PyObject* obj, const char* name, int64_t tokens, int64_t heads, int64_t dim, tensor* t) {
  if (read_tensor(obj, name, t_bf16, t_bf16, 3, t, NULL)) return -1;
  if ((tokens >= 0 && t->shape[0] != tokens) || (heads >= 0 && t->shape[1] != heads) || (dim >= 0 && t->shape[2] != dim)) {
    PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld, %lld, %lld), got (%lld, %lld, %lld) (-1: any)", name, (long long)tokens,
                 (long long)heads, (long long)dim, (long long)t->shape[0], (long long)t->shape[1], (long long)t->shape[2]);
    return -1;
  }
  if (t->shape[2] > 1 && t->stride[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: expected unit stride along the head", name);
    return -1;
  }
  if (t->shape[1] <= 1) t->stride[1] = t->shape[2];
  if (t->shape[0] <= 1) t->stride[0] = t->shape[1] * t->stride[1];
  return 0;
}

/* A 2-D tensor of `rows` rows (-1: any) and at least `cols` columns with unit column stride. */
static int read_rows(PyObject* obj, const char* name, PyObject* a, PyObject* b, int64_t rows, int64_t cols, tensor* t, PyObject** dtype) {
  if (read_tensor(obj, name, a, b, 2, t, dtype)) return -1;
  if ((rows >= 0 && t->shape[0] != rows) || t->shape[1] < cols) {
    PyErr_Format(PyExc_ValueError, "%s: expected [%lld, %lld], got [%lld, %lld]", name, (long long)rows, (long long)cols,
                 (long long)t->shape[0], (long long)t->shape[1]);
    return -1;
  }
  if (t->shape[1] > 1 && t->stride[1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: expected unit column stride", name);
    return -1;
  }
  if (t->shape[0] <= 1 && t->stride[0] < t->shape[1]) t->stride[0] = t->shape[1];
  return 0;
}

static int read_int(PyObject* obj, long long* out) {
  *out = PyLong_AsLongLong(obj);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int read_int32(PyObject* obj, const char* name, int32_t* out) {
  long long v;
  if (read_int(obj, &v)) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s=%lld is out of range", name, v);
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

static int read_rope(PyObject* obj, aq_rope_spec* r) {
  PyObject* freq = PyObject_GetAttr(obj, s_freq);
  if (!freq) return -1;
  tensor t;
  int bad = read_tensor(freq, "Rope.freq", t_i64, t_u64, 1, &t, NULL);
  Py_DECREF(freq);
  if (bad) return -1;
  if (!contiguous(&t)) {
    PyErr_SetString(PyExc_ValueError, "Rope.freq: expected a contiguous tensor");
    return -1;
  }
  PyObject* layout = PyObject_GetAttr(obj, s_layout);
  PyObject* magnitude = layout ? PyObject_GetAttr(obj, s_magnitude) : NULL;
  bad = !magnitude || read_int32(layout, "layout", &r->layout);
  if (!bad) r->magnitude = (float)PyFloat_AsDouble(magnitude);
  Py_XDECREF(layout);
  Py_XDECREF(magnitude);
  r->freq = (const uint64_t*)t.ptr;
  r->rotary_dim = (int32_t)(2 * t.shape[0]);
  return bad || PyErr_Occurred() ? -1 : 0;
}

static int32_t small(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }

static int read_cache(PyObject* obj, aq_kv_cache* c) {
  PyObject* part[4] = {PyObject_GetAttr(obj, s_k), PyObject_GetAttr(obj, s_v), PyObject_GetAttr(obj, s_k_scale),
                       PyObject_GetAttr(obj, s_v_scale)};
  tensor t[4];
  int bad = !part[0] || !part[1] || !part[2] || !part[3];
  const int scaled = !bad && part[2] != Py_None;
  PyObject* code = scaled ? t_u8 : t_bf16;
  bad = bad || read_tensor(part[0], "KvCache.k", code, code, 4, &t[0], NULL) || read_tensor(part[1], "KvCache.v", code, code, 4, &t[1], NULL);
  if (!bad && scaled != (part[3] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, "KvCache: k_scale and v_scale go together");
    bad = 1;
  }
  if (!bad && scaled)
    bad = read_tensor(part[2], "KvCache.k_scale", t_f32, t_f32, 3, &t[2], NULL) || read_tensor(part[3], "KvCache.v_scale", t_f32, t_f32, 3, &t[3], NULL);
  for (int i = 0; i < 4; ++i) Py_XDECREF(part[i]);
  if (bad) return -1;
  for (int i = 0; i < (scaled ? 4 : 2); ++i) {
    for (int k = 0; k < (i < 2 ? 4 : 3); ++k) bad = bad || t[i].shape[k] != t[0].shape[k];
    bad = bad || !contiguous(&t[i]);
  }
  if (bad) {
    PyErr_SetString(PyExc_ValueError, "KvCache: expected contiguous k and v of one shape [pages, kv_heads, page_size, head_dim], "
                                      "and scales of its first three dimensions");
    return -1;
  }
  c->k = (void*)t[0].ptr;
  c->v = (void*)t[1].ptr;
  c->k_scale = scaled ? (float*)t[2].ptr : NULL;
  c->v_scale = scaled ? (float*)t[3].ptr : NULL;
  c->pages = small(t[0].shape[0]);
  c->kv_heads = small(t[0].shape[1]);
  c->page_size = small(t[0].shape[2]);
  c->head_dim = small(t[0].shape[3]);
  c->type = scaled ? AQ_KV_E4M3 : AQ_KV_BF16;
  return 0;
}

static int want(Py_ssize_t got, Py_ssize_t n, const char* name) {
  if (got == n && f_rope) return 0;
  PyErr_Format(PyExc_TypeError, f_rope ? "%s: wrong number of arguments" : "%s: bind() has not been called", name);
  return -1;
}

static void* stream_of(PyObject* obj) { return (void*)(uintptr_t)PyLong_AsUnsignedLongLong(obj); }

/* rope(rope, pos, x, y, inverse, stream) */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  aq_rope_spec r;
  tensor pos, x, y;
  if (want(n, 6, "rope") || read_rope(a[0], &r) || read_heads(a[2], "x", -1, -1, -1, &x) ||
      read_heads(a[3], "y", x.shape[0], x.shape[1], x.shape[2], &y) || read_flat(a[1], "pos", t_i32, x.shape[0], &pos))
    return NULL;
  const int inverse = PyObject_IsTrue(a[4]);
  void* st = stream_of(a[5]);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong(f_rope(&r, (const int32_t*)pos.ptr, x.shape[0], small(x.shape[1]), small(x.shape[2]), (const void*)x.ptr,
                                x.stride[0], x.stride[1], (void*)y.ptr, y.stride[0], y.stride[1], inverse, st));
}

/* kv_write(cache, k, v, slots, rope, pos, q, q_out, stream) */
static PyObject* py_kv_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  aq_kv_cache c;
  aq_rope_spec r;
  tensor k, v, slots, pos = {0}, q = {0}, o = {0};
  if (want(n, 9, "kv_write") || read_cache(a[0], &c) || read_heads(a[1], "k", -1, c.kv_heads, c.head_dim, &k)) return NULL;
  const int64_t T = k.shape[0];
  if (read_heads(a[2], "v", T, c.kv_heads, c.head_dim, &v) || read_flat(a[3], "slots", t_i64, T, &slots)) return NULL;
  const int turned = a[4] != Py_None;
  if (turned && read_rope(a[4], &r)) return NULL;
  if (a[5] != Py_None && read_flat(a[5], "pos", t_i32, T, &pos)) return NULL;
  if (a[6] != Py_None && (read_heads(a[6], "q", T, -1, c.head_dim, &q) || read_heads(a[7], "q_out", T, q.shape[1], c.head_dim, &o))) return NULL;
  void* st = stream_of(a[8]);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong(f_kv_write(&c, (const int64_t*)slots.ptr, T, (const void*)k.ptr, k.stride[0], k.stride[1], (const void*)v.ptr,
                                    v.stride[0], v.stride[1], turned ? &r : NULL, (const int32_t*)pos.ptr, (const void*)q.ptr,
                                    small(q.shape[1]), q.stride[0], q.stride[1], (void*)o.ptr, o.stride[0], o.stride[1], st));
}

/* kv_read(cache, slots, k, v, stream) */
static PyObject* py_kv_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  aq_kv_cache c;
  tensor slots, k, v;
  if (want(n, 5, "kv_read") || read_cache(a[0], &c) || read_flat(a[1], "slots", t_i64, -1, &slots) ||
      read_heads(a[2], "k", slots.shape[0], c.kv_heads, c.head_dim, &k) || read_heads(a[3], "v", slots.shape[0], c.kv_heads, c.head_dim, &v))
    return NULL;
  void* st = stream_of(a[4]);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong(f_kv_read(&c, (const int64_t*)slots.ptr, slots.shape[0], (void*)k.ptr, k.stride[0], k.stride[1], (void*)v.ptr,
                                   v.stride[0], v.stride[1], st));
}

/* attention_bytes(cache, q_heads, batch, max_q, total_q): -1 where the call would be refused */
static PyObject* py_attention_bytes(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  aq_kv_cache c;
  aq_draft_batch d = {0};
  int32_t heads;
  long long total;
  if (want(n, 5, "attention_bytes") || read_cache(a[0], &c) || read_int32(a[1], "q_heads", &heads) || read_int32(a[2], "batch", &d.batch) ||
      read_int32(a[3], "max_q", &d.max_q) || read_int(a[4], &total))
    return NULL;
  d.total_q = total;
  const size_t need = f_attention_bytes(&c, &d, heads);
  return need == (size_t)-1 ? PyLong_FromLong(-1) : PyLong_FromSize_t(need);
}

/* attention(cache, q, cu_q, ctx, page_table, max_q, mask, depth, window, scale, out, lse, workspace, stream) */
static PyObject* py_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  aq_kv_cache c;
  aq_draft_batch d = {0};
  tensor q, cu, ctx, table, mask = {0}, depth = {0}, out, lse = {0}, ws = {0};
  if (want(n, 14, "attention") || read_cache(a[0], &c) || read_heads(a[1], "q", -1, -1, c.head_dim, &q) ||
      read_rows(a[4], "page_table", t_i32, t_i32, -1, 0, &table, NULL) || read_flat(a[2], "cu_q", t_i32, table.shape[0] + 1, &cu) ||
      read_flat(a[3], "ctx", t_i32, table.shape[0], &ctx) || read_int32(a[5], "max_q", &d.max_q))
    return NULL;
  const int64_t total = q.shape[0];
  if (a[6] != Py_None && read_rows(a[6], "mask", t_i64, t_i64, total, ((int64_t)d.max_q + 63) / 64, &mask, NULL)) return NULL;
  if (a[7] != Py_None && read_flat(a[7], "depth", t_i32, total, &depth)) return NULL;
  if (read_int32(a[8], "window", &d.window) || read_heads(a[10], "out", total, q.shape[1], c.head_dim, &out)) return NULL;
  const double scale = PyFloat_AsDouble(a[9]);
  if (a[11] != Py_None) {
    if (read_tensor(a[11], "lse", t_f32, t_f32, 2, &lse, NULL)) return NULL;
    if (lse.shape[0] != total || lse.shape[1] != q.shape[1] || !contiguous(&lse)) {
      PyErr_Format(PyExc_ValueError, "lse: expected a contiguous [%lld, %lld] tensor", (long long)total, (long long)q.shape[1]);
      return NULL;
    }
  }
  if (a[12] != Py_None && read_flat(a[12], "workspace", t_u8, -1, &ws)) return NULL;
  void* st = stream_of(a[13]);
  if (PyErr_Occurred()) return NULL;
  d.batch = small(table.shape[0]);
  d.total_q = total;
  d.cu_q = (const int32_t*)cu.ptr;
  d.ctx = (const int32_t*)ctx.ptr;
  d.page_table = (const int32_t*)table.ptr;
  d.pages_per_seq = small(table.shape[1]);
  d.ld_table = table.stride[0];
  d.mask = (const uint64_t*)mask.ptr;
  d.ld_mask = mask.stride[0];
  d.depth = (const int32_t*)depth.ptr;
  return PyLong_FromLong(f_attention(&c, &d, (const void*)q.ptr, small(q.shape[1]), q.stride[0], q.stride[1], (float)scale, (void*)out.ptr,
                                     out.stride[0], out.stride[1], (float*)lse.ptr, (void*)ws.ptr, (size_t)ws.shape[0], st));
}

/* verify(p, tokens, cu, u, noise, q, parent, path_cap, max_nodes, n_accepted, path, token, stream) */
static PyObject* py_verify(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  tensor p, tokens, cu, u, noise, q = {0}, parent = {0}, count, path, token;
  PyObject* dtype;
  int32_t cap, most;
  if (want(n, 13, "verify") || read_rows(a[0], "p", t_f32, t_bf16, -1, 0, &p, &dtype) || read_flat(a[1], "tokens", t_i32, -1, &tokens) ||
      read_flat(a[2], "cu", t_i32, -1, &cu) || read_flat(a[3], "u", t_f32, tokens.shape[0], &u))
    return NULL;
  const int64_t batch = cu.shape[0] - 1, vocab = p.shape[1];
  if (batch < 0) {
    PyErr_SetString(PyExc_ValueError, "cu: expected [batch + 1] elements");
    return NULL;
  }
  if (read_rows(a[4], "noise", t_f32, t_f32, batch, vocab, &noise, NULL)) return NULL;
  if (a[5] != Py_None && read_rows(a[5], "q", dtype, dtype, p.shape[0], vocab, &q, NULL)) return NULL;
  if (noise.shape[1] != vocab || (a[5] != Py_None && q.shape[1] != vocab)) {
    PyErr_Format(PyExc_ValueError, "noise and q: expected %lld columns", (long long)vocab);
    return NULL;
  }
  if ((a[6] != Py_None && read_flat(a[6], "parent", t_i32, tokens.shape[0], &parent)) || read_int32(a[7], "path_cap", &cap) ||
      read_int32(a[8], "max_nodes", &most) || read_flat(a[9], "n_accepted", t_i32, batch, &count) ||
      read_rows(a[10], "path", t_i32, t_i32, batch, cap, &path, NULL) || read_flat(a[11], "token", t_i32, batch, &token))
    return NULL;
  void* st = stream_of(a[12]);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong(f_verify(small(batch), small(vocab), (const int32_t*)cu.ptr, (const int32_t*)tokens.ptr, (const int32_t*)parent.ptr,
                                  tokens.shape[0], most, (const void*)p.ptr, p.stride[0], (const void*)q.ptr, q.stride[0], p.shape[0],
                                  dtype == t_f32 ? AQ_PROB_F32 : AQ_PROB_BF16, (const float*)u.ptr, (const float*)noise.ptr,
                                  noise.stride[0], (int32_t*)count.ptr, (int32_t*)path.ptr, path.stride[0], cap, (int32_t*)token.ptr, st));
}

/* bind((addresses of the entry points), (torch's bfloat16, float32, int32, int64, uint64, uint8)) */
static PyObject* py_bind(PyObject* self, PyObject* args) {
  unsigned long long f[6];
  PyObject* t[6];
  if (!PyArg_ParseTuple(args, "(KKKKKK)(OOOOOO)", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &t[0], &t[1], &t[2], &t[3], &t[4], &t[5]))
    return NULL;
  *(void**)&f_rope = (void*)(uintptr_t)f[0];
  *(void**)&f_kv_write = (void*)(uintptr_t)f[1];
  *(void**)&f_kv_read = (void*)(uintptr_t)f[2];
  *(void**)&f_attention_bytes = (void*)(uintptr_t)f[3];
  *(void**)&f_attention = (void*)(uintptr_t)f[4];
  *(void**)&f_verify = (void*)(uintptr_t)f[5];
  PyObject** kept[6] = {&t_bf16, &t_f32, &t_i32, &t_i64, &t_u64, &t_u8};
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(t[i]);
    *kept[i] = t[i];
  }
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(rope), FAST(kv_write), FAST(kv_read), FAST(attention_bytes), FAST(attention), FAST(verify),
                                {"bind", py_bind, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_data_ptr, "data_ptr"}, {&s_freq, "freq"},
               {&s_layout, "layout"}, {&s_magnitude, "magnitude"}, {&s_k, "k"}, {&s_v, "v"}, {&s_k_scale, "k_scale"}, {&s_v_scale, "v_scale"}};
  for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}

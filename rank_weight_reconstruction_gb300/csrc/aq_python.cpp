// aq_python.cpp -- the serving calls on torch tensors: checks, output allocation and the call into the C ABI, as a
// CPython module.
//
// A decode step makes these calls one after another on a few tokens, each a launch of a few microseconds, and what
// a call costs the host decides the step's time. Converted in Python (shapes, strides, pointers, then up to 23 ctypes
// arguments) a call took 13 to 18 us, its kernel 2 to 10. Here the tensors are read as the C++ objects they are and
// the outputs allocated without passing through Python: 2.4 us a call with outputs given, launch included, and 4.5 to 7.3 with outputs
// made, from process to process (a rotation of one token 4.8 us where the attributes read in C and torch.empty took 10.7; a cache
// write and its read 11.1 where 28.3).
// The module is given the library's entry points by address, so that it serves whichever build of the library the binding
// has loaded, and a function of the binding that raises for an aq_status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <math.h>
#include <stdint.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "aq.h"

namespace {

decltype(&aq_rope) f_rope;
decltype(&aq_kv_write) f_kv_write;
decltype(&aq_kv_read) f_kv_read;
decltype(&aq_tree_attention_workspace_bytes) f_attention_bytes;
decltype(&aq_tree_attention) f_attention;
decltype(&aq_verify_drafts) f_verify;
PyObject* f_check;   // raises for a status that is not AQ_OK

PyObject *s_freq, *s_layout, *s_magnitude, *s_k, *s_v, *s_k_scale, *s_v_scale;

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong, kU64 = at::kUInt64, kU8 = at::kByte;

using Device = std::optional<c10::Device>;   // of the tensors read so far in a call

struct Tensor {
  int64_t shape[4] = {0, 0, 0, 0}, stride[4] = {0, 0, 0, 0};
  int nd = 0;
  void* ptr = nullptr;
  const at::Tensor* t = nullptr;
};

void take(const at::Tensor& t, Tensor* x) {
  x->t = &t;
  x->nd = static_cast<int>(t.dim());
  for (int i = 0; i < x->nd; ++i) {
    x->shape[i] = t.size(i);
    x->stride[i] = t.stride(i);
  }
  x->ptr = t.data_ptr();
}

// A tensor of dtype a or b and nd dimensions; false with a Python error otherwise. The functions below take views of
// tensors that their caller's arguments keep alive.
bool read(Device& dev, PyObject* obj, const char* name, at::ScalarType a, at::ScalarType b, int nd, Tensor* x) {
  if (!THPVariable_Check(obj)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %R", name, reinterpret_cast<PyObject*>(Py_TYPE(obj)));
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (t.scalar_type() != a && t.scalar_type() != b) {
    PyErr_Format(PyExc_TypeError, "%s: expected a %s tensor, got %s", name, c10::toString(a), c10::toString(t.scalar_type()));
    return false;
  }
  if (t.layout() != at::kStrided || t.dim() != nd) {
    PyErr_Format(PyExc_ValueError, "%s: expected a strided tensor of %d dimensions, got %d", name, nd, static_cast<int>(t.dim()));
    return false;
  }
  if (!dev) dev = t.device();
  if (*dev != t.device()) {
    PyErr_Format(PyExc_ValueError, "%s: on %s, the call's other tensors on %s", name, t.device().str().c_str(), dev->str().c_str());
    return false;
  }
  take(t, x);
  return true;
}

bool contiguous(const Tensor& x) {
  int64_t want = 1;
  for (int i = x.nd - 1; i >= 0; --i) {
    if (x.shape[i] == 0) return true;
    if (x.shape[i] > 1 && x.stride[i] != want) return false;
    want *= x.shape[i];
  }
  return true;
}

// A contiguous 1-D tensor of n elements (n < 0: any number).
bool read_flat(Device& dev, PyObject* obj, const char* name, at::ScalarType dtype, int64_t n, Tensor* x) {
  if (!read(dev, obj, name, dtype, dtype, 1, x)) return false;
  if ((n < 0 || x->shape[0] == n) && contiguous(*x)) return true;
  if (n >= 0)
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor of %lld elements, got %lld", name, static_cast<long long>(n),
                 static_cast<long long>(x->shape[0]));
  else
    PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor", name);
  return false;
}

// Strides of [tokens, heads, head_dim] as the ABI takes them, with unit stride along the head.
bool head_strides(const char* name, Tensor* x) {
  if (x->shape[2] > 1 && x->stride[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: expected unit stride along the head", name);
    return false;
  }
  if (x->shape[1] <= 1) x->stride[1] = x->shape[2];
  if (x->shape[0] <= 1) x->stride[0] = x->shape[1] * x->stride[1];
  return true;
}

// A bf16 [tokens, heads, head_dim] tensor or view; -1: any.
bool read_heads(Device& dev, PyObject* obj, const char* name, int64_t tokens, int64_t heads, int64_t dim, Tensor* x) {
  if (!read(dev, obj, name, kBf16, kBf16, 3, x)) return false;
  if ((tokens >= 0 && x->shape[0] != tokens) || (heads >= 0 && x->shape[1] != heads) || (dim >= 0 && x->shape[2] != dim)) {
    PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld, %lld, %lld), got (%lld, %lld, %lld) (-1: any)", name,
                 static_cast<long long>(tokens), static_cast<long long>(heads), static_cast<long long>(dim),
                 static_cast<long long>(x->shape[0]), static_cast<long long>(x->shape[1]), static_cast<long long>(x->shape[2]));
    return false;
  }
  return head_strides(name, x);
}

// A 2-D tensor of `rows` rows (-1: any) and at least `cols` columns with unit column stride.
bool read_rows(Device& dev, PyObject* obj, const char* name, at::ScalarType a, at::ScalarType b, int64_t rows, int64_t cols, Tensor* x) {
  if (!read(dev, obj, name, a, b, 2, x)) return false;
  if ((rows >= 0 && x->shape[0] != rows) || x->shape[1] < cols) {
    PyErr_Format(PyExc_ValueError, "%s: expected [%lld, %lld], got [%lld, %lld]", name, static_cast<long long>(rows),
                 static_cast<long long>(cols), static_cast<long long>(x->shape[0]), static_cast<long long>(x->shape[1]));
    return false;
  }
  if (x->shape[1] > 1 && x->stride[1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: expected unit column stride", name);
    return false;
  }
  if (x->shape[0] <= 1 && x->stride[0] < x->shape[1]) x->stride[0] = x->shape[1];
  return true;
}

bool read_int32(PyObject* obj, const char* name, int32_t* out) {
  const long long v = PyLong_AsLongLong(obj);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s=%lld is out of range", name, v);
    return false;
  }
  *out = static_cast<int32_t>(v);
  return true;
}

struct Ref {   // a reference that this function owns
  PyObject* o;
  explicit Ref(PyObject* obj) : o(obj) {}
  ~Ref() { Py_XDECREF(o); }
  Ref(const Ref&) = delete;
};

// The attributes of a Rope or a KvCache are held by it, and by these, for the length of the call.
struct Rope {
  PyObject* freq = nullptr;
  aq_rope_spec spec = {};
  ~Rope() { Py_XDECREF(freq); }
  bool read_from(Device& dev, PyObject* obj) {
    Tensor t;
    freq = PyObject_GetAttr(obj, s_freq);
    if (!freq || !read(dev, freq, "Rope.freq", kI64, kU64, 1, &t)) return false;
    if (!contiguous(t)) {
      PyErr_SetString(PyExc_ValueError, "Rope.freq: expected a contiguous tensor");
      return false;
    }
    Ref layout(PyObject_GetAttr(obj, s_layout)), magnitude(PyObject_GetAttr(obj, s_magnitude));
    if (!layout.o || !magnitude.o || !read_int32(layout.o, "layout", &spec.layout)) return false;
    spec.magnitude = static_cast<float>(PyFloat_AsDouble(magnitude.o));
    spec.freq = static_cast<const uint64_t*>(t.ptr);
    spec.rotary_dim = static_cast<int32_t>(2 * t.shape[0]);
    return !PyErr_Occurred();
  }
};

int32_t small(int64_t v) { return v > INT32_MAX ? INT32_MAX : static_cast<int32_t>(v); }

struct Cache {
  PyObject* part[4] = {};
  aq_kv_cache c = {};
  ~Cache() {
    for (PyObject* o : part) Py_XDECREF(o);
  }
  bool read_from(Device& dev, PyObject* obj) {
    PyObject* const name[4] = {s_k, s_v, s_k_scale, s_v_scale};
    for (int i = 0; i < 4; ++i)
      if (!(part[i] = PyObject_GetAttr(obj, name[i]))) return false;
    Tensor t[4];
    const bool scaled = part[2] != Py_None;
    const at::ScalarType code = scaled ? kU8 : kBf16;
    if (!read(dev, part[0], "KvCache.k", code, code, 4, &t[0]) || !read(dev, part[1], "KvCache.v", code, code, 4, &t[1])) return false;
    if (scaled != (part[3] != Py_None)) {
      PyErr_SetString(PyExc_ValueError, "KvCache: k_scale and v_scale go together");
      return false;
    }
    if (scaled && (!read(dev, part[2], "KvCache.k_scale", kF32, kF32, 3, &t[2]) || !read(dev, part[3], "KvCache.v_scale", kF32, kF32, 3, &t[3]))) return false;
    bool bad = false;
    for (int i = 0; i < (scaled ? 4 : 2); ++i) {
      for (int k = 0; k < (i < 2 ? 4 : 3); ++k) bad = bad || t[i].shape[k] != t[0].shape[k];
      bad = bad || !contiguous(t[i]);
    }
    if (bad) {
      PyErr_SetString(PyExc_ValueError, "KvCache: expected contiguous k and v of one shape [pages, kv_heads, page_size, head_dim], "
                                        "and scales of its first three dimensions");
      return false;
    }
    c.k = t[0].ptr;
    c.v = t[1].ptr;
    c.k_scale = static_cast<float*>(t[2].ptr);
    c.v_scale = static_cast<float*>(t[3].ptr);
    c.pages = small(t[0].shape[0]);
    c.kv_heads = small(t[0].shape[1]);
    c.page_size = small(t[0].shape[2]);
    c.head_dim = small(t[0].shape[3]);
    c.type = scaled ? AQ_KV_E4M3 : AQ_KV_BF16;
    return true;
  }
};

bool want(Py_ssize_t got, Py_ssize_t n, const char* name) {
  if (got == n && f_check) return true;
  PyErr_Format(PyExc_TypeError, f_check ? "%s: wrong number of arguments" : "%s: bind() has not been called", name);
  return false;
}

// The stream of a call: the one it was given, or the current one of the tensors' device. What a call allocates comes from its
// own stream's memory: under the current stream, a workspace let go at the end of the call would be the next request's there
// while the given stream's kernels still use it, and a block freed there would be written before its last reader is through.
// Outputs that go back to the caller are noted as used by the current stream too, where they will be read.
class Stream {
 public:
  void* handle = nullptr;
  bool read_from(PyObject* obj, const Tensor& on) {
    const bool gpu = on.t->is_cuda();
    if (gpu) {   // the library takes the current device's facts and launches there
      c10::DeviceIndex now = -1;
      if (c10::cuda::GetDevice(&now) != cudaSuccess || now != on.t->get_device()) {
        PyErr_Format(PyExc_ValueError, "the tensors of a call are on %s, which is not the current device", on.t->device().str().c_str());
        return false;
      }
    }
    if (gpu) current_ = c10::cuda::getCurrentCUDAStream(on.t->get_device());
    if (obj == Py_None) {
      handle = gpu ? static_cast<void*>(current_->stream()) : nullptr;
      return true;
    }
    const uintptr_t given = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(obj));
    if (PyErr_Occurred()) return false;
    handle = reinterpret_cast<void*>(given);
    // 1 names the default stream; every other handle is a pointer, or 2 for the thread's own
    cudaStream_t own = given == 1 ? nullptr : static_cast<cudaStream_t>(handle);
    if ((given & 1) && given != 1) {
      PyErr_Format(PyExc_ValueError, "stream: %p is no stream handle", handle);
      return false;
    }
    if (gpu && own != current_->stream()) {
      guard_.reset_stream(c10::cuda::getStreamFromExternal(own, on.t->get_device()));
      elsewhere_ = true;
    }
    return true;
  }
  // An output of this call on its way to the caller.
  PyObject* hand_out(at::Tensor&& t) {
    if (elsewhere_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *current_);
    return THPVariable_Wrap(std::move(t));
  }

 private:
  std::optional<c10::cuda::CUDAStream> current_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
  bool elsewhere_ = false;
};

bool ok(aq_status st) {
  if (st == AQ_OK) return true;
  Ref r(PyObject_CallFunction(f_check, "i", static_cast<int>(st)));
  if (r.o) PyErr_SetString(PyExc_RuntimeError, "the call was refused");
  return false;
}

// The library takes device pointers: a host tensor's is not passed on.
bool on_gpu(const Device& dev) {
  if (dev && dev->is_cuda()) return true;
  PyErr_Format(PyExc_ValueError, "the tensors of a call must be on a CUDA device, not on %s", dev ? dev->str().c_str() : "none");
  return false;
}

at::Tensor like(const Tensor& x) { return at::empty_like(*x.t); }
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& on) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(on.t->device()));
}
PyObject* given(PyObject* obj) {
  Py_INCREF(obj);
  return obj;
}
PyObject* pack(std::initializer_list<PyObject*> items) {   // takes the references over
  PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (!o) Py_CLEAR(tuple);
    if (tuple) PyTuple_SET_ITEM(tuple, i++, o);
    else Py_XDECREF(o);
  }
  if (!tuple && !PyErr_Occurred()) PyErr_NoMemory();
  return tuple;
}

// rope(rope, pos, x, y, inverse, stream) -> y
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Rope r;
  Tensor pos, x, y;
  Stream st;
  if (!want(n, 6, "rope") || !r.read_from(dev, a[0]) || !read_heads(dev, a[2], "x", -1, -1, -1, &x) || !read_flat(dev, a[1], "pos", kI32, x.shape[0], &pos) ||
      (a[3] != Py_None && !read_heads(dev, a[3], "y", x.shape[0], x.shape[1], x.shape[2], &y)) || !st.read_from(a[5], x))
    return nullptr;
  const int inverse = PyObject_IsTrue(a[4]);
  if (inverse < 0) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;   // outputs without a history
  at::Tensor made;
  if (a[3] == Py_None) {
    made = like(x);
    take(made, &y);
    if (!head_strides("y", &y)) return nullptr;
  }
  if (!on_gpu(dev) || !ok(f_rope(&r.spec, static_cast<const int32_t*>(pos.ptr), x.shape[0], small(x.shape[1]), small(x.shape[2]), x.ptr, x.stride[0], x.stride[1],
                 y.ptr, y.stride[0], y.stride[1], inverse, st.handle)))
    return nullptr;
  return made.defined() ? st.hand_out(std::move(made)) : given(a[3]);
  END_HANDLE_TH_ERRORS
}

// kv_write(cache, k, v, slots, rope, pos, q, q_out, stream) -> q_out
PyObject* py_kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Cache c;
  Rope r;
  Tensor k, v, slots, pos, q, o;
  Stream st;
  if (!want(n, 9, "kv_write") || !c.read_from(dev, a[0]) || !read_heads(dev, a[1], "k", -1, c.c.kv_heads, c.c.head_dim, &k)) return nullptr;
  const int64_t T = k.shape[0];
  const bool turned = a[4] != Py_None, queries = a[6] != Py_None;
  if (!read_heads(dev, a[2], "v", T, c.c.kv_heads, c.c.head_dim, &v) || !read_flat(dev, a[3], "slots", kI64, T, &slots) || (turned && !r.read_from(dev, a[4])) ||
      (a[5] != Py_None && !read_flat(dev, a[5], "pos", kI32, T, &pos)) || (queries && !read_heads(dev, a[6], "q", T, -1, c.c.head_dim, &q)) ||
      (queries && a[7] != Py_None && !read_heads(dev, a[7], "q_out", T, q.shape[1], c.c.head_dim, &o)) || !st.read_from(a[8], k))
    return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made;
  if (queries && a[7] == Py_None) {
    made = like(q);
    take(made, &o);
    if (!head_strides("q_out", &o)) return nullptr;
  }
  if (!on_gpu(dev) || !ok(f_kv_write(&c.c, static_cast<const int64_t*>(slots.ptr), T, k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1],
                     turned ? &r.spec : nullptr, static_cast<const int32_t*>(pos.ptr), q.ptr, small(q.shape[1]), q.stride[0], q.stride[1], o.ptr,
                     o.stride[0], o.stride[1], st.handle)))
    return nullptr;
  return made.defined() ? st.hand_out(std::move(made)) : given(a[7]);
  END_HANDLE_TH_ERRORS
}

// kv_read(cache, slots, k, v, stream) -> (k, v)
PyObject* py_kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Cache c;
  Tensor slots, x[2];
  Stream st;
  if (!want(n, 5, "kv_read") || !c.read_from(dev, a[0]) || !read_flat(dev, a[1], "slots", kI64, -1, &slots)) return nullptr;
  const char* const name[2] = {"k", "v"};
  for (int i = 0; i < 2; ++i)
    if (a[2 + i] != Py_None && !read_heads(dev, a[2 + i], name[i], slots.shape[0], c.c.kv_heads, c.c.head_dim, &x[i])) return nullptr;
  if (!st.read_from(a[4], slots)) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made[2];
  for (int i = 0; i < 2; ++i)
    if (a[2 + i] == Py_None) {
      made[i] = fresh({slots.shape[0], c.c.kv_heads, c.c.head_dim}, kBf16, slots);
      take(made[i], &x[i]);
      if (!head_strides(name[i], &x[i])) return nullptr;
    }
  if (!on_gpu(dev) || !ok(f_kv_read(&c.c, static_cast<const int64_t*>(slots.ptr), slots.shape[0], x[0].ptr, x[0].stride[0], x[0].stride[1], x[1].ptr, x[1].stride[0],
                    x[1].stride[1], st.handle)))
    return nullptr;
  return pack({made[0].defined() ? st.hand_out(std::move(made[0])) : given(a[2]), made[1].defined() ? st.hand_out(std::move(made[1])) : given(a[3])});
  END_HANDLE_TH_ERRORS
}

// attention_bytes(cache, q_heads, batch, max_q, total_q)
PyObject* py_attention_bytes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Cache c;
  aq_draft_batch d = {};
  int32_t heads;
  if (!want(n, 5, "attention_bytes") || !c.read_from(dev, a[0]) || !read_int32(a[1], "q_heads", &heads) || !read_int32(a[2], "batch", &d.batch) ||
      !read_int32(a[3], "max_q", &d.max_q))
    return nullptr;
  d.total_q = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  const size_t need = f_attention_bytes(&c.c, &d, heads);
  if (need == static_cast<size_t>(-1)) {
    ok(AQ_ERR_INVALID_ARG);
    return nullptr;
  }
  return PyLong_FromSize_t(need);
  END_HANDLE_TH_ERRORS
}

// attention(cache, q, cu_q, ctx, page_table, max_q, mask, depth, window, scale, out, lse, return_lse, workspace, stream)
//   -> out or (out, lse); scale None: head_dim^-1/2
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Cache c;
  aq_draft_batch d = {};
  Tensor q, cu, ctx, table, mask, depth, out, lse, ws;
  Stream st;
  if (!want(n, 15, "attention") || !c.read_from(dev, a[0]) || !read_heads(dev, a[1], "q", -1, -1, c.c.head_dim, &q) ||
      !read_rows(dev, a[4], "page_table", kI32, kI32, -1, 0, &table) || !read_flat(dev, a[2], "cu_q", kI32, table.shape[0] + 1, &cu) ||
      !read_flat(dev, a[3], "ctx", kI32, table.shape[0], &ctx) || !read_int32(a[5], "max_q", &d.max_q))
    return nullptr;
  const int64_t total = q.shape[0], heads = q.shape[1];
  if ((a[6] != Py_None && !read_rows(dev, a[6], "mask", kI64, kI64, total, (static_cast<int64_t>(d.max_q) + 63) / 64, &mask)) ||
      (a[7] != Py_None && !read_flat(dev, a[7], "depth", kI32, total, &depth)) || !read_int32(a[8], "window", &d.window) ||
      (a[10] != Py_None && !read_heads(dev, a[10], "out", total, heads, c.c.head_dim, &out)))
    return nullptr;
  const double scale = a[9] == Py_None ? 1.0 / sqrt(static_cast<double>(c.c.head_dim)) : PyFloat_AsDouble(a[9]);
  const int with_lse = PyObject_IsTrue(a[12]);
  if (PyErr_Occurred()) return nullptr;
  if (a[11] != Py_None) {
    if (!read(dev, a[11], "lse", kF32, kF32, 2, &lse)) return nullptr;
    if (lse.shape[0] != total || lse.shape[1] != heads || !contiguous(lse)) {
      PyErr_Format(PyExc_ValueError, "lse: expected a contiguous [%lld, %lld] tensor", static_cast<long long>(total), static_cast<long long>(heads));
      return nullptr;
    }
  }
  if ((a[13] != Py_None && !read_flat(dev, a[13], "workspace", kU8, -1, &ws)) || !st.read_from(a[14], q)) return nullptr;
  d.batch = small(table.shape[0]);
  d.total_q = total;
  d.cu_q = static_cast<const int32_t*>(cu.ptr);
  d.ctx = static_cast<const int32_t*>(ctx.ptr);
  d.page_table = static_cast<const int32_t*>(table.ptr);
  d.pages_per_seq = small(table.shape[1]);
  d.ld_table = table.stride[0];
  d.mask = static_cast<const uint64_t*>(mask.ptr);
  d.ld_mask = mask.stride[0];
  d.depth = static_cast<const int32_t*>(depth.ptr);
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made_out, made_lse, made_ws;
  if (a[10] == Py_None) {
    made_out = like(q);
    take(made_out, &out);
    if (!head_strides("out", &out)) return nullptr;
  }
  if (a[11] == Py_None && with_lse) {
    made_lse = fresh({total, heads}, kF32, q);
    take(made_lse, &lse);
  }
  if (a[13] == Py_None) {
    const size_t need = f_attention_bytes(&c.c, &d, small(heads));
    if (need == static_cast<size_t>(-1)) {
      ok(AQ_ERR_INVALID_ARG);
      return nullptr;
    }
    if (need) {
      made_ws = fresh({static_cast<int64_t>(need)}, kU8, q);
      take(made_ws, &ws);
    }
  }
  if (!on_gpu(dev) || !ok(f_attention(&c.c, &d, q.ptr, small(heads), q.stride[0], q.stride[1], static_cast<float>(scale), out.ptr, out.stride[0], out.stride[1],
                      static_cast<float*>(lse.ptr), ws.ptr, static_cast<size_t>(ws.shape[0]), st.handle)))
    return nullptr;
  PyObject* o = made_out.defined() ? st.hand_out(std::move(made_out)) : given(a[10]);
  if (!with_lse) return o;
  return pack({o, made_lse.defined() ? st.hand_out(std::move(made_lse)) : given(a[11])});
  END_HANDLE_TH_ERRORS
}

// verify(p, tokens, cu, u, noise, q, parent, path_cap, max_nodes, stream) -> (n_accepted, path, token)
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Tensor p, tokens, cu, u, noise, q, parent, count, path, token;
  int32_t cap = AQ_MAX_DRAFT_NODES, most = AQ_MAX_DRAFT_NODES;
  Stream st;
  if (!want(n, 10, "verify") || !read_rows(dev, a[0], "p", kF32, kBf16, -1, 0, &p) || !read_flat(dev, a[1], "tokens", kI32, -1, &tokens) ||
      !read_flat(dev, a[2], "cu", kI32, -1, &cu) || !read_flat(dev, a[3], "u", kF32, tokens.shape[0], &u))
    return nullptr;
  const int64_t nodes = tokens.shape[0], batch = cu.shape[0] - 1, vocab = p.shape[1];
  const at::ScalarType dtype = p.t->scalar_type();
  if (batch < 0) {
    PyErr_SetString(PyExc_ValueError, "cu: expected [batch + 1] elements");
    return nullptr;
  }
  const bool sampled = a[5] != Py_None;
  if (!read_rows(dev, a[4], "noise", kF32, kF32, batch, vocab, &noise) || (sampled && !read_rows(dev, a[5], "q", dtype, dtype, p.shape[0], vocab, &q)))
    return nullptr;
  if (noise.shape[1] != vocab || (sampled && q.shape[1] != vocab)) {
    PyErr_Format(PyExc_ValueError, "noise and q: expected %lld columns", static_cast<long long>(vocab));
    return nullptr;
  }
  if (nodes < cap) cap = most = static_cast<int32_t>(nodes);
  if ((a[6] != Py_None && !read_flat(dev, a[6], "parent", kI32, nodes, &parent)) || (a[7] != Py_None && !read_int32(a[7], "path_cap", &cap)) ||
      (a[8] != Py_None && !read_int32(a[8], "max_nodes", &most)) || !st.read_from(a[9], p))
    return nullptr;
  if (cap < 0) {
    PyErr_Format(PyExc_ValueError, "path_cap=%d is negative", cap);
    return nullptr;
  }
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made[3] = {fresh({batch}, kI32, p), fresh({batch, cap}, kI32, p), fresh({batch}, kI32, p)};
  take(made[0], &count);
  take(made[1], &path);
  take(made[2], &token);
  if (!on_gpu(dev) || !ok(f_verify(small(batch), small(vocab), static_cast<const int32_t*>(cu.ptr), static_cast<const int32_t*>(tokens.ptr),
                   static_cast<const int32_t*>(parent.ptr), nodes, most, p.ptr, p.stride[0], q.ptr, q.stride[0], p.shape[0],
                   dtype == kF32 ? AQ_PROB_F32 : AQ_PROB_BF16, static_cast<const float*>(u.ptr), static_cast<const float*>(noise.ptr), noise.stride[0],
                   static_cast<int32_t*>(count.ptr), static_cast<int32_t*>(path.ptr), cap, cap, static_cast<int32_t*>(token.ptr), st.handle)))
    return nullptr;
  return pack({st.hand_out(std::move(made[0])), st.hand_out(std::move(made[1])), st.hand_out(std::move(made[2]))});
  END_HANDLE_TH_ERRORS
}

// bind((addresses of the entry points), check)
PyObject* py_bind(PyObject*, PyObject* args) {
  unsigned long long f[6];
  PyObject* check;
  if (!PyArg_ParseTuple(args, "(KKKKKK)O", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &check)) return nullptr;
  auto set = [](auto& to, unsigned long long at) { to = reinterpret_cast<std::decay_t<decltype(to)>>(static_cast<uintptr_t>(at)); };
  set(f_rope, f[0]);
  set(f_kv_write, f[1]);
  set(f_kv_read, f[2]);
  set(f_attention_bytes, f[3]);
  set(f_attention, f[4]);
  set(f_verify, f[5]);
  Py_INCREF(check);
  f_check = check;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rope), FAST(kv_write), FAST(kv_read), FAST(attention_bytes), FAST(attention), FAST(verify),
                         {"bind", py_bind, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_freq, "freq"}, {&s_layout, "layout"}, {&s_magnitude, "magnitude"}, {&s_k, "k"}, {&s_v, "v"}, {&s_k_scale, "k_scale"}, {&s_v_scale, "v_scale"}};
  for (auto& n : names)
    if (!(*n.to = PyUnicode_InternFromString(n.name))) return nullptr;
  return PyModule_Create(&module);
}

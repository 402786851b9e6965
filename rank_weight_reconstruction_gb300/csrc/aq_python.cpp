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

#include <ATen/Context.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/TensorImpl.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
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
decltype(&aq_kv_read) f_kv_read;
decltype(&aq_tree_attention_workspace_bytes) f_attention_bytes;
decltype(&aq_tree_attention) f_attention;
decltype(&aq_verify_drafts) f_verify;
decltype(&aq_kv_write_norm) f_kv_write_norm;
decltype(&aq_qk_norm_rope) f_norm;
decltype(&aq_qk_norm_rope_backward_workspace_bytes) f_norm_bytes;
decltype(&aq_qk_norm_rope_backward) f_norm_backward;
decltype(&aq_nvfp4_linear_multi) f_nvfp4;
decltype(&aq_token_logprobs) f_scores;
decltype(&aq_token_logprobs_backward) f_scores_backward;
PyObject* f_check;   // raises for a status that is not AQ_OK

PyObject *s_freq, *s_layout, *s_magnitude, *s_k, *s_v, *s_k_scale, *s_v_scale, *s_weight, *s_eps, *s_offset, *s_q, *s_sf, *s_global_scale;

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

// A dimension as the ABI takes it; more than 32 bits hold is an error (of the calls' own handling), not fewer of them.
int32_t dim32(int64_t v, const char* name) {
  TORCH_CHECK_VALUE(v <= INT32_MAX, name, ": ", v, " are more than 32 bits hold");
  return static_cast<int32_t>(v);
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
  dim32(x->shape[1], name), dim32(x->shape[2], name);
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

bool read_float(PyObject* obj, float* out) {
  *out = static_cast<float>(PyFloat_AsDouble(obj));
  return !PyErr_Occurred();
}

// A HeadNorm over heads of `dim`, or None.
struct Norm {
  PyObject* weight = nullptr;
  Tensor w;
  aq_head_norm n = {};
  bool given = false;
  ~Norm() { Py_XDECREF(weight); }
  const aq_head_norm* c() const { return given ? &n : nullptr; }
  bool read_from(Device& dev, PyObject* obj, int64_t dim) {
    if (obj == Py_None) return true;
    given = true;
    weight = PyObject_GetAttr(obj, s_weight);
    Ref eps(PyObject_GetAttr(obj, s_eps)), offset(PyObject_GetAttr(obj, s_offset));
    if (!weight || !eps.o || !offset.o || !read_float(eps.o, &n.eps) || !read_float(offset.o, &n.offset)) return false;
    if (weight == Py_None) return true;
    if (!read_flat(dev, weight, "HeadNorm.weight", kBf16, dim, &w)) return false;
    n.weight = w.ptr;
    return true;
  }
};

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
    c.pages = dim32(t[0].shape[0], "KvCache pages");
    c.kv_heads = dim32(t[0].shape[1], "KvCache kv_heads");
    c.page_size = dim32(t[0].shape[2], "KvCache page_size");
    c.head_dim = dim32(t[0].shape[3], "KvCache head_dim");
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

// Whether someone asks to see allocations or to have them filled: a dispatch mode is on, or new memory is to be deterministic.
bool watched() {
  return c10::impl::TorchDispatchModeTLS::any_modes_set() ||
         (at::globalContext().deterministicAlgorithms() && at::globalContext().deterministicFillUninitializedMemory());
}
// A new tensor on the given one's device, from the current stream's memory: what at::empty does there, without the way through the
// dispatcher (0.5 us where at::empty takes 1.4) unless that would be missed.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& on) {
  if (!on.t->is_cuda() || watched()) return at::empty(shape, at::TensorOptions().dtype(dtype).device(on.t->device()));
  int64_t bytes = static_cast<int64_t>(c10::elementSize(dtype));
  for (const int64_t n : shape) bytes *= n;
  c10::Allocator* const memory = c10::cuda::CUDACachingAllocator::get();
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(c10::Storage::use_byte_size_t(), static_cast<size_t>(bytes), memory->allocate(static_cast<size_t>(bytes)), memory, true),
      c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(dtype));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}
// A part of a contiguous tensor's storage, elements of the same size from `first` on.
at::Tensor part(const at::Tensor& of, int64_t first, at::IntArrayRef shape, at::ScalarType dtype) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(dtype));
  t.unsafeGetTensorImpl()->set_storage_offset(first);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}
// As at::empty_like: the same order of strides.
at::Tensor like(const Tensor& x) {
  bool falling = true;
  for (int i = 1; i < x.nd; ++i) falling = falling && x.t->stride(i - 1) >= x.t->stride(i);
  return falling && x.t->is_cuda() && !watched() ? fresh(x.t->sizes(), x.t->scalar_type(), x) : at::empty_like(*x.t);
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
  if (!on_gpu(dev) || !ok(f_rope(&r.spec, static_cast<const int32_t*>(pos.ptr), x.shape[0], dim32(x.shape[1], "heads"), dim32(x.shape[2], "head_dim"), x.ptr, x.stride[0], x.stride[1],
                 y.ptr, y.stride[0], y.stride[1], inverse, st.handle)))
    return nullptr;
  return made.defined() ? st.hand_out(std::move(made)) : given(a[3]);
  END_HANDLE_TH_ERRORS
}

// kv_write(cache, k, v, slots, rope, pos, q, q_out, q_norm, k_norm, stream) -> q_out
PyObject* py_kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Cache c;
  Rope r;
  Norm qn, kn;
  Tensor k, v, slots, pos, q, o;
  Stream st;
  if (!want(n, 11, "kv_write") || !c.read_from(dev, a[0]) || !read_heads(dev, a[1], "k", -1, c.c.kv_heads, c.c.head_dim, &k)) return nullptr;
  const int64_t T = k.shape[0];
  const bool turned = a[4] != Py_None, queries = a[6] != Py_None;
  if (!read_heads(dev, a[2], "v", T, c.c.kv_heads, c.c.head_dim, &v) || !read_flat(dev, a[3], "slots", kI64, T, &slots) || (turned && !r.read_from(dev, a[4])) ||
      (a[5] != Py_None && !read_flat(dev, a[5], "pos", kI32, T, &pos)) || (queries && !read_heads(dev, a[6], "q", T, -1, c.c.head_dim, &q)) ||
      (queries && a[7] != Py_None && !read_heads(dev, a[7], "q_out", T, q.shape[1], c.c.head_dim, &o)) || !qn.read_from(dev, a[8], c.c.head_dim) ||
      !kn.read_from(dev, a[9], c.c.head_dim) || !st.read_from(a[10], k))
    return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made;
  if (queries && a[7] == Py_None) {
    made = like(q);
    take(made, &o);
    if (!head_strides("q_out", &o)) return nullptr;
  }
  if (!on_gpu(dev) || !ok(f_kv_write_norm(&c.c, static_cast<const int64_t*>(slots.ptr), T, k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1],
                     turned ? &r.spec : nullptr, static_cast<const int32_t*>(pos.ptr), q.ptr, dim32(q.shape[1], "q heads"), q.stride[0], q.stride[1], o.ptr,
                     o.stride[0], o.stride[1], qn.c(), kn.c(), st.handle)))
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
  d.batch = dim32(table.shape[0], "batch");
  d.total_q = total;
  d.cu_q = static_cast<const int32_t*>(cu.ptr);
  d.ctx = static_cast<const int32_t*>(ctx.ptr);
  d.page_table = static_cast<const int32_t*>(table.ptr);
  d.pages_per_seq = dim32(table.shape[1], "pages of a sequence");
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
    const size_t need = f_attention_bytes(&c.c, &d, dim32(heads, "q heads"));
    if (need == static_cast<size_t>(-1)) {
      ok(AQ_ERR_INVALID_ARG);
      return nullptr;
    }
    if (need) {
      made_ws = fresh({static_cast<int64_t>(need)}, kU8, q);
      take(made_ws, &ws);
    }
  }
  if (!on_gpu(dev) || !ok(f_attention(&c.c, &d, q.ptr, dim32(heads, "q heads"), q.stride[0], q.stride[1], static_cast<float>(scale), out.ptr, out.stride[0], out.stride[1],
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
  if (!on_gpu(dev) || !ok(f_verify(dim32(batch, "batch"), dim32(vocab, "vocab"), static_cast<const int32_t*>(cu.ptr), static_cast<const int32_t*>(tokens.ptr),
                   static_cast<const int32_t*>(parent.ptr), nodes, most, p.ptr, p.stride[0], q.ptr, q.stride[0], p.shape[0],
                   dtype == kF32 ? AQ_PROB_F32 : AQ_PROB_BF16, static_cast<const float*>(u.ptr), static_cast<const float*>(noise.ptr), noise.stride[0],
                   static_cast<int32_t*>(count.ptr), static_cast<int32_t*>(path.ptr), cap, cap, static_cast<int32_t*>(token.ptr), st.handle)))
    return nullptr;
  return pack({st.hand_out(std::move(made[0])), st.hand_out(std::move(made[1])), st.hand_out(std::move(made[2]))});
  END_HANDLE_TH_ERRORS
}

aq_heads heads_of(const Tensor& x) { return {x.ptr, x.stride[0], x.stride[1], dim32(x.shape[1], "heads")}; }

// qk_norm_rope(q, k, q_norm, k_norm, rope, pos, q_out, k_out, stream) -> (q_out, k_out)
PyObject* py_qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Rope r;
  Norm norm[2];
  Tensor pos, x[2], y[2];
  Stream st;
  if (!want(n, 9, "qk_norm_rope") || !read_heads(dev, a[0], "q", -1, -1, -1, &x[0])) return nullptr;
  const int64_t T = x[0].shape[0], D = x[0].shape[2];
  const int sets = a[1] == Py_None ? 1 : 2;
  const bool turned = a[4] != Py_None;
  if ((sets == 2 && !read_heads(dev, a[1], "k", T, -1, D, &x[1])) || !norm[0].read_from(dev, a[2], D) || !norm[1].read_from(dev, a[3], D) ||
      (turned && !r.read_from(dev, a[4])) || (a[5] != Py_None && !read_flat(dev, a[5], "pos", kI32, T, &pos)))
    return nullptr;
  const char* const name[2] = {"q_out", "k_out"};
  for (int i = 0; i < sets; ++i)
    if (a[6 + i] != Py_None && !read_heads(dev, a[6 + i], name[i], T, x[i].shape[1], D, &y[i])) return nullptr;
  if (!st.read_from(a[8], x[0])) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made[2];
  for (int i = 0; i < sets; ++i)
    if (a[6 + i] == Py_None) {
      made[i] = like(x[i]);
      take(made[i], &y[i]);
      if (!head_strides(name[i], &y[i])) return nullptr;
    }
  const aq_heads q = heads_of(x[0]), k = heads_of(x[1]), qo = heads_of(y[0]), ko = heads_of(y[1]);
  if (!on_gpu(dev) || !ok(f_norm(norm[0].c(), norm[1].c(), turned ? &r.spec : nullptr, static_cast<const int32_t*>(pos.ptr), T, dim32(D, "head_dim"), &q, &qo,
                                 sets == 2 ? &k : nullptr, sets == 2 ? &ko : nullptr, st.handle)))
    return nullptr;
  PyObject* out[2];
  for (int i = 0; i < 2; ++i) out[i] = i < sets && made[i].defined() ? st.hand_out(std::move(made[i])) : given(i < sets ? a[6 + i] : Py_None);
  return pack({out[0], out[1]});
  END_HANDLE_TH_ERRORS
}

// qk_norm_rope_backward(dq_out, dk_out, q, k, q_norm, k_norm, rope, pos, dq, dk, workspace, stream) -> (dq, dk, dq_weight, dk_weight)
PyObject* py_qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Rope r;
  Norm norm[2];
  Tensor pos, dy[2], x[2], dx[2], ws;
  Stream st;
  if (!want(n, 12, "qk_norm_rope_backward") || !read_heads(dev, a[2], "q", -1, -1, -1, &x[0])) return nullptr;
  const int64_t T = x[0].shape[0], D = x[0].shape[2];
  const int sets = a[3] == Py_None ? 1 : 2;
  const bool turned = a[6] != Py_None;
  const char* const names[2][2] = {{"dq_out", "dq"}, {"dk_out", "dk"}};
  if ((sets == 2 && !read_heads(dev, a[3], "k", T, -1, D, &x[1])) || !norm[0].read_from(dev, a[4], D) || !norm[1].read_from(dev, a[5], D) ||
      (turned && !r.read_from(dev, a[6])) || (a[7] != Py_None && !read_flat(dev, a[7], "pos", kI32, T, &pos)) ||
      (a[10] != Py_None && !read_flat(dev, a[10], "workspace", kU8, -1, &ws)))
    return nullptr;
  if (!norm[0].given || (sets == 2) != norm[1].given || (sets == 2) != (a[1] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, "q comes with q_norm, and k, k_norm and dk_out together");
    return nullptr;
  }
  for (int i = 0; i < sets; ++i)
    if (!read_heads(dev, a[i], names[i][0], T, x[i].shape[1], D, &dy[i]) || (a[8 + i] != Py_None && !read_heads(dev, a[8 + i], names[i][1], T, x[i].shape[1], D, &dx[i])))
      return nullptr;
  if (!st.read_from(a[11], x[0])) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made[2], made_w[2], made_ws;
  float* dw[2] = {nullptr, nullptr};
  for (int i = 0; i < sets; ++i) {
    if (a[8 + i] == Py_None) {
      made[i] = like(x[i]);
      take(made[i], &dx[i]);
      if (!head_strides(names[i][1], &dx[i])) return nullptr;
    }
    if (norm[i].n.weight) {
      made_w[i] = fresh({D}, kF32, x[0]);
      dw[i] = static_cast<float*>(made_w[i].data_ptr());
    }
  }
  if (a[10] == Py_None && (dw[0] || dw[1])) {
    const size_t need = f_norm_bytes(T, dim32(D, "head_dim"), dim32(x[0].shape[1], "q heads"), sets == 2 ? dim32(x[1].shape[1], "k heads") : 0);
    if (need == static_cast<size_t>(-1)) {
      ok(AQ_ERR_INVALID_ARG);
      return nullptr;
    }
    made_ws = fresh({static_cast<int64_t>(need)}, kU8, x[0]);
    take(made_ws, &ws);
  }
  aq_heads h[2][3];
  for (int i = 0; i < 2; ++i) {
    h[i][0] = heads_of(dy[i]);
    h[i][1] = heads_of(x[i]);
    h[i][2] = heads_of(dx[i]);
  }
  const bool two = sets == 2;
  if (!on_gpu(dev) || !ok(f_norm_backward(norm[0].c(), norm[1].c(), turned ? &r.spec : nullptr, static_cast<const int32_t*>(pos.ptr), T, dim32(D, "head_dim"), &h[0][0],
                                          &h[0][1], &h[0][2], dw[0], two ? &h[1][0] : nullptr, two ? &h[1][1] : nullptr, two ? &h[1][2] : nullptr, dw[1], ws.ptr,
                                          static_cast<size_t>(ws.shape[0]), st.handle)))
    return nullptr;
  PyObject* out[4];
  for (int i = 0; i < 2; ++i) {
    out[i] = made[i].defined() ? st.hand_out(std::move(made[i])) : given(i < sets ? a[8 + i] : Py_None);
    out[2 + i] = made_w[i].defined() ? st.hand_out(std::move(made_w[i])) : given(Py_None);
  }
  return pack({out[0], out[1], out[2], out[3]});
  END_HANDLE_TH_ERRORS
}

// An Nvfp4Weight.
struct Weight4 {
  PyObject *q = nullptr, *sf = nullptr, *g = nullptr;
  aq_nvfp4_weight w = {};
  ~Weight4() {
    Py_XDECREF(q);
    Py_XDECREF(sf);
    Py_XDECREF(g);
  }
  bool read_from(Device& dev, PyObject* obj) {
    Tensor t, one;
    q = PyObject_GetAttr(obj, s_q);
    sf = PyObject_GetAttr(obj, s_sf);
    g = PyObject_GetAttr(obj, s_global_scale);
    Ref layout(PyObject_GetAttr(obj, s_layout));
    if (!q || !sf || !g || !layout.o || !read_int32(layout.o, "layout", &w.sf_layout) || !read_rows(dev, q, "Nvfp4Weight.q", kU8, kU8, -1, 0, &t) ||
        !read(dev, g, "Nvfp4Weight.global_scale", kF32, kF32, 1, &one))
      return false;
    if (one.shape[0] != 1) {
      PyErr_SetString(PyExc_ValueError, "Nvfp4Weight.global_scale: expected one element");
      return false;
    }
    w.q = t.ptr;
    w.ldq = t.stride[0];
    w.out = dim32(t.shape[0], "Nvfp4Weight.q rows");
    w.in = dim32(2 * t.shape[1], "Nvfp4Weight.q columns");
    w.global_scale = static_cast<const float*>(one.ptr);
    const int64_t cols = t.shape[1] / 8;
    const int64_t need = w.sf_layout == AQ_SF_128X4 ? (t.shape[0] + 127) / 128 * 128 * ((cols + 3) / 4 * 4) : t.shape[0] * cols;
    Tensor s;
    const bool flat = THPVariable_Check(sf) && THPVariable_Unpack(sf).dim() == 1;
    if (!read(dev, sf, "Nvfp4Weight.sf", kU8, kU8, flat ? 1 : 2, &s)) return false;
    if (!contiguous(s) || (flat ? s.shape[0] : s.shape[0] * s.shape[1]) != need) {
      PyErr_Format(PyExc_ValueError, "Nvfp4Weight.sf: expected a contiguous tensor of %lld elements", static_cast<long long>(need));
      return false;
    }
    w.sf = s.ptr;
    return true;
  }
};

// nvfp4_linear(weights, x, ys, stream) -> [y, ...]
PyObject* py_nvfp4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Weight4 w[AQ_MAX_FAMILIES];
  Tensor x, y[AQ_MAX_FAMILIES];
  Stream st;
  if (!want(n, 4, "nvfp4_linear")) return nullptr;
  Ref list(PySequence_Fast(a[0], "weights: expected a sequence of Nvfp4Weight")), outs(a[2] == Py_None ? nullptr : PySequence_Fast(a[2], "ys: expected a sequence of tensors"));
  if (!list.o || (a[2] != Py_None && !outs.o)) return nullptr;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(list.o);
  if (count < 1 || count > AQ_MAX_FAMILIES || (outs.o && PySequence_Fast_GET_SIZE(outs.o) != count)) {
    PyErr_Format(PyExc_ValueError, "expected one to %d weights, and as many ys", AQ_MAX_FAMILIES);
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < count; ++i)
    if (!w[i].read_from(dev, PySequence_Fast_GET_ITEM(list.o, i))) return nullptr;
  if (!read_rows(dev, a[1], "x", kBf16, kBf16, -1, 0, &x)) return nullptr;
  if (x.shape[1] != w[0].w.in) {
    PyErr_Format(PyExc_ValueError, "x: expected %d columns, got %lld", w[0].w.in, static_cast<long long>(x.shape[1]));
    return nullptr;
  }
  const int64_t M = x.shape[0];
  for (Py_ssize_t i = 0; outs.o && i < count; ++i) {
    if (!read_rows(dev, PySequence_Fast_GET_ITEM(outs.o, i), "y", kBf16, kBf16, M, w[i].w.out, &y[i])) return nullptr;
    if (y[i].shape[1] != w[i].w.out) {
      PyErr_Format(PyExc_ValueError, "y: expected %d columns, got %lld", w[i].w.out, static_cast<long long>(y[i].shape[1]));
      return nullptr;
    }
  }
  if (!st.read_from(a[3], x)) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made[AQ_MAX_FAMILIES];
  aq_nvfp4_weight cw[AQ_MAX_FAMILIES];
  void* yp[AQ_MAX_FAMILIES];
  int64_t ldy[AQ_MAX_FAMILIES];
  for (Py_ssize_t i = 0; i < count; ++i) {
    if (!outs.o) {
      made[i] = fresh({M, w[i].w.out}, kBf16, x);
      take(made[i], &y[i]);
    }
    cw[i] = w[i].w;
    yp[i] = y[i].ptr;
    ldy[i] = y[i].stride[0];
  }
  if (!on_gpu(dev) || !ok(f_nvfp4(cw, static_cast<int32_t>(count), x.ptr, M, x.stride[0], yp, ldy, st.handle))) return nullptr;
  Ref result(PyList_New(count));
  if (!result.o) return nullptr;
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject* o = made[i].defined() ? st.hand_out(std::move(made[i])) : given(PySequence_Fast_GET_ITEM(outs.o, i));
    if (!o) return nullptr;
    PyList_SET_ITEM(result.o, i, o);
  }
  return given(result.o);
  END_HANDLE_TH_ERRORS
}

// scores(logits, tokens, scale, top, stream) -> (logprob, lse, entropy, top_logprob, top_token)
PyObject* py_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Tensor x, tokens;
  float scale;
  int32_t top;
  Stream st;
  if (!want(n, 5, "scores") || !read_rows(dev, a[0], "logits", kF32, kBf16, -1, 0, &x) || (a[1] != Py_None && !read_flat(dev, a[1], "tokens", kI32, x.shape[0], &tokens)) ||
      !read_float(a[2], &scale) || !read_int32(a[3], "top", &top) || !st.read_from(a[4], x))
    return nullptr;
  if (top < 0 || top > AQ_MAX_TOP) {
    PyErr_Format(PyExc_ValueError, "top=%d outside [0, %d]", top, AQ_MAX_TOP);
    return nullptr;
  }
  if (!on_gpu(dev)) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  const int64_t rows = x.shape[0];
  // one allocation: [rows] three times (twice without tokens), then [rows, top] twice
  at::Tensor made[5];
  const bool scored = a[1] != Py_None;
  const int64_t words = rows * ((scored ? 3 : 2) + 2 * static_cast<int64_t>(top));
  const at::Tensor all = fresh({words}, kF32, x);
  int64_t first = 0;
  for (int i = scored ? 0 : 1; i < (top ? 5 : 3); ++i) {
    made[i] = i < 3 ? part(all, first, {rows}, kF32) : part(all, first, {rows, top}, i == 3 ? kF32 : kI32);
    first += i < 3 ? rows : rows * top;
  }
  auto f32 = [&](int i) { return made[i].defined() ? static_cast<float*>(made[i].data_ptr()) : nullptr; };
  if (!ok(f_scores(x.ptr, x.stride[0], rows, dim32(x.shape[1], "vocab"), x.t->scalar_type() == kF32 ? AQ_PROB_F32 : AQ_PROB_BF16, static_cast<const int32_t*>(tokens.ptr), scale,
                   f32(0), f32(1), f32(2), top, f32(3), top ? static_cast<int32_t*>(made[4].data_ptr()) : nullptr, st.handle)))
    return nullptr;
  PyObject* out[5];
  for (int i = 0; i < 5; ++i) out[i] = made[i].defined() ? st.hand_out(std::move(made[i])) : given(Py_None);
  return pack({out[0], out[1], out[2], out[3], out[4]});
  END_HANDLE_TH_ERRORS
}

// scores_backward(logits, tokens, lse, entropy, dlogprob, dentropy, dlse, scale, dlogits, stream) -> dlogits
PyObject* py_scores_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Device dev;
  Tensor x, tokens, side[5], out;   // side: lse, entropy, dlogprob, dentropy, dlse
  float scale;
  Stream st;
  if (!want(n, 10, "scores_backward") || !read_rows(dev, a[0], "logits", kF32, kBf16, -1, 0, &x)) return nullptr;
  const int64_t rows = x.shape[0];
  const char* const names[5] = {"lse", "entropy", "dlogprob", "dentropy", "dlse"};
  const at::ScalarType dtype = x.t->scalar_type();
  if (a[1] != Py_None && !read_flat(dev, a[1], "tokens", kI32, rows, &tokens)) return nullptr;
  for (int i = 0; i < 5; ++i)
    if (a[2 + i] != Py_None && !read_flat(dev, a[2 + i], names[i], kF32, rows, &side[i])) return nullptr;
  if (!read_float(a[7], &scale) || (a[8] != Py_None && !read_rows(dev, a[8], "dlogits", dtype, dtype, rows, x.shape[1], &out)) || !st.read_from(a[9], x)) return nullptr;
  if (a[8] != Py_None && out.shape[1] != x.shape[1]) {
    PyErr_Format(PyExc_ValueError, "dlogits: expected %lld columns", static_cast<long long>(x.shape[1]));
    return nullptr;
  }
  if (!on_gpu(dev)) return nullptr;
  at::AutoDispatchBelowADInplaceOrView plain;
  at::Tensor made;
  if (a[8] == Py_None) {
    made = like(x);   // rows as the logits have them, where those are not spread out
    take(made, &out);
    if (rows <= 1) out.stride[0] = x.shape[1];
  }
  auto f32 = [&](int i) { return static_cast<const float*>(side[i].ptr); };
  // tokens matter to the gradient of logprob alone
  if (!ok(f_scores_backward(x.ptr, x.stride[0], rows, dim32(x.shape[1], "vocab"), dtype == kF32 ? AQ_PROB_F32 : AQ_PROB_BF16,
                            side[2].ptr ? static_cast<const int32_t*>(tokens.ptr) : nullptr, scale, f32(0), f32(1), f32(2), f32(3), f32(4), out.ptr, out.stride[0], st.handle)))
    return nullptr;
  return made.defined() ? st.hand_out(std::move(made)) : given(a[8]);
  END_HANDLE_TH_ERRORS
}

// bind((addresses of the entry points), check)
PyObject* py_bind(PyObject*, PyObject* args) {
  unsigned long long f[12];
  PyObject* check;
  if (!PyArg_ParseTuple(args, "(KKKKKKKKKKKK)O", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9], &f[10], &f[11], &check)) return nullptr;
  auto set = [](auto& to, unsigned long long at) { to = reinterpret_cast<std::decay_t<decltype(to)>>(static_cast<uintptr_t>(at)); };
  set(f_rope, f[0]);
  set(f_kv_write_norm, f[1]);
  set(f_kv_read, f[2]);
  set(f_attention_bytes, f[3]);
  set(f_attention, f[4]);
  set(f_verify, f[5]);
  set(f_norm, f[6]);
  set(f_norm_bytes, f[7]);
  set(f_norm_backward, f[8]);
  set(f_nvfp4, f[9]);
  set(f_scores, f[10]);
  set(f_scores_backward, f[11]);
  Py_INCREF(check);
  f_check = check;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rope), FAST(kv_write), FAST(kv_read), FAST(attention_bytes), FAST(attention), FAST(verify),
                         FAST(qk_norm_rope), FAST(qk_norm_rope_backward), FAST(nvfp4_linear), FAST(scores), FAST(scores_backward),
                         {"bind", py_bind, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_freq, "freq"}, {&s_layout, "layout"}, {&s_magnitude, "magnitude"}, {&s_k, "k"}, {&s_v, "v"}, {&s_k_scale, "k_scale"}, {&s_v_scale, "v_scale"},
               {&s_weight, "weight"}, {&s_eps, "eps"}, {&s_offset, "offset"}, {&s_q, "q"}, {&s_sf, "sf"}, {&s_global_scale, "global_scale"}};
  for (auto& n : names)
    if (!(*n.to = PyUnicode_InternFromString(n.name))) return nullptr;
  return PyModule_Create(&module);
}

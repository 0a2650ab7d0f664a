// mnw_calls.cpp -- the calls on a paged cache and the adapters from Python, in
// C++: checks of the tensors, results, scratch memory and the C call in one.
//
// A call of one token is bound by the host.  Of the 19 us that an attention call
// took through ctypes the launch is 2; checking some 15 tensors attribute by
// attribute, two results by torch.empty and the conversion of 28 arguments were
// the rest.  Here it takes 5.8 (two results 2.6, scratch 0.5, launch and all else
// 2.7); an adapters' call 2.5 for 10; an append and two values' calls 6.9 for 21.
//
// Each function takes the Python function's arguments (all but the stream: the
// current one's) and returns its result; the status as an int where the C call
// refuses; or NotImplemented where anything is not as it has to be, or not
// plain (a subclass), or where any tensor is on another device than the current
// one, without having done anything: the Python function then goes on by itself
// and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <initializer_list>

#include "mnw_moe.h"

namespace {

// The library's functions, as loaded by the package.
struct Library {
  decltype(&mnw_kv_append) kv_append;
  decltype(&mnw_attn_paged) attn_paged;
  decltype(&mnw_attn_paged_workspace_size) attn_paged_workspace_size;
  decltype(&mnw_kv_values) kv_values;
  decltype(&mnw_lora_add) lora_add;
  decltype(&mnw_lora_workspace_size) lora_workspace_size;
} lib;

struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// Scratch memory of a call: given back behind its launches, so the next user on that stream comes after them.
struct Scratch {
  void* p = nullptr;
  Scratch(size_t bytes, cudaStream_t st) {
    if (bytes) p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, st);
  }
  ~Scratch() {
    if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
};

// The current device, looked up once a call, at its first CUDA tensor.  (One for all threads: it is used with the
// interpreter's lock held, and no Python code runs between a call's beginning and current_stream().)
int device_now = -1;
// The plain CUDA tensor of that device behind an argument, or null.  Every tensor of a call comes through here.
const at::Tensor* cuda(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided) return nullptr;
  if (device_now < 0) device_now = c10::cuda::current_device();
  return t.get_device() == device_now ? &t : nullptr;
}
// A contiguous one of the given type and shape; *p its address, null for None where that may be.
bool whole(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, void** p, bool may_be_none = false) {
  *p = nullptr;
  if (o == Py_None) return may_be_none;
  const at::Tensor* t = cuda(o);
  if (!t || t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  return true;
}
// The error word: the first four bytes of any CUDA tensor that has them, or None.
bool word(PyObject* o, uint32_t** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = cuda(o);
  if (!t || (t->numel() > 0 && t->numel() * t->itemsize() < 4)) return false;
  *p = static_cast<uint32_t*>(t->data_ptr());
  return (reinterpret_cast<uintptr_t>(*p) & 3) == 0;
}
// A workspace given by the caller, contiguous (its elements are the bytes that may be written), or None.
bool workspace(PyObject* o, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = cuda(o);
  if (!t || t->scalar_type() != at::kByte || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  *bytes = static_cast<size_t>(t->numel());
  return true;
}
bool integer(PyObject* o, int* v) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long x = PyLong_AsLongAndOverflow(o, &over);
  *v = static_cast<int>(x);
  return !over && x >= INT_MIN && x <= INT_MAX;
}
bool real(PyObject* o, float* v) {
  if (PyFloat_Check(o)) {
    *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
    return true;
  }
  int i;
  if (!integer(o, &i)) return false;
  *v = static_cast<float>(i);
  return true;
}
bool fits(std::initializer_list<int64_t> sizes) {
  return std::all_of(sizes.begin(), sizes.end(), [](int64_t n) { return n <= INT_MAX; });
}

// bf16 [T, heads, d], a token's heads contiguous
struct Tokens {
  void* p = nullptr;
  int64_t T = 0, h = 0, d = 0, stride = 0;
  bool read(const at::Tensor* t, int64_t want_d) {
    if (!t || t->scalar_type() != at::kBFloat16 || t->dim() != 3) return false;
    T = t->size(0);
    h = t->size(1);
    d = t->size(2);
    if (d != want_d || (t->stride(2) != 1 && d > 1) || (h > 1 && t->stride(1) != d)) return false;
    stride = T > 1 ? t->stride(0) : std::max(h * d, t->stride(0) / 8 * 8);
    p = t->data_ptr();
    return fits({T, h});
  }
};

// bf16 [T, n], rows contiguous
struct Rows {
  void* p = nullptr;
  int64_t T = 0, n = 0, stride = 0;
  bool read(const at::Tensor* t) {
    if (!t || t->scalar_type() != at::kBFloat16 || t->dim() != 2) return false;
    T = t->size(0);
    n = t->size(1);
    if (t->stride(1) != 1 && n > 1) return false;
    stride = T > 1 ? t->stride(0) : std::max(n, t->stride(0) / 8 * 8);
    p = t->data_ptr();
    return fits({T, n});
  }
};

// [n_pages, Hkv, page_size, d] with its scales or records
struct Pages {
  int fmt = 0;
  int64_t n = 0, h = 0, page = 0, d = 0, stride = 0;
  bool read(const at::Tensor* t) {
    if (!t || t->dim() != 4) return false;
    n = t->size(0);
    h = t->size(1);
    page = t->size(2);
    d = t->size(3);
    if ((page > 1 && t->stride(2) != d) || (h > 1 && t->stride(1) != page * d) || (d > 1 && t->stride(3) != 1)) return false;
    stride = n > 1 ? t->stride(0) : h * page * d;
    const auto type = t->scalar_type();
    if (type == at::kByte) {
      fmt = MNW_KV_INT4;
      d *= 2;
      stride *= 2;
    } else if (type == at::kChar) {
      fmt = MNW_KV_INT8;
    } else if (type == at::kBFloat16) {
      fmt = MNW_KV_BF16;
    } else {
      return false;
    }
    return fits({n, h, page, d});
  }
  bool scale(PyObject* o, void** p) const {
    *p = nullptr;
    if (fmt == MNW_KV_BF16) return o == Py_None;
    return fmt == MNW_KV_INT8 ? whole(o, at::kFloat, {n, h, page}, p) : whole(o, at::kByte, {n, h, page, 8}, p);
  }
};
struct Cache : Pages {
  void *k = nullptr, *v = nullptr, *ks = nullptr, *vs = nullptr;
  bool read(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso) {
    const at::Tensor *kt = cuda(ko), *vt = cuda(vo);
    if (!kt || !vt || kt->scalar_type() != vt->scalar_type() || kt->sizes() != vt->sizes() || !Pages::read(kt) ||
        kt->strides() != vt->strides() || !scale(kso, &ks) || !scale(vso, &vs))
      return false;
    k = kt->data_ptr();
    v = vt->data_ptr();
    return true;
  }
};
// block table and lengths
struct Batch {
  int64_t B = 0, most = 0;
  void *table = nullptr, *lens = nullptr, *start = nullptr;
  bool read(PyObject* to, PyObject* lo, PyObject* so) {
    const at::Tensor* t = cuda(to);
    if (!t || t->scalar_type() != at::kInt || t->dim() != 2 || !t->is_contiguous()) return false;
    B = t->size(0);
    most = t->size(1);
    table = t->data_ptr();
    return fits({B, most}) && whole(lo, at::kInt, {B}, &lens) && whole(so, at::kInt, {B + 1}, &start, true);
  }
};

// The stream to launch on.
cudaStream_t current_stream() { return c10::cuda::getCurrentCUDAStream(device_now).stream(); }
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
template <class T>
const T* as(void* p) {
  return static_cast<const T*>(p);
}

PyObject* kv_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  device_now = -1;
  // q, k, v, k_cache, v_cache, block_table, cache_lens, inv_freq, layout, mscale, k_scale, v_scale, q_start, q_out, err
  if (n != 15) Py_RETURN_NOTIMPLEMENTED;
  const at::Tensor *kt = cuda(o[1]), *qt = o[0] == Py_None ? nullptr : cuda(o[0]);
  Cache c;
  Batch b;
  Tokens q, k, v;
  uint32_t* err;
  int layout;
  float mscale;
  void *freq = nullptr, *qo = nullptr;
  int64_t rot = 0;
  if (!kt || !c.read(o[3], o[4], o[10], o[11]) || !b.read(o[5], o[6], o[12]) || !k.read(kt, c.d) || !v.read(cuda(o[2]), c.d) ||
      k.h != c.h || v.h != c.h || v.T != k.T || !integer(o[8], &layout) || !real(o[9], &mscale) || !word(o[14], &err))
    Py_RETURN_NOTIMPLEMENTED;
  if (o[0] == Py_None ? o[13] != Py_None : (!q.read(qt, c.d) || q.T != k.T || !whole(o[13], at::kBFloat16, {q.T, q.h, q.d}, &qo, true)))
    Py_RETURN_NOTIMPLEMENTED;
  if (o[7] != Py_None) {
    const at::Tensor* f = cuda(o[7]);
    if (!f || f->numel() > INT_MAX / 2 || !whole(o[7], at::kFloat, {f->numel()}, &freq)) Py_RETURN_NOTIMPLEMENTED;
    rot = 2 * f->numel();
  }
  at::Tensor made;
  const cudaStream_t st = current_stream();
  int rc;
  {
    NoGil free;
    if (qt && !qo) {
      made = fresh({q.T, q.h, q.d}, at::kBFloat16, *qt);
      qo = made.data_ptr();
    }
    rc = lib.kv_append(q.p, q.stride, k.p, k.stride, v.p, v.stride, b.B, k.T, q.h, c.h, c.d, as<float>(freq), rot, layout, mscale, c.k, c.v,
                       static_cast<float*>(c.ks), static_cast<float*>(c.vs), c.fmt, c.n, c.page, c.stride, as<int32_t>(b.table), b.most,
                       as<int32_t>(b.lens), as<int32_t>(b.start), qo, err, st);
  }
  if (rc) return PyLong_FromLong(rc);
  return made.defined() ? THPVariable_Wrap(made) : same(o[13]);
  END_HANDLE_TH_ERRORS
}

PyObject* attn_paged(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  device_now = -1;
  // q, k_cache, v_cache, block_table, cache_lens, blk, scale, k_scale, v_scale, q_start, out, lse, want_lse, ws, err
  if (n != 15) Py_RETURN_NOTIMPLEMENTED;
  const at::Tensor* qt = cuda(o[0]);
  Cache c;
  Batch b;
  Tokens q;
  uint32_t* err;
  int blk;
  float scale;
  void *out, *lse, *ws;
  size_t bytes;
  if (!qt || !c.read(o[1], o[2], o[7], o[8]) || !b.read(o[3], o[4], o[9]) || !q.read(qt, c.d) || !integer(o[5], &blk) || !real(o[6], &scale) ||
      !whole(o[10], at::kBFloat16, {q.T, q.h, q.d}, &out, true) || !whole(o[11], at::kFloat, {q.T, q.h}, &lse, true) ||
      !workspace(o[13], &ws, &bytes) || !word(o[14], &err))
    Py_RETURN_NOTIMPLEMENTED;
  const cudaStream_t st = current_stream();
  const int want = o[11] != Py_None ? 0 : PyObject_IsTrue(o[12]);
  if (want < 0) return nullptr;
  at::Tensor made, made_lse;
  int rc;
  {
    NoGil free;
    if (!out) {
      made = fresh({q.T, q.h, q.d}, at::kBFloat16, *qt);
      out = made.data_ptr();
    }
    if (want) {
      made_lse = fresh({q.T, q.h}, at::kFloat, *qt);
      lse = made_lse.data_ptr();
    }
    const bool own = o[13] == Py_None;
    if (own) bytes = std::max<size_t>(256, lib.attn_paged_workspace_size(b.B, q.T, q.h, c.h, c.d));
    Scratch scratch(own ? bytes : 0, st);
    rc = lib.attn_paged(q.p, q.stride, b.B, q.T, q.h, c.h, c.d, c.k, c.v, as<float>(c.ks), as<float>(c.vs), c.fmt, c.n, c.page, c.stride,
                        as<int32_t>(b.table), b.most, as<int32_t>(b.lens), as<int32_t>(b.start), blk, scale, out, static_cast<float*>(lse),
                        own ? scratch.p : ws, bytes, err, st);
  }
  if (rc) return PyLong_FromLong(rc);
  PyObject* first = made.defined() ? THPVariable_Wrap(made) : same(o[10]);
  if (!first || (!want && o[11] == Py_None)) return first;
  PyObject* second = want ? THPVariable_Wrap(made_lse) : same(o[11]);
  PyObject* both = second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_DECREF(first);
  Py_XDECREF(second);
  return both;
  END_HANDLE_TH_ERRORS
}

PyObject* kv_values(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  device_now = -1;
  // cache, scale, out
  if (n != 3) Py_RETURN_NOTIMPLEMENTED;
  const at::Tensor* t = cuda(o[0]);
  Pages c;
  void *scale, *out;
  if (!c.read(t) || c.fmt == MNW_KV_BF16 || !c.scale(o[1], &scale) || !whole(o[2], at::kBFloat16, {c.n, c.h, c.page, c.d}, &out, true))
    Py_RETURN_NOTIMPLEMENTED;
  at::Tensor made;
  const cudaStream_t st = current_stream();
  int rc;
  {
    NoGil free;
    if (!out) {
      made = fresh({c.n, c.h, c.page, c.d}, at::kBFloat16, *t);
      out = made.data_ptr();
    }
    rc = lib.kv_values(t->data_ptr(), scale, c.fmt, c.n, c.page, c.h, c.d, c.stride, out, st);
  }
  if (rc) return PyLong_FromLong(rc);
  return made.defined() ? THPVariable_Wrap(made) : same(o[2]);
  END_HANDLE_TH_ERRORS
}

PyObject* lora_add(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  device_now = -1;
  // y, x, a, b, adapter, scale, ranks, out, ws, err
  if (n != 10) Py_RETURN_NOTIMPLEMENTED;
  const at::Tensor *yt = cuda(o[0]), *at_ = cuda(o[2]), *ot = o[7] == Py_None ? nullptr : cuda(o[7]);
  Rows y, x, out;
  uint32_t* err;
  void *a, *b, *ids, *scale, *ranks, *ws;
  size_t bytes;
  if (!y.read(yt) || !x.read(cuda(o[1])) || x.T != y.T || !at_ || at_->dim() != 3) Py_RETURN_NOTIMPLEMENTED;
  const int64_t many = at_->size(0), R = at_->size(1);
  if (!fits({many, R}) || !whole(o[2], at::kBFloat16, {many, R, x.n}, &a) || !whole(o[3], at::kBFloat16, {many, y.n, R}, &b) ||
      !whole(o[4], at::kInt, {y.T}, &ids) || !whole(o[5], at::kFloat, {many}, &scale, true) || !whole(o[6], at::kInt, {many}, &ranks, true) ||
      !workspace(o[8], &ws, &bytes) || !word(o[9], &err))
    Py_RETURN_NOTIMPLEMENTED;
  if (o[7] != Py_None && (!out.read(ot) || out.T != y.T || out.n != y.n)) Py_RETURN_NOTIMPLEMENTED;
  at::Tensor made;
  const cudaStream_t st = current_stream();
  int rc;
  {
    NoGil free;
    if (o[7] == Py_None) {
      made = fresh({y.T, y.n}, at::kBFloat16, *yt);
      out.p = made.data_ptr();
      out.stride = y.n;
    }
    const bool own = o[8] == Py_None;
    if (own) bytes = lib.lora_workspace_size(y.T, x.n, R, many);
    Scratch scratch(own ? bytes : 0, st);
    rc = lib.lora_add(x.p, x.stride, a, b, as<float>(scale), as<int32_t>(ranks), many, R, as<int32_t>(ids), y.T, x.n, y.n, y.p, y.stride,
                      out.p, out.stride, own ? scratch.p : ws, bytes, err, st);
  }
  if (rc) return PyLong_FromLong(rc);
  return made.defined() ? THPVariable_Wrap(made) : same(o[7]);
  END_HANDLE_TH_ERRORS
}

// Addresses of the library's functions, in the order of `Library`.
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
  void* at[6];
  if (n != 6) return PyErr_Format(PyExc_TypeError, "bind: expected 6 addresses");
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(o[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  lib.kv_append = reinterpret_cast<decltype(lib.kv_append)>(at[0]);
  lib.attn_paged = reinterpret_cast<decltype(lib.attn_paged)>(at[1]);
  lib.attn_paged_workspace_size = reinterpret_cast<decltype(lib.attn_paged_workspace_size)>(at[2]);
  lib.kv_values = reinterpret_cast<decltype(lib.kv_values)>(at[3]);
  lib.lora_add = reinterpret_cast<decltype(lib.lora_add)>(at[4]);
  lib.lora_workspace_size = reinterpret_cast<decltype(lib.lora_workspace_size)>(at[5]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F* f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"kv_append", fast(kv_append), METH_FASTCALL, nullptr},
                         {"attn_paged", fast(attn_paged), METH_FASTCALL, nullptr},
                         {"kv_values", fast(kv_values), METH_FASTCALL, nullptr},
                         {"lora_add", fast(lora_add), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mnw_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mnw_calls() { return PyModule_Create(&module); }

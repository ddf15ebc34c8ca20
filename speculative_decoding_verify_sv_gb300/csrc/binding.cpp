// The Python calls of the operators around the KV cache, compiled: check the tensors against the
// ABI's layouts, take pointers and the current stream, make the outputs and call libsv.so.
//
// These operators run once per layer, or for a single token, where the host side of a call is
// what counts: the same checks written in Python cost 7 to 16 us a call on the Grace cores of a
// GB300, more than the kernels of the small calls run.  Everything is computed in libsv.so; a
// status other than SV_OK becomes the package's SVError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <optional>

#include "sv.h"

namespace {

PyObject *g_error = nullptr;  // SVError(code, message)

struct Refused {};  // the Python error is set

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Refused();
}

// Runs a call of libsv.so and turns its status into an error.  The interpreter's lock is given up
// meanwhile: a launch waits while the device's queue of launches is full, and what would empty it may
// need another thread of this process (a host function of a stream, the feeder of a copy).
// (The call touches no Python object.)
template <typename Call>
void check(Call &&call) {
  struct Unlocked {
    PyThreadState *const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  };
  const sv_status st = [&] {
    const Unlocked unlocked;
    return call();
  }();
  if (st == SV_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, sv_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

bool given(PyObject *o) { return o != nullptr && o != Py_None; }

const at::Tensor &cuda_tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return t;
}

PyObject *shape_text(at::IntArrayRef s) {
  PyObject *l = PyTuple_New((Py_ssize_t)s.size());
  for (size_t i = 0; l && i < s.size(); ++i) PyTuple_SET_ITEM(l, (Py_ssize_t)i, PyLong_FromLongLong(s[i]));
  return l;
}

// A contiguous CUDA tensor of this type and shape on device `dev`.
const at::Tensor &tensor(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor &t = cuda_tensor(o, name);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()), c10::toString(type));
  if (t.sizes() != shape) {
    PyObject *a = shape_text(t.sizes()), *b = shape_text(shape);
    PyErr_Format(PyExc_ValueError, "%s has shape %R, expected %R", name, a, b);
    Py_XDECREF(a);
    Py_XDECREF(b);
    throw Refused();
  }
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, "%s is on cuda:%d, the other tensors on cuda:%d: one call works on one device", name,
           (int)t.get_device(), dev);
  return t;
}
const at::Tensor &tensor(PyObject *o, const char *name, at::ScalarType type, int dev) {
  return tensor(o, name, type, cuda_tensor(o, name).sizes(), dev);
}

int number(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s = %lld is not a 32-bit number", name, v);
  return (int)v;
}
float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

sv_dtype dtype_of(const at::Tensor &t) {
  if (t.scalar_type() == at::kBFloat16) return SV_BF16;
  if (t.scalar_type() == at::kFloat) return SV_F32;
  refuse(PyExc_TypeError, "unsupported dtype %s (bfloat16 or float32)", c10::toString(t.scalar_type()));
}

at::Tensor make(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// A part of a new buffer, from element `offset` on, as a tensor of its own (one allocation for a
// call's outputs).
at::Tensor part(const at::Tensor &buffer, int64_t offset, at::IntArrayRef shape) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(buffer.storage()),
                                                          buffer.key_set(), buffer.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(buffer.storage_offset() + offset);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// The stream of a call on device `dev`: the one given (a torch stream or a handle), else the
// device's current one.  While it stands it is the current one, so that what the call makes
// (outputs, a zero-filled workspace) belongs to it and is not in use on another stream.
class Stream {
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> given_;
  c10::cuda::CUDAStream stream_;

  static c10::cuda::CUDAStream of(PyObject *o, int dev) {
    if (!given(o)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
    PyObject *h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (!h) throw Refused();
    void *s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!s && PyErr_Occurred()) throw Refused();
    return s ? c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), (c10::DeviceIndex)dev)
             : c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev);
  }

 public:
  Stream(PyObject *o, int dev) : stream_(of(o, dev)) {
    if (given(o)) given_.emplace(stream_);
    else device_.emplace((c10::DeviceIndex)dev);
  }
  operator void *() const { return stream_.stream(); }
};

// A tree argument: a host sequence [N] shared by the batch (stride 0), or a CUDA int32 tensor
// [B, >= N] with one tree per sequence.
struct Tree {
  int32_t rows[SV_MAX_TREE_NODES];
  const int32_t *ptr;
  int stride;
  Tree(PyObject *o, int64_t B, int64_t N, int dev) {
    PyObject *list = nullptr;
    if (THPVariable_Check(o)) {
      const at::Tensor &t = THPVariable_Unpack(o);
      if (t.is_cuda()) {
        if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B)
          refuse(PyExc_ValueError, "per-sequence parents must be a CUDA int32 tensor [B=%lld, >= N]", (long long)B);
        if (t.size(1) < N || t.stride(1) != 1 || t.stride(0) < N || t.stride(0) > INT32_MAX)
          refuse(PyExc_ValueError, "per-sequence parents need contiguous rows of at least N=%lld", (long long)N);
        if (t.get_device() != dev)
          refuse(PyExc_ValueError, "parent is on cuda:%d, the other tensors on cuda:%d", (int)t.get_device(), dev);
        ptr = t.const_data_ptr<int32_t>();
        stride = (int)t.stride(0);
        return;
      }
      list = PyObject_CallMethod(o, "tolist", nullptr);
    } else {
      list = PySequence_Fast(o, "parent must be a sequence or a CUDA int32 tensor");
    }
    if (!list) throw Refused();
    PyObject *fast = PySequence_Fast(list, "parent must be a sequence");
    Py_DECREF(list);
    if (!fast) throw Refused();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    bool ok = n == N;
    if (!ok) PyErr_Format(PyExc_ValueError, "parent has %zd entries, the tree has %lld rows", n, (long long)N);
    for (Py_ssize_t i = 0; ok && i < n && i < SV_MAX_TREE_NODES; ++i) {
      const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(fast, i));
      ok = !(v == -1 && PyErr_Occurred());
      rows[i] = v < INT32_MIN || v > INT32_MAX ? INT32_MIN : (int32_t)v;  // (no node either way)
    }
    Py_DECREF(fast);
    if (!ok) throw Refused();
    ptr = rows;
    stride = 0;
  }
};

template <typename F>
PyObject *guarded(F &&body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
}

// A cache (k, v, prefix_len, block_table, block_size) of B sequences with Hkv heads of D.
struct Cache {
  sv_kv_cache c{};
  Cache(PyObject *const *a, at::ScalarType type, int64_t B, int64_t Hkv, int64_t D, int dev) {
    const at::Tensor &k0 = cuda_tensor(a[0], "cache.k");
    const bool paged = given(a[3]);
    if (k0.scalar_type() != type) refuse(PyExc_TypeError, "cache dtype differs from q");
    if (k0.dim() != 4 || k0.size(2) != Hkv || k0.size(3) != D || (!paged && k0.size(0) != B))
      refuse(PyExc_ValueError, "cache.k does not hold %lld heads of %lld%s", (long long)Hkv, (long long)D,
             paged ? " in pages" : " of q's sequences");
    const at::Tensor &k = tensor(a[0], "cache.k", type, k0.sizes(), dev);
    const at::Tensor &v = tensor(a[1], "cache.v", type, k0.sizes(), dev);
    const at::Tensor &len = tensor(a[2], "cache.prefix_len", at::kInt, {B}, dev);
    if (B > INT32_MAX || Hkv > INT32_MAX || k.size(0) > INT32_MAX || k.size(1) > INT32_MAX)
      refuse(PyExc_ValueError, "a size is not a 32-bit number");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.prefix_len = len.data_ptr<int32_t>();
    if (paged) {
      const int block_size = number(a[4], "block_size");
      const at::Tensor &bt = cuda_tensor(a[3], "cache.block_table");
      if (bt.dim() != 2 || k.size(1) != block_size || bt.size(1) > INT32_MAX)
        refuse(PyExc_ValueError, "blocks of %lld rows need block_size %lld and a block_table [B, max_blocks]",
               (long long)k.size(1), (long long)k.size(1));
      c.block_table = tensor(a[3], "cache.block_table", at::kInt, {B, bt.size(1)}, dev).const_data_ptr<int32_t>();
      c.block_size = block_size;
      c.max_blocks = (int)bt.size(1);
      c.num_blocks = (int)k.size(0);
    } else {
      c.Lmax = (int)k.size(1);
    }
  }
  int max_prefix() const {
    const long long cap = c.block_table ? (long long)c.max_blocks * c.block_size : c.Lmax;
    return (int)std::min<long long>(cap, INT32_MAX);
  }
};

// The arguments that the attentions have in common: (q, k_tree, v_tree, cache k, v, prefix_len,
// block_table, block_size, parent, scale, ...).
struct Attention {
  const at::Tensor &q0;
  const int dev;
  const sv_dtype dt;
  const at::ScalarType type;
  int64_t B, N, Hq, Hkv, D;
  const at::Tensor *q, *kt, *vt;
  std::optional<Cache> cache;
  float scale;
  std::optional<Tree> tree;
  explicit Attention(PyObject *const *a)
      : q0(cuda_tensor(a[0], "q")), dev(q0.get_device()), dt(dtype_of(q0)), type(q0.scalar_type()) {
    if (q0.dim() != 4) refuse(PyExc_ValueError, "q must be [B, N, Hq, D]");
    q = &tensor(a[0], "q", type, q0.sizes(), dev);
    B = q->size(0), N = q->size(1), Hq = q->size(2), D = q->size(3);
    const at::Tensor &kt0 = cuda_tensor(a[1], "k_tree");
    if (kt0.dim() != 4) refuse(PyExc_ValueError, "k_tree must be [B, N, Hkv, D]");
    Hkv = kt0.size(2);
    kt = &tensor(a[1], "k_tree", type, {B, N, Hkv, D}, dev);
    vt = &tensor(a[2], "v_tree", type, {B, N, Hkv, D}, dev);
    cache.emplace(a + 3, type, B, Hkv, D, dev);
    if (N > INT32_MAX || Hq > INT32_MAX) refuse(PyExc_ValueError, "a size is not a 32-bit number");
    scale = real(a[9]);
    tree.emplace(a[8], B, N, dev);
  }
  at::Tensor output(PyObject *o) const { return given(o) ? tensor(o, "out", type, q->sizes(), dev) : make(q->sizes(), *q, type); }
};

// (q, k_tree, v_tree, cache k, v, prefix_len, block_table, block_size, parent, scale, window, sinks,
//  out, workspace, stream) -> out
PyObject *window_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 15);
    const Attention t(a);
    const int window = number(a[10], "window"), sinks = number(a[11], "sinks");
    const Stream stream(a[14], t.dev);
    at::Tensor out = t.output(a[12]);
    // (a workspace passed in must have been zero-filled before its first use; the library checks
    // its size)
    at::Tensor ws;
    if (given(a[13])) {
      ws = tensor(a[13], "workspace", cuda_tensor(a[13], "workspace").scalar_type(), t.dev);
    } else {
      const size_t need = sv_window_attention_workspace_size(t.dt, (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D,
                                                             t.cache->max_prefix(), window);
      if (need) ws = at::zeros({(int64_t)need}, t.q->options().dtype(at::kByte));
    }
    check([&] {
      return sv_window_attention(t.dt, (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D, t.q->data_ptr(), t.kt->data_ptr(),
                                 t.vt->data_ptr(), t.cache->c, t.tree->ptr, t.tree->stride, t.scale, window, sinks,
                                 out.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, stream);
    });
    return THPVariable_Wrap(std::move(out));
  });
}

// The workspace given, or a new one of the size that need() says.
template <typename Need>
at::Tensor workspace_of(PyObject *o, const at::Tensor &like, int dev, Need &&need) {
  if (given(o)) return tensor(o, "workspace", cuda_tensor(o, "workspace").scalar_type(), dev);
  const size_t bytes = need();
  return bytes ? make({(int64_t)bytes}, like, at::kByte) : at::Tensor();
}

// (q, k_tree, v_tree, cache k, v, prefix_len, block_table, block_size, parent, scale, group_start, shared_len,
//  out, workspace, stream) -> out
PyObject *shared_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 15);
    const Attention t(a);
    const at::Tensor &len = cuda_tensor(a[11], "shared_len");
    if (len.dim() != 1 || len.size(0) < 1 || len.size(0) > SV_MAX_SHARED_GROUPS)
      refuse(PyExc_ValueError, "shared_len must be [groups], 1 to %d of them", SV_MAX_SHARED_GROUPS);
    const int groups = (int)len.size(0);
    const int32_t *lens = tensor(a[11], "shared_len", at::kInt, {groups}, t.dev).const_data_ptr<int32_t>();
    const int32_t *starts = tensor(a[10], "group_start", at::kInt, {groups + 1}, t.dev).const_data_ptr<int32_t>();
    const Stream stream(a[14], t.dev);
    at::Tensor out = t.output(a[12]);
    const at::Tensor ws = workspace_of(a[13], *t.q, t.dev, [&] {
      return sv_shared_attention_workspace_size(t.dt, (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D, t.cache->max_prefix(), groups);
    });
    check([&] {
      return sv_shared_attention(t.dt, (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D, t.q->data_ptr(), t.kt->data_ptr(),
                                 t.vt->data_ptr(), t.cache->c, t.tree->ptr, t.tree->stride, t.scale, starts, lens, groups,
                                 out.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, stream);
    });
    return THPVariable_Wrap(std::move(out));
  });
}

// (q, k_tree, v_tree, cache k, v, prefix_len, block_table, block_size, parent, scale, pages, out, workspace,
//  stream) -> out
PyObject *sparse_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 14);
    const Attention t(a);
    const at::Tensor &p0 = cuda_tensor(a[10], "pages");
    if (p0.dim() != 4 || p0.size(3) > INT32_MAX || (p0.size(1) != 1 && p0.size(1) != t.N))
      refuse(PyExc_ValueError, "pages must be [B, 1 or N, Hkv, K]");
    const int64_t sets = p0.size(1), K = p0.size(3);
    const at::Tensor &pages = tensor(a[10], "pages", at::kInt, {t.B, sets, t.Hkv, K}, t.dev);
    const int page_size = number(a[7], "block_size");
    const Stream stream(a[13], t.dev);
    at::Tensor out = t.output(a[11]);
    const at::Tensor ws = workspace_of(a[12], *t.q, t.dev, [&] {
      return sv_sparse_attention_workspace_size(t.dt, (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D, page_size, (int)K, (int)sets);
    });
    check([&] {
      return sv_sparse_attention(t.dt, (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D, t.q->data_ptr(), t.kt->data_ptr(),
                                 t.vt->data_ptr(), t.cache->c, t.tree->ptr, t.tree->stride, t.scale,
                                 pages.const_data_ptr<int32_t>(), (int)sets, (int)K, page_size, out.data_ptr(),
                                 ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, stream);
    });
    return THPVariable_Wrap(std::move(out));
  });
}

// (cache k, v, prefix_len, block_table, block_size, bounds, start, stream) -> bounds
PyObject *page_bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 8);
    const at::Tensor &k = cuda_tensor(a[0], "cache.k"), &len = cuda_tensor(a[2], "cache.prefix_len");
    const int dev = k.get_device();
    const sv_dtype dt = dtype_of(k);
    if (k.dim() != 4 || len.dim() != 1) refuse(PyExc_ValueError, "cache.k must be [.., .., Hkv, D] and cache.prefix_len [B]");
    const int64_t B = len.size(0), Hkv = k.size(2), D = k.size(3);
    const Cache cache(a, k.scalar_type(), B, Hkv, D, dev);
    const int page_size = number(a[4], "block_size");
    if (page_size < 1) refuse(PyExc_ValueError, "block_size = %d", page_size);
    const int64_t seq_pages = (cache.c.Lmax + (int64_t)page_size - 1) / page_size;
    const int32_t *start = given(a[6]) ? tensor(a[6], "start", at::kInt, {B}, dev).const_data_ptr<int32_t>() : nullptr;
    const Stream stream(a[7], dev);
    const bool paged = cache.c.block_table != nullptr;
    at::Tensor bounds;
    if (given(a[5])) {
      bounds = paged ? tensor(a[5], "bounds", k.scalar_type(), {k.size(0), Hkv, 2, D}, dev)
                     : tensor(a[5], "bounds", k.scalar_type(), {B, seq_pages, Hkv, 2, D}, dev);
    } else {  // (rows of pages that hold nothing yet are not written)
      bounds = paged ? make({k.size(0), Hkv, 2, D}, k, k.scalar_type()) : make({B, seq_pages, Hkv, 2, D}, k, k.scalar_type());
    }
    check([&] { return sv_page_bounds(dt, (int)B, (int)Hkv, (int)D, page_size, cache.c, start, bounds.data_ptr(), stream); });
    return THPVariable_Wrap(std::move(bounds));
  });
}

// (q, bounds, prefix_len, page_size, block_table, per_node, out, stream) -> out
PyObject *page_scores(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 8);
    const at::Tensor &q0 = cuda_tensor(a[0], "q"), &b0 = cuda_tensor(a[1], "bounds");
    const int dev = q0.get_device();
    const sv_dtype dt = dtype_of(q0);
    if (q0.dim() != 4) refuse(PyExc_ValueError, "q must be [B, N, Hq, D]");
    const at::Tensor &q = tensor(a[0], "q", q0.scalar_type(), q0.sizes(), dev);
    const int64_t B = q.size(0), N = q.size(1), Hq = q.size(2), D = q.size(3);
    const bool paged = given(a[4]);
    if (b0.dim() != (paged ? 4 : 5)) refuse(PyExc_ValueError, "bounds must be %s", paged ? "[num_blocks, Hkv, 2, D]" : "[B, P, Hkv, 2, D]");
    const int64_t Hkv = b0.size(-3);
    int64_t P, blocks = 0;
    const int32_t *table = nullptr;
    const at::Tensor *bounds;
    if (paged) {
      const at::Tensor &bt = cuda_tensor(a[4], "block_table");
      if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table must be [B, max_blocks]");
      P = bt.size(1), blocks = b0.size(0);
      table = tensor(a[4], "block_table", at::kInt, {B, P}, dev).const_data_ptr<int32_t>();
      bounds = &tensor(a[1], "bounds", q.scalar_type(), {blocks, Hkv, 2, D}, dev);
    } else {
      P = b0.size(1);
      bounds = &tensor(a[1], "bounds", q.scalar_type(), {B, P, Hkv, 2, D}, dev);
    }
    const int32_t *len = tensor(a[2], "prefix_len", at::kInt, {B}, dev).const_data_ptr<int32_t>();
    if (B > INT32_MAX || N > INT32_MAX || Hq > INT32_MAX || Hkv > INT32_MAX || P > INT32_MAX || blocks > INT32_MAX)
      refuse(PyExc_ValueError, "a size is not a 32-bit number");
    const int page_size = number(a[3], "page_size"), per_node = PyObject_IsTrue(a[5]);
    if (per_node < 0) throw Refused();
    const int64_t sets = per_node ? N : 1;
    const Stream stream(a[7], dev);
    at::Tensor out = given(a[6]) ? tensor(a[6], "out", at::kFloat, {B, sets, Hkv, P}, dev) : make({B, sets, Hkv, P}, q, at::kFloat);
    check([&] {
      return sv_page_scores(dt, (int)B, (int)N, (int)Hq, (int)Hkv, (int)D, q.data_ptr(), bounds->data_ptr(), len, page_size, (int)P,
                            table, (int)blocks, (int)sets, out.data_ptr<float>(), stream);
    });
    return THPVariable_Wrap(std::move(out));
  });
}

// (scores, prefix_len, page_size, count, first, last, out, stream) -> out
PyObject *select_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 8);
    const at::Tensor &s0 = cuda_tensor(a[0], "scores");
    const int dev = s0.get_device();
    if (s0.dim() != 4) refuse(PyExc_ValueError, "scores must be [B, sets, Hkv, P]");
    const at::Tensor &scores = tensor(a[0], "scores", at::kFloat, s0.sizes(), dev);
    const int64_t B = scores.size(0), sets = scores.size(1), Hkv = scores.size(2), P = scores.size(3);
    if (B > INT32_MAX || sets > INT32_MAX || Hkv > INT32_MAX || sets * Hkv > INT32_MAX || P > INT32_MAX)
      refuse(PyExc_ValueError, "a size is not a 32-bit number");
    const int32_t *len = tensor(a[1], "prefix_len", at::kInt, {B}, dev).const_data_ptr<int32_t>();
    const int page_size = number(a[2], "page_size"), K = number(a[3], "count"), first = number(a[4], "first"), last = number(a[5], "last");
    if (K < 0) refuse(PyExc_ValueError, "count = %d", K);
    const Stream stream(a[7], dev);
    at::Tensor out = given(a[6]) ? tensor(a[6], "out", at::kInt, {B, sets, Hkv, K}, dev) : make({B, sets, Hkv, K}, scores, at::kInt);
    check([&] {
      return sv_select_pages((int)B, (int)(sets * Hkv), (int)P, scores.const_data_ptr<float>(), len, page_size, K, first, last,
                             out.data_ptr<int32_t>(), stream);
    });
    return THPVariable_Wrap(std::move(out));
  });
}

// The outputs of a batch without requests (no kernel runs for it): no tokens, the head as it was.
void empty_tables(PyObject *outs, const char *const *names, PyObject *head) {
  at::Tensor t[4];
  for (int i = 0; i < 4; ++i) t[i] = THPVariable_Unpack(PyDict_GetItemString(outs, names[i]));
  t[0].zero_();
  t[1].fill_(-1);
  t[2].fill_(-1);
  if (given(head)) t[3].copy_(THPVariable_Unpack(head));
  else t[3].zero_();
}

// (length, new_tokens, block_table, free_blocks, block_size, num_blocks, num_slots, free_head, outs,
//  stream, held) -> outs, a dict, filled up with the outputs it lacks
PyObject *block_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 11);
    const at::Tensor &len0 = cuda_tensor(a[0], "length");
    const int dev = len0.get_device();
    if (len0.dim() != 1) refuse(PyExc_ValueError, "length must be [B]");
    const int64_t B = len0.size(0), T = number(a[6], "num_slots");
    if (T < 0) refuse(PyExc_ValueError, "num_slots = %lld", (long long)T);
    const at::Tensor &len = tensor(a[0], "length", at::kInt, {B}, dev);
    const at::Tensor &add = tensor(a[1], "new_tokens", at::kInt, {B}, dev);
    const at::Tensor &bt0 = cuda_tensor(a[2], "block_table");
    if (bt0.dim() != 2) refuse(PyExc_ValueError, "block_table must be [B, max_blocks]");
    const at::Tensor &bt = tensor(a[2], "block_table", at::kInt, {B, bt0.size(1)}, dev);
    const at::Tensor &free = tensor(a[3], "free_blocks", at::kInt, dev);
    if (B > INT32_MAX || bt.size(1) > INT32_MAX || free.numel() > INT32_MAX)
      refuse(PyExc_ValueError, "a size is not a 32-bit number");
    const int block_size = number(a[4], "block_size"), num_blocks = number(a[5], "num_blocks");
    const int32_t *head = given(a[7]) ? tensor(a[7], "free_head", at::kInt, {1}, dev).const_data_ptr<int32_t>() : nullptr;
    const int32_t *held = given(a[10]) ? tensor(a[10], "held", at::kInt, {B}, dev).const_data_ptr<int32_t>() : nullptr;
    const Stream stream(a[9], dev);
    static const char *const names[5] = {"token_start", "slots", "positions", "free_head", "held"};
    static PyObject *const keys[5] = {PyUnicode_InternFromString(names[0]), PyUnicode_InternFromString(names[1]),
                                      PyUnicode_InternFromString(names[2]), PyUnicode_InternFromString(names[3]),
                                      PyUnicode_InternFromString(names[4])};
    const int64_t sizes[5] = {B + 1, T, T, 1, B};
    const int made = given(a[10]) ? 5 : 4;  // outputs
    PyObject *outs = given(a[8]) ? a[8] : PyDict_New();
    if (!outs) throw Refused();
    if (given(a[8])) {
      if (!PyDict_Check(outs)) refuse(PyExc_TypeError, "outs must be a dict");
      Py_INCREF(outs);
    }
    try {
      // new outputs are parts of one buffer, the slots and positions on 16-byte boundaries
      const int64_t padded = (T + 3) / 4 * 4, offsets[5] = {2 * padded, 0, padded, 2 * padded + B + 1, 2 * padded + B + 2};
      at::Tensor buffer, kept[5];  // (another thread may change the dict while the call is under way)
      int32_t *ptr[5];
      for (int i = 0; i < made; ++i) {
        PyObject *o = given(a[8]) ? PyDict_GetItemWithError(outs, keys[i]) : nullptr;
        if (!o && PyErr_Occurred()) throw Refused();
        if (o) {
          kept[i] = tensor(o, names[i], at::kInt, {sizes[i]}, dev);
          ptr[i] = kept[i].data_ptr<int32_t>();
        } else {
          if (!buffer.defined()) buffer = make({2 * padded + B + 2 + (made == 5 ? B : 0)}, len, at::kInt);
          ptr[i] = buffer.data_ptr<int32_t>() + offsets[i];
          PyObject *w = THPVariable_Wrap(part(buffer, offsets[i], {sizes[i]}));
          if (!w || PyDict_SetItem(outs, keys[i], w) != 0) {
            Py_XDECREF(w);
            throw Refused();
          }
          Py_DECREF(w);
        }
      }
      const int32_t *lengths = len.const_data_ptr<int32_t>(), *added = add.const_data_ptr<int32_t>(), *ids = free.const_data_ptr<int32_t>();
      const int columns = (int)bt.size(1), num_free = (int)free.numel();
      if (made == 5)
        check([&] {
          return sv_block_tables_held((int)B, lengths, added, block_size, columns, num_blocks, ids, num_free, head, held,
                                      bt.data_ptr<int32_t>(), (int)T, ptr[0], ptr[1], ptr[2], ptr[3], ptr[4], stream);
        });
      else
        check([&] {
          return sv_block_tables((int)B, lengths, added, block_size, columns, num_blocks, ids, num_free, head,
                                 bt.data_ptr<int32_t>(), (int)T, ptr[0], ptr[1], ptr[2], ptr[3], stream);
        });
      if (B == 0) empty_tables(outs, names, a[7]);  // (the arguments are checked)
    } catch (...) {
      Py_DECREF(outs);
      throw;
    }
    return outs;
  });
}

// A projection qkv [*, (Hq + 2 Hkv) * D] of `lead` leading dimensions with evenly spaced rows, its
// weights and frequencies.
struct Projection {
  const at::Tensor &qkv, &qw, &kw, &freq;
  int dev;
  sv_dtype dt;
  int64_t Hq, Hkv, D, rows, ld;
  Projection(PyObject *const *a, int lead)
      : qkv(cuda_tensor(a[0], "qkv")), qw(cuda_tensor(a[3], "q_weight")), kw(cuda_tensor(a[4], "k_weight")),
        freq(cuda_tensor(a[5], "inv_freq")), dev(qkv.get_device()), dt(dtype_of(qkv)), Hq(number(a[1], "Hq")),
        Hkv(number(a[2], "Hkv")), D(qw.numel()) {
    tensor(a[3], "q_weight", at::kFloat, {D}, dev);
    tensor(a[4], "k_weight", at::kFloat, {D}, dev);
    tensor(a[5], "inv_freq", at::kDouble, {freq.numel()}, dev);
    if (Hq < 1 || Hkv < 1 || D < 1 || D > 4096 || freq.numel() > 4096)
      refuse(PyExc_ValueError, "Hq = %lld, Hkv = %lld, head dim %lld, %lld frequencies", (long long)Hq, (long long)Hkv,
             (long long)D, (long long)freq.numel());
    const int64_t width = (Hq + 2 * Hkv) * D;
    if (qkv.dim() != lead + 1 || qkv.size(lead) != width) {
      PyObject *s = shape_text(qkv.sizes());
      PyErr_Format(PyExc_ValueError, "qkv has shape %R, expected %d leading dimensions and rows of %lld", s, lead,
                   (long long)width);
      Py_XDECREF(s);
      throw Refused();
    }
    rows = qkv.size(0) * (lead == 2 ? qkv.size(1) : 1);
    ld = width;
    if (rows > 1) {
      ld = lead == 1 ? qkv.stride(0) : (qkv.size(1) != 1 ? qkv.stride(1) : qkv.stride(0));
      if (lead == 2 && qkv.size(0) != 1 && qkv.stride(0) != qkv.size(1) * ld)
        refuse(PyExc_ValueError, "the rows of qkv must be evenly spaced");
    }
    if (rows > 0 && (qkv.stride(lead) != 1 || ld < width))
      refuse(PyExc_ValueError, "the rows of qkv must be contiguous and apart");
    if (rows > INT32_MAX) refuse(PyExc_ValueError, "%lld tokens", (long long)rows);
  }
};

// (qkv, Hq, Hkv, q_weight, k_weight, inv_freq, positions, eps, interleaved, slots, q_out, k_out, v_out,
//  stream) -> (q, k, v)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 14);
    const Projection p(a, 1);
    const int64_t T = p.rows;
    const at::ScalarType type = p.qkv.scalar_type();
    const at::Tensor &at_pos = tensor(a[6], "positions", at::kInt, {T}, p.dev);
    const int32_t *slots = nullptr;
    if (given(a[9])) {
      if (!given(a[11]) || !given(a[12])) refuse(PyExc_ValueError, "slots need k_out and v_out");
      slots = tensor(a[9], "slots", at::kInt, {T}, p.dev).const_data_ptr<int32_t>();
    }
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0) throw Refused();
    const float eps = real(a[7]);
    const Stream stream(a[13], p.dev);
    at::Tensor q = given(a[10]) ? tensor(a[10], "q_out", type, {T, p.Hq, p.D}, p.dev) : make({T, p.Hq, p.D}, p.qkv, type);
    at::Tensor k = given(a[11]) ? tensor(a[11], "k_out", type, p.dev) : make({T, p.Hkv, p.D}, p.qkv, type);
    if (k.dim() < 3 || k.size(-2) != p.Hkv || k.size(-1) != p.D) {
      PyObject *s = shape_text(k.sizes());
      PyErr_Format(PyExc_ValueError, "k_out has shape %R, expected [..., %lld, %lld]", s, (long long)p.Hkv, (long long)p.D);
      Py_XDECREF(s);
      throw Refused();
    }
    at::Tensor v = given(a[12]) ? tensor(a[12], "v_out", type, k.sizes(), p.dev) : make(k.sizes(), p.qkv, type);
    check([&] {
      return sv_qk_norm_rope(p.dt, (int)T, (int)p.Hq, (int)p.Hkv, (int)p.D, 2 * (int)p.freq.numel(), interleaved,
                             p.qkv.data_ptr(), p.ld, p.qw.const_data_ptr<float>(), p.kw.const_data_ptr<float>(), eps,
                             p.freq.const_data_ptr<double>(), at_pos.const_data_ptr<int32_t>(), slots,
                             k.numel() / (p.Hkv * p.D), q.data_ptr(), k.data_ptr(), v.data_ptr(), stream);
    });
    return Py_BuildValue("NNN", THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(k)),
                         THPVariable_Wrap(std::move(v)));
  });
}

// (qkv, Hq, Hkv, q_weight, k_weight, inv_freq, prefix_len, parent, eps, interleaved, outs, stream)
//  -> (q, k_tree, v_tree)
PyObject *tree_qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    expect(n, 12);
    const Projection p(a, 2);
    const int64_t B = p.qkv.size(0), N = p.qkv.size(1);
    const at::ScalarType type = p.qkv.scalar_type();
    const at::Tensor &len = tensor(a[6], "prefix_len", at::kInt, {B}, p.dev);
    const Tree tree(a[7], B, N, p.dev);
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0) throw Refused();
    const float eps = real(a[8]);
    const Stream stream(a[11], p.dev);
    at::Tensor q, k, v;
    if (given(a[10])) {
      PyObject *f = PySequence_Fast(a[10], "outs must be (q, k_tree, v_tree)");
      if (!f) throw Refused();
      const bool three = PySequence_Fast_GET_SIZE(f) == 3;
      PyObject *o[3] = {nullptr, nullptr, nullptr};
      for (int i = 0; three && i < 3; ++i) o[i] = PySequence_Fast_GET_ITEM(f, i);
      Py_DECREF(f);  // (the caller's sequence keeps its items)
      if (!three) refuse(PyExc_ValueError, "outs must be (q, k_tree, v_tree)");
      q = tensor(o[0], "q", type, {B, N, p.Hq, p.D}, p.dev);
      k = tensor(o[1], "k_tree", type, {B, N, p.Hkv, p.D}, p.dev);
      v = tensor(o[2], "v_tree", type, {B, N, p.Hkv, p.D}, p.dev);
    } else {
      const int64_t head = B * N * p.D;
      const at::Tensor buffer = make({head * (p.Hq + 2 * p.Hkv)}, p.qkv, type);
      q = part(buffer, 0, {B, N, p.Hq, p.D});
      k = part(buffer, head * p.Hq, {B, N, p.Hkv, p.D});
      v = part(buffer, head * (p.Hq + p.Hkv), {B, N, p.Hkv, p.D});
    }
    check([&] {
      return sv_tree_qk_norm_rope(p.dt, (int)B, (int)N, (int)p.Hq, (int)p.Hkv, (int)p.D, 2 * (int)p.freq.numel(), interleaved,
                                  p.qkv.data_ptr(), p.ld, p.qw.const_data_ptr<float>(), p.kw.const_data_ptr<float>(), eps,
                                  p.freq.const_data_ptr<double>(), len.const_data_ptr<int32_t>(), tree.ptr, tree.stride,
                                  q.data_ptr(), k.data_ptr(), v.data_ptr(), stream);
    });
    return Py_BuildValue("NNN", THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(k)),
                         THPVariable_Wrap(std::move(v)));
  });
}

PyObject *set_error(PyObject *, PyObject *type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"window_attention", FAST(window_attention), METH_FASTCALL, nullptr},
                         {"shared_attention", FAST(shared_attention), METH_FASTCALL, nullptr},
                         {"sparse_attention", FAST(sparse_attention), METH_FASTCALL, nullptr},
                         {"page_bounds", FAST(page_bounds), METH_FASTCALL, nullptr},
                         {"page_scores", FAST(page_scores), METH_FASTCALL, nullptr},
                         {"select_pages", FAST(select_pages), METH_FASTCALL, nullptr},
                         {"block_tables", FAST(block_tables), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", FAST(qk_norm_rope), METH_FASTCALL, nullptr},
                         {"tree_qk_norm_rope", FAST(tree_qk_norm_rope), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "sv_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_sv_binding(void) { return PyModule_Create(&module); }

// Python calls of the norm, rotation and paged-cache entry points: checks of tensors, outputs, and the C call, compiled.
//
// These kernels take 2 to 10 us at decode sizes. Marshalled in Python through ctypes their calls took 10 to 36 us of
// the host (tens of attribute reads and a conversion for each of up to 37 arguments). Everything here is that
// marshalling (3 to 11 us now, 2.2 us of them each launch); all compute runs in libattn_gb300.so, which this module
// links to. Functions take their arguments by position, None for one that is not given, and launch on the current
// stream of the current device. binding.py holds the signatures, defaults and documentation.
#include <Python.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn.h"

namespace {

PyObject *g_attn_error = nullptr, *g_out_of_memory = nullptr;   // binding.AttnError, torch.OutOfMemoryError

struct Refused : std::runtime_error {   // ValueError
  using std::runtime_error::runtime_error;
};
struct WrongType : std::runtime_error {   // TypeError
  using std::runtime_error::runtime_error;
};
struct Raised {};   // a Python error is set already

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

// A tensor argument; null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a torch tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) throw WrongType(std::string(name) + " must be a torch tensor");
  return *t;
}

[[noreturn]] void refuse_device(const std::string& device) {
  refuse("every tensor of a call must be a CUDA tensor on the current device, got one on " + device);
}

// The current stream of the current device. Kernels launch there: all of the call's tensors have to be on it (null: one
// not given).
cudaStream_t launch_stream(std::initializer_list<const at::Tensor*> tensors) {
  int dev = -1;
  for (const at::Tensor* t : tensors) {
    if (!t) continue;
    if (!t->is_cuda()) refuse_device(t->device().str());   // before the first CUDA call: there may be no GPU
    if (dev < 0) dev = c10::cuda::current_device();
    if (t->get_device() != dev) refuse_device(t->device().str());
  }
  return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
}

void* pointer(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

struct Rows {   // bf16 rows [T, heads, d] or [B, N, heads, d]: tokens, heads, values, tokens of a sequence, strides
  long long T = 0, heads = 0, d = 0, N = 0, st = 0, sh = 0;
};

int as_int(long long x, const char* what) {
  if (x < 0 || x > INT32_MAX) refuse(std::string(what) + " is out of range");
  return (int)x;
}

Rows rows_of(const at::Tensor& t, const char* name) {
  const int64_t n = t.dim();
  if (t.scalar_type() != at::kBFloat16 || (n != 3 && n != 4) || t.stride(n - 1) != 1)
    refuse(std::string(name) + " must be a bfloat16 CUDA tensor [T, heads, d] or [B, N, heads, d] with contiguous rows");
  Rows r;
  r.heads = t.size(n - 2), r.d = t.size(n - 1);
  r.sh = r.heads > 1 ? t.stride(n - 2) : r.d;   // a stride of one head or one token says nothing
  if (n == 3) {
    r.T = r.N = t.size(0), r.st = t.stride(0);
  } else {
    const int64_t B = t.size(0);
    r.N = t.size(1), r.T = B * r.N, r.st = r.N == 1 ? t.stride(0) : t.stride(1);
    if (r.N > 1 && B > 1 && t.stride(0) != r.N * t.stride(1))
      refuse(std::string("the tokens of ") + name + " must be evenly spaced over the batch");
  }
  if (r.T == 1) r.st = r.heads * r.d;
  return r;
}

struct Rope {   // angle tables [max_pos, rope_dim / 2]
  const float *cos = nullptr, *sin = nullptr;
  int dim = 0, max_pos = 0;
};

// For tokens of them: a table without entries has no address, and would read as none given.
Rope rope_of(const at::Tensor* cos, const at::Tensor* sin, long long tokens) {
  Rope r;
  if (!cos && !sin) return r;
  if (!cos || !sin || cos->scalar_type() != at::kFloat || sin->scalar_type() != at::kFloat || cos->dim() != 2 ||
      cos->sizes() != sin->sizes() || !cos->is_contiguous() || !sin->is_contiguous())
    refuse("cos and sin must be contiguous float32 CUDA tensors [max_pos, rope_dim / 2], both or neither");
  if (tokens > 0 && cos->numel() == 0) refuse("cos and sin hold no angles");
  r.cos = (const float*)cos->data_ptr(), r.sin = (const float*)sin->data_ptr();
  r.dim = as_int(2 * cos->size(1), "rope_dim"), r.max_pos = as_int(cos->size(0), "max_pos");
  return r;
}

float* vector_of(const at::Tensor* w, const char* name, long long d) {
  if (!w) return nullptr;
  if (w->scalar_type() != at::kFloat || w->dim() != 1 || w->size(0) != d || !w->is_contiguous())
    refuse(std::string(name) + " must be a contiguous float32 CUDA tensor of d values");
  return (float*)w->data_ptr();
}

void check_like(const at::Tensor* t, const char* name, const at::Tensor& like) {
  if (t && (t->sizes() != like.sizes() || t->scalar_type() != at::kBFloat16 || !t->is_contiguous()))
    refuse(std::string(name) + " must be a contiguous bfloat16 CUDA tensor with the shape of its input");
}

// torch's allocator without its dispatcher: 0.5 us less an output.
at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

// A workspace argument; null for None. Its bytes are its values' only where it is contiguous.
const at::Tensor* workspace(PyObject* o) {
  const at::Tensor* t = tensor(o, "workspace");
  if (t && !t->is_contiguous()) refuse("workspace must be a contiguous CUDA tensor");
  return t;
}

// Memory of the call's own on the current stream: the tensor given, or an allocation that lives as long as this.
struct Workspace {
  c10::DataPtr made;
  void* ptr;
  size_t bytes;
  Workspace(const at::Tensor* given, size_t need) : ptr(pointer(given)), bytes(given ? given->nbytes() : need) {
    if (!given && need) made = c10::cuda::CUDACachingAllocator::get()->allocate(need), ptr = made.get();
  }
};

// An output: the tensor given, or a new one.
struct Out {
  PyObject* given;
  at::Tensor made;
  void* ptr = nullptr;
  Out(PyObject* o, const at::Tensor* t, at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) : given(o) {
    if (!t) made = make(sizes, type, like);
    ptr = t ? t->data_ptr() : made.data_ptr();
  }
  PyObject* object() {
    if (!made.defined()) return Py_INCREF(given), given;
    return THPVariable_Wrap(std::move(made));
  }
};

PyObject* none() { return Py_INCREF(Py_None), Py_None; }

// A tuple of new references; all are released if one is missing.
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  bool ok = t != nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    ok = ok && o;
    if (t) PyTuple_SET_ITEM(t, i++, o);   // null is allowed until the tuple goes
    else Py_XDECREF(o);
  }
  if (!ok) {
    Py_XDECREF(t);
    throw Raised();
  }
  return t;
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised();
  return x;
}

long long whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  return x;
}

int truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised();
  return x;
}

void check_status(attn_status_t st, const char* what) {
  if (st == ATTN_OK) return;
  PyObject* e = PyObject_CallFunction(g_attn_error, "is", (int)st, what);
  if (e) {
    PyErr_SetObject(g_attn_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// Runs f with C++ errors turned into Python's.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const WrongType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());   // as torch's own allocations do
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <class F>
attn_status_t launch(F&& f) {   // other Python threads run while a launch waits for room in its queue
  attn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// What the norm's forward and backward share: q, k, cos, sin, positions, wq, wk, eps, norm, interleaved, pair_axis (bytes, the
// axis of every pair; positions then hold one more dim, the axes; None: one axis).
struct NormRope {
  const at::Tensor &q, *k, *cos, *sin, *positions, *wq, *wk;
  float eps;
  int norm, interleaved;
  Rows rq, rk;
  Rope rope;
  const float *wqp, *wkp;
  int T, H, Hkv, d, N;
  int axes = 0;                            // 0: the entries with one axis
  const unsigned char* pair_axis = nullptr;

  explicit NormRope(PyObject* const* a)
      : q(needed(a[0], "q")), k(tensor(a[1], "k")), cos(tensor(a[2], "cos")), sin(tensor(a[3], "sin")),
        positions(tensor(a[4], "positions")), wq(tensor(a[5], "wq")), wk(tensor(a[6], "wk")),
        eps((float)number(a[7])), norm(truth(a[8])), interleaved(truth(a[9])) {
    rq = rows_of(q, "q");
    if (k) {
      rk = rows_of(*k, "k");
      if (k->dim() != q.dim() || rk.T != rq.T || rk.N != rq.N || rk.d != rq.d)
        refuse("q and k must hold the same tokens and values of one size");
    } else if (wk) {
      refuse("wk needs k");
    }
    if (a[10] != Py_None) {
      if (!PyBytes_Check(a[10])) throw WrongType("pair_axis must be bytes");
      pair_axis = (const unsigned char*)PyBytes_AS_STRING(a[10]);
      const int64_t n = q.dim() - 2;
      if (!positions || !cos || positions->scalar_type() != at::kInt || positions->dim() != n + 1 ||
          positions->sizes().slice(1) != q.sizes().slice(0, n) || !positions->is_contiguous())
        refuse("positions must be a contiguous int32 CUDA tensor [axes, ...], one per axis and token, with cos and sin");
      axes = as_int(positions->size(0), "the number of axes");
      if (axes < 1 || axes > 4 || cos->dim() != 2 || PyBytes_GET_SIZE(a[10]) != cos->size(1))
        refuse("pair_axis must hold the axis of every pair (a column of cos), of 1 to 4 axes");
    } else if (positions && (positions->scalar_type() != at::kInt || positions->sizes() != q.sizes().slice(0, q.dim() - 2) ||
                             !positions->is_contiguous())) {
      refuse("positions must be a contiguous int32 CUDA tensor, one per token");
    }
    rope = rope_of(cos, sin, rq.T);
    wqp = vector_of(wq, "wq", rq.d), wkp = vector_of(wk, "wk", rq.d);
    T = as_int(rq.T, "the number of tokens"), H = as_int(rq.heads, "heads"), Hkv = as_int(rk.heads, "heads");
    d = as_int(rq.d, "d"), N = as_int(rq.N, "the number of tokens");
  }
};

PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const NormRope x(a);
    const at::Tensor *qo = tensor(a[11], "q_out"), *ko = tensor(a[12], "k_out");
    if (ko && !x.k) refuse("k_out needs k");
    check_like(qo, "q_out", x.q);
    if (x.k) check_like(ko, "k_out", *x.k);
    const cudaStream_t s = launch_stream({&x.q, x.k, x.cos, x.sin, x.positions, x.wq, x.wk, qo, ko});
    Out q_out(a[11], qo, x.q.sizes(), at::kBFloat16, x.q);
    std::optional<Out> k_out;
    if (x.k) k_out.emplace(a[12], ko, x.k->sizes(), at::kBFloat16, x.q);
    if (x.T > 0)
      check_status(launch([&] {
        if (x.axes)
          return attn_qk_norm_rope_axes(x.q.data_ptr(), pointer(x.k), q_out.ptr, k_out ? k_out->ptr : nullptr, x.T, x.H, x.Hkv,
                                        x.d, x.rq.st, x.rq.sh, x.rk.st, x.rk.sh, x.norm, x.wqp, x.wkp, x.eps, x.rope.cos,
                                        x.rope.sin, x.rope.dim, x.rope.max_pos, x.interleaved, (const int*)pointer(x.positions),
                                        x.T, x.axes, x.pair_axis, s);
        return attn_qk_norm_rope(x.q.data_ptr(), pointer(x.k), q_out.ptr, k_out ? k_out->ptr : nullptr, x.T, x.H, x.Hkv, x.d,
                                 x.rq.st, x.rq.sh, x.rk.st, x.rk.sh, x.norm, x.wqp, x.wkp, x.eps, x.rope.cos, x.rope.sin,
                                 x.rope.dim, x.rope.max_pos, x.interleaved, (const int*)pointer(x.positions), x.N, s);
      }), x.axes ? "attn_qk_norm_rope_axes" : "attn_qk_norm_rope");
    return tuple({q_out.object(), k_out ? k_out->object() : none()});
  });
}

// The eleven shared arguments, then dq_out, dk_out, dq, dk, dwq, dwk, workspace.
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&] {
    const NormRope x(a);
    const at::Tensor &gq = needed(a[11], "dq_out"), *gk = tensor(a[12], "dk_out"), *dq = tensor(a[13], "dq"),
                     *dk = tensor(a[14], "dk"), *dwq = tensor(a[15], "dwq"), *dwk = tensor(a[16], "dwk"),
                     *ws = workspace(a[17]);
    if ((gk != nullptr) != (x.k != nullptr)) refuse("dk_out is given exactly with k");
    if ((dk && !x.k) || (dwq && !x.wq) || (dwk && !x.wk)) refuse("dk needs k, dwq needs wq and dwk needs wk");
    check_like(&gq, "dq_out", x.q), check_like(dq, "dq", x.q);
    if (x.k) check_like(gk, "dk_out", *x.k), check_like(dk, "dk", *x.k);
    vector_of(dwq, "dwq", x.d), vector_of(dwk, "dwk", x.d);
    const cudaStream_t s = launch_stream({&x.q, x.k, x.cos, x.sin, x.positions, x.wq, x.wk, &gq, gk, dq, dk, dwq, dwk, ws});
    Out o_q(a[13], dq, x.q.sizes(), at::kBFloat16, x.q);
    at::Tensor made_k, made_wq, made_wk;
    if (x.k && !dk) made_k = make(x.k->sizes(), at::kBFloat16, x.q), dk = &made_k;
    if (x.wq && !dwq) made_wq = make({x.d}, at::kFloat, x.q), dwq = &made_wq;
    if (x.wk && !dwk) made_wk = make({x.d}, at::kFloat, x.q), dwk = &made_wk;
    if (x.T == 0) {
      if (dwq) dwq->zero_();
      if (dwk) dwk->zero_();
    } else {
      const Workspace work(ws, dwq || dwk ? attn_qk_norm_rope_bwd_workspace_bytes(x.T, x.H, x.Hkv, x.d) : 0);
      check_status(launch([&] {
        if (x.axes)
          return attn_qk_norm_rope_axes_bwd(x.q.data_ptr(), pointer(x.k), gq.data_ptr(), pointer(gk), o_q.ptr, pointer(dk),
                                            (float*)pointer(dwq), (float*)pointer(dwk), x.T, x.H, x.Hkv, x.d, x.rq.st, x.rq.sh,
                                            x.rk.st, x.rk.sh, x.norm, x.wqp, x.wkp, x.eps, x.rope.cos, x.rope.sin, x.rope.dim,
                                            x.rope.max_pos, x.interleaved, (const int*)pointer(x.positions), x.T, x.axes,
                                            x.pair_axis, work.ptr, work.bytes, s);
        return attn_qk_norm_rope_bwd(x.q.data_ptr(), pointer(x.k), gq.data_ptr(), pointer(gk), o_q.ptr, pointer(dk),
                                     (float*)pointer(dwq), (float*)pointer(dwk), x.T, x.H, x.Hkv, x.d, x.rq.st, x.rq.sh,
                                     x.rk.st, x.rk.sh, x.norm, x.wqp, x.wkp, x.eps, x.rope.cos, x.rope.sin, x.rope.dim,
                                     x.rope.max_pos, x.interleaved, (const int*)pointer(x.positions), x.N, work.ptr, work.bytes,
                                     s);
      }), x.axes ? "attn_qk_norm_rope_axes_bwd" : "attn_qk_norm_rope_bwd");
    }
    auto object = [&](PyObject* given, const at::Tensor* t, at::Tensor& made) {
      if (!t) return none();
      return made.defined() ? THPVariable_Wrap(std::move(made)) : (Py_INCREF(given), given);
    };
    return tuple({o_q.object(), object(a[14], dk, made_k), object(a[15], dwq, made_wq), object(a[16], dwk, made_wk)});
  });
}

// A cache (address of its attn_paged_cache_t, device index), a page table int32 [B, max_pages] with contiguous rows.
struct Paged {
  const attn_paged_cache_t* cache;
  int device;
  const at::Tensor& table;
  long long stride;
  int B, max_pages;

  // launch_stream with the cache's tensors, which are all on one device (-1: the CPU)
  cudaStream_t stream(std::initializer_list<const at::Tensor*> tensors) const {
    if (device < 0) refuse_device("cpu");
    const cudaStream_t s = launch_stream(tensors);
    if (table.get_device() != device) refuse_device("cuda:" + std::to_string(device));
    return s;
  }

  Paged(PyObject* address, PyObject* dev, PyObject* t) : table(needed(t, "page_table")) {
    cache = (const attn_paged_cache_t*)PyLong_AsVoidPtr(address);
    if (!cache) throw Raised();
    device = (int)whole(dev);
    if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
      refuse("page_table must be an int32 CUDA tensor [B, max_pages] with contiguous rows");
    stride = table.stride(0), B = as_int(table.size(0), "B"), max_pages = as_int(table.size(1), "max_pages");
  }

  const int* ints(const at::Tensor& t, const char* name, int more) const {
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != (int64_t)B + more || !t.is_contiguous())
      refuse(std::string(name) + " must be a contiguous int32 CUDA tensor of " + std::to_string(B + more) + " values");
    return (const int*)t.data_ptr();
  }
};

// cache address, device, k, v, cu_seqlens, cache_lens, page_table, cos, sin, interleaved
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Paged p(a[0], a[1], a[6]);
    const at::Tensor &k = needed(a[2], "k"), &v = needed(a[3], "v"), &cu = needed(a[4], "cu_seqlens"),
                     &lens = needed(a[5], "cache_lens"), *cos = tensor(a[7], "cos"), *sin = tensor(a[8], "sin");
    const int* cup = p.ints(cu, "cu_seqlens", 1);
    const int* lenp = p.ints(lens, "cache_lens", 0);
    const Rows rk = rows_of(k, "k"), rv = rows_of(v, "v");
    if (k.dim() != 3 || v.sizes() != k.sizes() || rk.heads != p.cache->Hkv || rk.d != p.cache->d)
      refuse("k and v must be [total, Hkv, d] with the cache's heads");
    const Rope rope = rope_of(cos, sin, rk.T);
    const int total = as_int(rk.T, "the number of tokens"), interleaved = truth(a[9]);
    const cudaStream_t s = p.stream({&p.table, &k, &v, &cu, &lens, cos, sin});
    if (total > 0 && p.B > 0)
      check_status(launch([&] {
        return attn_paged_append(p.cache, k.data_ptr(), v.data_ptr(), rk.st, rk.sh, rv.st, rv.sh, cup, lenp,
                                 (const int*)p.table.data_ptr(), p.stride, p.max_pages, p.B, total, rope.cos, rope.sin,
                                 rope.dim, rope.max_pos, interleaved, s);
      }), "attn_paged_append");
    return none();
  });
}

// cache address, device, cu_seqlens, page_table, total, k, v
PyObject* paged_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Paged p(a[0], a[1], a[3]);
    const at::Tensor &cu = needed(a[2], "cu_seqlens"), *k = tensor(a[5], "k"), *v = tensor(a[6], "v");
    const int* cup = p.ints(cu, "cu_seqlens", 1);
    const int total = as_int(whole(a[4]), "total");
    const int64_t shape[3] = {total, p.cache->Hkv, p.cache->d};
    for (const at::Tensor* t : {k, v})
      if (t && (t->sizes() != at::IntArrayRef(shape, 3) || t->scalar_type() != at::kBFloat16 || !t->is_contiguous()))
        refuse("k and v must be contiguous bfloat16 CUDA tensors [total, Hkv, d]");
    const cudaStream_t s = p.stream({&p.table, &cu, k, v});
    Out ko(a[5], k, at::IntArrayRef(shape, 3), at::kBFloat16, p.table);
    Out vo(a[6], v, at::IntArrayRef(shape, 3), at::kBFloat16, p.table);
    if (total > 0 && p.B > 0)
      check_status(launch([&] {
        return attn_paged_gather(p.cache, ko.ptr, vo.ptr, cup, (const int*)p.table.data_ptr(), p.stride, p.max_pages, p.B,
                                 total, s);
      }), "attn_paged_gather");
    return tuple({ko.object(), vo.object()});
  });
}

// cache address, device, q, page_table, seqlens, causal, scale (None: 1 / sqrt(d)), workspace, out, lse
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Paged p(a[0], a[1], a[3]);
    const at::Tensor &q = needed(a[2], "q"), &lens = needed(a[4], "seqlens"), *ws = workspace(a[7]),
                     *out = tensor(a[8], "out"), *lse = tensor(a[9], "lse");
    const int* lenp = p.ints(lens, "seqlens", 0);
    if (q.dim() != 4 || q.scalar_type() != at::kBFloat16 || !q.is_contiguous())
      refuse("q must be a contiguous bfloat16 CUDA tensor [B, Nq, H, d]");
    const int Nq = as_int(q.size(1), "Nq"), H = as_int(q.size(2), "H"), d = p.cache->d;
    if (q.size(0) != p.B || q.size(3) != d || p.cache->Hkv <= 0 || H % p.cache->Hkv != 0)
      refuse("q must be [B, Nq, H, d] with the page table's B, the cache's d and a multiple of its heads");
    check_like(out, "out", q);
    const int64_t rows[3] = {p.B, H, Nq};
    if (lse && (lse->sizes() != at::IntArrayRef(rows, 3) || lse->scalar_type() != at::kFloat || !lse->is_contiguous()))
      refuse("lse must be a contiguous float32 CUDA tensor [B, H, Nq]");
    const int causal = truth(a[5]);
    const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)number(a[6]);
    const cudaStream_t s = p.stream({&p.table, &q, &lens, ws, out, lse});
    const bool any_rows = p.B > 0 && Nq > 0;   // nothing to launch for otherwise
    const Workspace work(ws, ws || !any_rows ? 0 : attn_fwd_paged_workspace_bytes(p.B, H, p.cache->Hkv, Nq, d, p.cache->type));
    Out o(a[8], out, q.sizes(), at::kBFloat16, q), l(a[9], lse, at::IntArrayRef(rows, 3), at::kFloat, q);
    if (any_rows)
      check_status(launch([&] {
        return attn_fwd_paged(q.data_ptr(), p.cache, o.ptr, (float*)l.ptr, (const int*)p.table.data_ptr(), p.stride, p.max_pages,
                              lenp, p.B, H, Nq, scale, causal, work.ptr, work.bytes, s);
      }), "attn_fwd_paged");
    return tuple({o.object(), l.object()});
  });
}

// cache address, device, q, page_table, cu_seqlens_q, seqlens, causal, scale (None: 1 / sqrt(d)), workspace, out, lse
PyObject* fwd_paged_varlen(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const Paged p(a[0], a[1], a[3]);
    const at::Tensor &q = needed(a[2], "q"), &cu = needed(a[4], "cu_seqlens_q"), &lens = needed(a[5], "seqlens"),
                     *ws = workspace(a[8]), *out = tensor(a[9], "out"), *lse = tensor(a[10], "lse");
    const int* cup = p.ints(cu, "cu_seqlens_q", 1);
    const int* lenp = p.ints(lens, "seqlens", 0);
    if (q.dim() != 3 || q.scalar_type() != at::kBFloat16 || !q.is_contiguous())
      refuse("q must be a contiguous bfloat16 CUDA tensor [total_q, H, d]");
    const int total = as_int(q.size(0), "total_q"), H = as_int(q.size(1), "H"), d = p.cache->d;
    if (q.size(2) != d || p.cache->Hkv <= 0 || H < 1 || H % p.cache->Hkv != 0)
      refuse("q must be [total_q, H, d] with the cache's d and a multiple of its heads");
    check_like(out, "out", q);
    const int64_t rows[2] = {H, total};
    if (lse && (lse->sizes() != at::IntArrayRef(rows, 2) || lse->scalar_type() != at::kFloat || !lse->is_contiguous()))
      refuse("lse must be a contiguous float32 CUDA tensor [H, total_q]");
    const int causal = truth(a[6]);
    const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)number(a[7]);
    const cudaStream_t s = p.stream({&p.table, &q, &cu, &lens, ws, out, lse});
    const bool any_rows = p.B > 0 && total > 0;   // nothing to launch for otherwise
    const Workspace work(ws, ws || !any_rows ? 0 : attn_fwd_paged_varlen_workspace_bytes(p.B, H, p.cache->Hkv, total, d, p.cache->type));
    Out o(a[9], out, q.sizes(), at::kBFloat16, q), l(a[10], lse, at::IntArrayRef(rows, 2), at::kFloat, q);
    if (any_rows)
      check_status(launch([&] {
        return attn_fwd_paged_varlen(q.data_ptr(), p.cache, o.ptr, (float*)l.ptr, (const int*)p.table.data_ptr(), p.stride,
                                     p.max_pages, cup, lenp, p.B, H, total, scale, causal, work.ptr, work.bytes, s);
      }), "attn_fwd_paged_varlen");
    return tuple({o.object(), l.object()});
  });
}

// AttnError, torch.OutOfMemoryError: once, before the first call.
PyObject* set_errors(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&] {
    Py_INCREF(a[0]), Py_INCREF(a[1]);
    Py_XSETREF(g_attn_error, a[0]);
    Py_XSETREF(g_out_of_memory, a[1]);
    return none();
  });
}

#define FAST(f) (PyCFunction)(void (*)())(f), METH_FASTCALL
PyMethodDef methods[] = {{"qk_norm_rope", FAST(qk_norm_rope), nullptr},
                         {"qk_norm_rope_bwd", FAST(qk_norm_rope_bwd), nullptr},
                         {"paged_append", FAST(paged_append), nullptr},
                         {"paged_gather", FAST(paged_gather), nullptr},
                         {"fwd_paged", FAST(fwd_paged), nullptr},
                         {"fwd_paged_varlen", FAST(fwd_paged_varlen), nullptr},
                         {"set_errors", FAST(set_errors), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }

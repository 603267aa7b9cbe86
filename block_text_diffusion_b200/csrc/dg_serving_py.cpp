// Python side of the serving operators (serving.py): tensor checks and
// marshalling in C++.  The calls take the GPU a few microseconds; doing this
// in Python took three times as long as the launch itself.  The work is in
// libdg.so, whose entry points serving.py hands over by address.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <initializer_list>

#include "../../include/dg.h"

namespace {

struct {
  decltype(&dg_qk_norm_rope) norm_rope;
  decltype(&dg_paged_append) append;
  decltype(&dg_paged_attention) attention;
  decltype(&dg_paged_attention_workspace) workspace;
  PyObject* error;   // DGError
} g;

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_ValueError, fmt, ap);
  va_end(ap);
  throw Refused{};
}

// Interned attribute names.
#define DG_NAMES(X)                                                                                                 \
  X(_at) X(index) X(inv_freq) X(q_gain) X(k_gain) X(k) X(v) X(cu_q) X(kv_lens) X(page_table) X(prefix_pages) X(_words) \
  X(cuda_stream) X(device)
#define X(n) PyObject* s_##n;
DG_NAMES(X)
#undef X

struct Ref {   // an owned reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {
    if (!o) throw Refused{};
  }
  ~Ref() { Py_DECREF(p); }
  Ref(const Ref&) = delete;
};

long long attr_int(PyObject* o, PyObject* name) {
  Ref v(PyObject_GetAttr(o, name));
  const long long x = PyLong_AsLongLong(v.p);
  if (x == -1 && PyErr_Occurred()) throw Refused{};
  return x;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "bfloat16" : t == at::kFloat ? "float32" : t == at::kDouble ? "float64" : "int32";
}

// Nothing is recorded for a backward pass, so a tensor that wants a gradient is
// an error while gradients are recorded, not one silently dropped.
void no_gradient(const at::Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    refuse("%s requires a gradient, which this call does not record: call it under torch.no_grad()", name);
}

// A tensor of a type and shape on a device.
const at::Tensor& check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int index,
                        bool contiguous) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != index ||
      (contiguous && !t.is_contiguous()) || t.layout() != at::kStrided) {
    Ref want(PyTuple_New((Py_ssize_t)shape.size()));
    for (size_t i = 0; i < shape.size(); ++i) PyTuple_SET_ITEM(want.p, (Py_ssize_t)i, PyLong_FromLongLong(shape[i]));
    refuse("%s must be a %s%s tensor of shape %R on cuda:%d", name, contiguous ? "contiguous " : "", type_name(type),
           want.p, index);
  }
  no_gradient(t, name);
  return t;
}

const at::Tensor& check(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int index,
                        bool contiguous) {
  return check(tensor(o, name), name, type, shape, index, contiguous);
}

// [tokens, heads, head_dim] with contiguous components.
dg_heads rows(PyObject* o, const char* name, at::ScalarType type, int64_t tokens, int64_t heads, int64_t dim, int index,
              bool out) {
  const int64_t shape[3] = {tokens, heads, dim};
  const at::Tensor& t = check(o, name, type, at::IntArrayRef(shape, 3), index, false);
  // (the stride of a dimension of one entry means nothing)
  const int64_t st = tokens == 1 ? 0 : t.stride(0), sh = heads == 1 ? 0 : t.stride(1), n = tokens * heads;
  if (t.stride(2) != 1 && dim > 1 && n > 0) refuse("%s: the components of a head must be contiguous", name);
  if (out && n > 0) {
    // rows that share memory would be written by several warps at once
    const bool heads_inner = sh <= st;
    const int64_t a = heads_inner ? sh : st, na = heads_inner ? heads : tokens;
    const int64_t b = heads_inner ? st : sh, nb = heads_inner ? tokens : heads;
    if ((na > 1 && a < dim) || (nb > 1 && b < (na - 1) * a + dim)) refuse("%s: rows overlap", name);
  }
  return dg_heads{t.data_ptr(), st, sh};
}

at::ScalarType model_type(const at::Tensor& t) {
  if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16) refuse("tensors must be float32 or bfloat16");
  return t.scalar_type();
}

// A tensor whose address an argument object noted when it was made: its memory
// may have been replaced since (a module moved to another type or device).
// What else was noted (shape, type, order) is checked beside it.
const at::Tensor& held(PyObject* o, const char* name, const void* noted) {
  const at::Tensor& t = tensor(o, name);
  if (t.data_ptr() != noted) refuse("%s has other memory than when it was given: make the argument object anew", name);
  return t;
}
const at::Tensor& held(const Ref& r, const char* name, const void* noted) { return held(r.p, name, noted); }

const dg_rope* rope_of(PyObject* o, int index) {
  if (o == Py_None) return nullptr;
  Ref freq(PyObject_GetAttr(o, s_inv_freq));   // (only a Rope has it)
  const dg_rope* r = reinterpret_cast<const dg_rope*>(attr_int(o, s__at));
  const int64_t pairs = r->rot_dim / 2;
  check(held(freq, "inv_freq", r->inv_freq), "inv_freq", at::kDouble, at::IntArrayRef(&pairs, 1), index, true);
  return r;
}

const dg_head_norm* norm_of(PyObject* o, at::ScalarType type, int64_t dim, int index) {
  if (o == Py_None) return nullptr;
  Ref q_gain(PyObject_GetAttr(o, s_q_gain)), k_gain(PyObject_GetAttr(o, s_k_gain));   // (only a HeadNorm has them)
  const dg_head_norm* h = reinterpret_cast<const dg_head_norm*>(attr_int(o, s__at));
  if (q_gain.p != Py_None) check(held(q_gain, "q_gain", h->q_gain), "q_gain", type, at::IntArrayRef(&dim, 1), index, true);
  if (k_gain.p != Py_None) check(held(k_gain, "k_gain", h->k_gain), "k_gain", type, at::IntArrayRef(&dim, 1), index, true);
  return h;
}

struct Cache {
  const dg_paged_kv* c;
  at::ScalarType type;
  int index;
  PyObject *k, *v;   // the cache's, which lives as long as the call
};
Cache cache_of(PyObject* o) {
  Cache r;
  Ref k(PyObject_GetAttr(o, s_k)), v(PyObject_GetAttr(o, s_v));   // (only a PagedKV has them)
  r.c = reinterpret_cast<const dg_paged_kv*>(attr_int(o, s__at));
  r.k = k.p;
  r.v = v.p;
  r.index = (int)attr_int(o, s_index);
  r.type = r.c->dtype == DG_BF16 ? at::kBFloat16 : at::kFloat;
  const int64_t shape[4] = {r.c->n_pages, r.c->n_kv_heads, r.c->page_size, r.c->head_dim};
  check(held(k, "the cache's k", r.c->k), "the cache's k", r.type, at::IntArrayRef(shape, 4), r.index, true);
  check(held(v, "the cache's v", r.c->v), "the cache's v", r.type, at::IntArrayRef(shape, 4), r.index, true);
  return r;
}

dg_paged_batch batch_of(PyObject* o, const Cache& c, int64_t tokens) {
  // index, n_seqs, the addresses, entries of prefix_pages; the four tensors
  Ref w(PyObject_GetAttr(o, s__words));
  long long v[10];
  if (!PyTuple_Check(w.p) || PyTuple_GET_SIZE(w.p) != 14) refuse("batch must be a PagedBatch");
  for (int i = 0; i < 10; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(w.p, i));
    if (v[i] == -1 && PyErr_Occurred()) throw Refused{};
  }
  if (v[0] != c.index) refuse("the batch and the cache are on different devices");
  dg_paged_batch b;
  b.n_seqs = (int32_t)v[1];
  if (tokens >= (1ll << 31)) refuse("too many tokens");
  b.n_tokens = (int32_t)tokens;
  b.cu_q = (const int32_t*)v[2];
  b.kv_lens = (const int32_t*)v[3];
  b.page_table = (const int32_t*)v[4];
  b.table_stride = v[5];
  b.max_pages = (int32_t)v[6];
  b.prefix_pages = (const int32_t*)v[7];
  b.prefix_len = (int32_t)v[8];
  // every tensor still has the memory and the shape that were noted (a table
  // that grew in place moved, and the old memory belongs to someone else)
  auto same = [&](int i, const char* name, const void* noted, at::IntArrayRef shape, bool contiguous) -> const at::Tensor& {
    return check(held(PyTuple_GET_ITEM(w.p, 10 + i), name, noted), name, at::kInt, shape, c.index, contiguous);
  };
  const int64_t offsets = v[1] + 1, seqs = v[1], table[2] = {v[1], v[6]}, prefix = v[9];
  same(0, "cu_q", b.cu_q, at::IntArrayRef(&offsets, 1), true);
  same(1, "kv_lens", b.kv_lens, at::IntArrayRef(&seqs, 1), true);
  const at::Tensor& t = same(2, "page_table", b.page_table, at::IntArrayRef(table, 2), false);
  if (std::max(t.stride(0), t.size(1)) != b.table_stride || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("page_table has other strides than when it was given: make the argument object anew");
  if (b.prefix_len > 0) same(3, "prefix_pages", b.prefix_pages, at::IntArrayRef(&prefix, 1), true);
  if (v[9] * c.c->page_size < b.prefix_len) refuse("prefix_pages has fewer pages than prefix_len needs");
  return b;
}

int32_t* status_of(PyObject* o, int index) {
  if (o == Py_None) return nullptr;
  const int64_t one = 1;
  return (int32_t*)check(o, "status", at::kInt, at::IntArrayRef(&one, 1), index, true).data_ptr();
}

// The tensors' device is current for the length of a call.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  const int index;
  void* stream;
  bool other = false;   // a stream of the caller's, not the current one
  On(int index_, PyObject* s) : index(index_) {
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    if (s != Py_None) {
      Ref dev(PyObject_GetAttr(s, s_device));
      if (attr_int(dev.p, s_index) != index) refuse("stream must be one of cuda:%d", index);
      void* const own = (void*)attr_int(s, s_cuda_stream);
      other = own != stream;
      stream = own;
    }
    if (c10::cuda::current_device() != index) guard.set_index((c10::DeviceIndex)index);
  }
  // Tensors were mostly made on the current stream; freed while a call on
  // another still uses them, their memory must not be given out yet.
  void uses(PyObject* o) const {
    if (other && THPVariable_Check(o))
      c10::cuda::CUDACachingAllocator::recordStream(
          THPVariable_Unpack(o).storage().data_ptr(),
          c10::cuda::getStreamFromExternal((cudaStream_t)stream, (c10::DeviceIndex)index));
  }
  void uses(PyObject* o, std::initializer_list<PyObject*> names) const {   // an argument object's tensors
    if (!other || o == Py_None) return;
    for (PyObject* n : names) {
      Ref t(PyObject_GetAttr(o, n));
      uses(t.p);
    }
  }
};

// A tensor the call writes: what autograd saved of it is no longer what it was.
// (Inference tensors keep no count.)
void wrote(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Ends a call whose outputs are `out`.
PyObject* finish(dg_status st, const char* name, std::initializer_list<PyObject*> out) {
  if (st == DG_OK) {
    for (PyObject* o : out) wrote(o);
    Py_RETURN_NONE;
  }
  Ref args(Py_BuildValue("(is)", (int)st, name));
  Ref e(PyObject_CallObject(g.error, args.p));
  PyErr_SetObject(g.error, e.p);
  return nullptr;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  try {
    if (n != want) refuse("wrong number of arguments");
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {   // no exception leaves an entry point
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (q, k, positions, q_out, k_out, rope, norm, stream)
PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    PyObject *q = a[0], *k = a[1];
    const at::Tensor& x = tensor(q != Py_None ? q : k, "q or k");
    if (!x.is_cuda() || x.dim() != 3) refuse("q or k must be a 3-D tensor on a GPU");
    if ((q == Py_None) != (a[3] == Py_None) || (k == Py_None) != (a[4] == Py_None))
      refuse("q and q_out, k and k_out go together");
    const at::ScalarType type = model_type(x);
    const int64_t tokens = x.size(0), dim = x.size(2);
    const int index = x.get_device();
    int64_t hq = 0, hk = 0;
    dg_heads qr{}, qo{}, kr{}, ko{};
    if (q != Py_None) {
      hq = x.size(1);
      qr = rows(q, "q", type, tokens, hq, dim, index, false);
      qo = rows(a[3], "q_out", type, tokens, hq, dim, index, true);
    }
    if (k != Py_None) {
      const at::Tensor& t = tensor(k, "k");
      hk = t.dim() == 3 ? t.size(1) : 0;
      kr = rows(k, "k", type, tokens, hk, dim, index, false);
      ko = rows(a[4], "k_out", type, tokens, hk, dim, index, true);
    }
    if (std::max({tokens, hq, hk, dim}) >= (1ll << 31)) refuse("too many tokens");
    const int32_t* positions = nullptr;
    if (a[2] != Py_None)
      positions = (const int32_t*)check(a[2], "positions", at::kInt, at::IntArrayRef(&tokens, 1), index, true).data_ptr();
    const dg_rope* rope = rope_of(a[5], index);
    if (rope && a[2] == Py_None) refuse("rope needs positions");
    const dg_head_norm* norm = norm_of(a[6], type, dim, index);
    On on(index, a[7]);
    for (int i : {0, 1, 2, 3, 4}) on.uses(a[i]);
    on.uses(a[5], {s_inv_freq});
    on.uses(a[6], {s_q_gain, s_k_gain});
    return finish(g.norm_rope(type == at::kBFloat16 ? DG_BF16 : DG_FP32, (int32_t)tokens, (int32_t)hq, (int32_t)hk,
                              (int32_t)dim, &qr, &qo, &kr, &ko, positions, rope, norm, on.stream),
                  "dg_qk_norm_rope", {a[3], a[4]});
  });
}

// (cache, batch, k, v, rope, norm, q, q_out, status, stream)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Cache c = cache_of(a[0]);
    const at::Tensor& k = tensor(a[2], "k");
    if (k.dim() != 3) refuse("k must be a 3-D tensor");
    if ((a[6] == Py_None) != (a[7] == Py_None)) refuse("q and q_out go together");
    const int64_t tokens = k.size(0), hk = c.c->n_kv_heads, dim = c.c->head_dim;
    const dg_heads kr = rows(a[2], "k", c.type, tokens, hk, dim, c.index, false);
    const dg_heads vr = rows(a[3], "v", c.type, tokens, hk, dim, c.index, false);
    int64_t hq = 0;
    dg_heads qr{}, qo{};
    if (a[6] != Py_None) {
      const at::Tensor& q = tensor(a[6], "q");
      hq = q.dim() == 3 ? q.size(1) : 0;
      if (hq >= (1ll << 31)) refuse("too many heads");
      qr = rows(a[6], "q", c.type, tokens, hq, dim, c.index, false);
      qo = rows(a[7], "q_out", c.type, tokens, hq, dim, c.index, true);
    }
    const dg_rope* rope = rope_of(a[4], c.index);
    const dg_head_norm* norm = norm_of(a[5], c.type, dim, c.index);
    const dg_paged_batch b = batch_of(a[1], c, tokens);
    int32_t* status = status_of(a[8], c.index);
    On on(c.index, a[9]);
    for (int i : {2, 3, 6, 7, 8}) on.uses(a[i]);
    on.uses(c.k);
    on.uses(c.v);
    on.uses(a[1], {s_cu_q, s_kv_lens, s_page_table, s_prefix_pages});
    on.uses(a[4], {s_inv_freq});
    on.uses(a[5], {s_q_gain, s_k_gain});
    return finish(g.append(c.c, &b, &kr, &vr, rope, norm, (int32_t)hq, &qr, &qo, status, on.stream), "dg_paged_append",
                  {c.k, c.v, a[7], a[8]});
  });
}

// (cache, batch, q, out, scale or None, causal, lse, workspace or None, status, stream); without a
// workspace: the number of bytes the call needs, and nothing runs
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Cache c = cache_of(a[0]);
    const at::Tensor& q = tensor(a[2], "q");
    if (q.dim() != 3) refuse("q must be a 3-D tensor");
    const int64_t tokens = q.size(0), hq = q.size(1), dim = c.c->head_dim;
    const dg_heads qr = rows(a[2], "q", c.type, tokens, hq, dim, c.index, false);
    const dg_heads o = rows(a[3], "out", c.type, tokens, hq, dim, c.index, true);
    if (hq < 1 || hq >= (1ll << 31) || hq % c.c->n_kv_heads)
      refuse("%lld query heads over %d key heads", (long long)hq, c.c->n_kv_heads);
    float* lse = nullptr;
    if (a[6] != Py_None) {
      const int64_t shape[2] = {tokens, hq};
      lse = (float*)check(a[6], "lse", at::kFloat, at::IntArrayRef(shape, 2), c.index, true).data_ptr();
    }
    const dg_paged_batch b = batch_of(a[1], c, tokens);
    double scale;
    if (a[4] == Py_None) {
      scale = 1.0 / std::sqrt((double)dim);
    } else {
      scale = PyFloat_AsDouble(a[4]);
      if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
    }
    const int causal = PyObject_IsTrue(a[5]);
    if (causal < 0) throw Refused{};
    int32_t* status = status_of(a[8], c.index);
    if (a[7] == Py_None)
      return PyLong_FromSize_t(g.workspace(b.n_tokens, (int32_t)hq, (int32_t)dim, b.prefix_len > 0));
    const at::Tensor& ws = tensor(a[7], "workspace");
    if (ws.scalar_type() != at::kByte || ws.dim() != 1 || !ws.is_cuda() || ws.get_device() != c.index || !ws.is_contiguous())
      refuse("workspace must be a contiguous 1-D uint8 tensor on cuda:%d", c.index);
    On on(c.index, a[9]);
    for (int i : {2, 3, 6, 7, 8}) on.uses(a[i]);
    on.uses(c.k);
    on.uses(c.v);
    on.uses(a[1], {s_cu_q, s_kv_lens, s_page_table, s_prefix_pages});
    return finish(g.attention(c.c, &b, (int32_t)hq, &qr, (float)scale, causal, &o, lse, ws.data_ptr(),
                              (size_t)ws.numel(), status, on.stream),
                  "dg_paged_attention", {a[3], a[6], a[7], a[8]});
  });
}

// (addresses of the four entry points of libdg.so, DGError)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    void* p[4];
    for (int i = 0; i < 4; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) {
        if (PyErr_Occurred()) throw Refused{};
        refuse("a missing entry point");
      }
    }
    g.norm_rope = (decltype(g.norm_rope))p[0];
    g.append = (decltype(g.append))p[1];
    g.attention = (decltype(g.attention))p[2];
    g.workspace = (decltype(g.workspace))p[3];
    Py_INCREF(a[4]);
    Py_XDECREF(g.error);
    g.error = a[4];
    Py_RETURN_NONE;
  });
}

PyMethodDef kMethods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, nullptr},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))py_norm_rope, METH_FASTCALL, nullptr},
    {"paged_append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) {
#define X(n) \
  if (!(s_##n = PyUnicode_InternFromString(#n))) return nullptr;
  DG_NAMES(X)
#undef X
  return PyModule_Create(&kModule);
}

// Python fast path of the operators round the paged cache and of those for
// serving a batch (the module _fast).
//
// A decode step calls these operators once a layer, next to kernels of a few
// microseconds, and checking a dozen tensors' types, shapes and devices from
// Python and marshalling twenty arguments through ctypes took 4 to 15 of them
// (rope 6.6 us a call, kv_append 12.5, of which the library's own part is 2).
// Here the same checks read the tensors directly. A call whose arguments are
// all as expected goes straight to the C ABI and its status is returned; any
// other returns None, and the caller in qsa.py goes through the checks that
// say what is wrong. No arithmetic, no state but the entry points' addresses.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "qsa_serve.h"

namespace {

decltype(&qsa_rope) p_rope;
decltype(&qsa_kv_append) p_append;
decltype(&qsa_kv_gather) p_gather;
decltype(&qsa_paged_attn) p_attn;
decltype(&qsa_prefix_attn) p_prefix;
decltype(&qsa_kv_weight) p_weight;
decltype(&qsa_kv_evict) p_evict;
decltype(&qsa_verify_drafts) p_verify;
PyObject* g_current_device;  // torch.cuda's current device and raw stream, as Python callables
PyObject* g_raw_stream;

// A ctypes structure's memory.
template <typename T>
class Struct {
 public:
  explicit Struct(PyObject* o) {
    if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      return;
    }
    held_ = true;
    if ((size_t)view_.len == sizeof(T)) p = static_cast<const T*>(view_.buf);
  }
  ~Struct() {
    if (held_) PyBuffer_Release(&view_);
  }
  Struct(const Struct&) = delete;
  Struct& operator=(const Struct&) = delete;
  const T* p = nullptr;

 private:
  Py_buffer view_;
  bool held_ = false;
};

// The current device and the stream of a call (`o`: None, a raw handle or a
// stream object); false: it has none (no device, no such stream).
struct Where {
  long device = -1;
  void* stream = nullptr;
  bool get(PyObject* o) {
    const bool ok = find(o);
    if (!ok) PyErr_Clear();
    return ok;
  }

 private:
  bool find(PyObject* o) {
    PyObject* d = PyObject_CallNoArgs(g_current_device);
    if (!d) return false;
    device = PyLong_AsLong(d);
    PyObject* s = nullptr;
    if (o == Py_None) {
      s = PyObject_CallOneArg(g_raw_stream, d);
    } else if (PyLong_Check(o)) {
      s = Py_NewRef(o);
    } else {
      s = PyObject_GetAttrString(o, "cuda_stream");
      if (!s && PyErr_ExceptionMatches(PyExc_AttributeError)) {
        PyErr_Clear();
        s = PyNumber_Long(o);
      }
    }
    Py_DECREF(d);
    if (!s) return false;
    stream = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return !PyErr_Occurred();
  }
};

const at::Tensor* tensor(PyObject* o, long device, at::ScalarType type) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type) return nullptr;
  return &t;
}

bool has_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) {
  return t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
}

// Address of a contiguous tensor of this type and shape; null where it is not
// (or holds nothing).
void* dense(PyObject* o, long device, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const at::Tensor* t = tensor(o, device, type);
  return t && has_shape(*t, shape) && t->is_contiguous() ? t->data_ptr() : nullptr;
}

// A BF16 [batch][token][head][dim] tensor with a contiguous last dimension.
struct Rows {
  void* p = nullptr;
  qsa_strides st;
  explicit Rows(const at::Tensor* t) {
    if (t && t->dim() == 4 && t->stride(3) == 1) {
      p = t->data_ptr();
      st = {t->stride(0), t->stride(1), t->stride(2)};
    }
  }
  Rows(PyObject* o, long device, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(o, device, at::kBFloat16);
    if (t && has_shape(*t, shape) && t->stride(3) == 1) {
      p = t->data_ptr();
      st = {t->stride(0), t->stride(1), t->stride(2)};
    }
  }
};

// The paged cache's addresses.
struct Cache {
  void *k = nullptr, *v = nullptr, *table = nullptr;
  float *ks = nullptr, *vs = nullptr;
  bool get(const qsa_dims& d, long dev, PyObject* const* a) {  // k_cache, v_cache, k_scale, v_scale, page_table
    const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
    const at::ScalarType type = fp8 ? at::kByte : at::kBFloat16;
    k = dense(a[0], dev, type, {d.num_pages, d.n_kv_heads, d.page_size, d.head_dim});
    v = dense(a[1], dev, type, {d.num_pages, d.n_kv_heads, d.page_size, d.head_dim});
    if (fp8 || a[2] != Py_None || a[3] != Py_None) {
      ks = static_cast<float*>(dense(a[2], dev, at::kFloat, {d.n_kv_heads}));
      vs = static_cast<float*>(dense(a[3], dev, at::kFloat, {d.n_kv_heads}));
      if (!ks || !vs) return false;
    }
    table = dense(a[4], dev, at::kInt, {d.batch, d.max_pages});
    return k && v && table;
  }
};

struct Workspace {
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, long device) {
    if (!THPVariable_Check(o)) return;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) return;
    p = t.data_ptr();
    bytes = t.nbytes();
  }
};

bool small_int(PyObject* o, long& v) {
  if (!PyLong_Check(o)) return false;
  v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return v >= 0 && v <= INT32_MAX;
}

template <typename F>
PyObject* call(F&& f) {
  qsa_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong((long)st);
}

const int32_t* i32(void* p) { return static_cast<const int32_t*>(p); }

// rope(args, table_device, x, pos, y, inverse, stream)
PyObject* fast_rope(PyObject* const* a, Py_ssize_t n) {
  if (n != 7) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[6])) Py_RETURN_NONE;
  long table_device, inverse;
  if (!small_int(a[1], table_device) || table_device != w.device || !small_int(a[5], inverse)) Py_RETURN_NONE;
  Struct<qsa_rope_args> rope(a[0]);
  const at::Tensor* x = tensor(a[2], w.device, at::kBFloat16);
  if (!rope.p || !x || x->dim() != 4) Py_RETURN_NONE;
  const int64_t B = x->size(0), N = x->size(1), H = x->size(2), D = x->size(3);
  if (B > INT32_MAX || N > INT32_MAX || H > INT32_MAX || D > INT32_MAX) Py_RETURN_NONE;
  const Rows xs(x), ys(a[4], w.device, {B, N, H, D});
  void* pos = dense(a[3], w.device, at::kInt, {B, N});
  if (!xs.p || !ys.p || !pos) Py_RETURN_NONE;
  return call([&] {
    return p_rope(rope.p, (int32_t)B, (int32_t)N, (int32_t)H, (int32_t)D, (int32_t)inverse, xs.p, &xs.st, i32(pos),
                  ys.p, &ys.st, w.stream);
  });
}

// kv_append(d, k, v, k_cache, v_cache, k_scale, v_scale, page_table, pos, ws, rope args or None, rope's device, q,
//           q_out, stream)
PyObject* fast_append(PyObject* const* a, Py_ssize_t n) {
  if (n != 15) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[14])) Py_RETURN_NONE;
  Struct<qsa_dims> d(a[0]);
  const at::Tensor* kt = tensor(a[1], w.device, at::kBFloat16);
  if (!d.p || !kt || kt->dim() != 4 || kt->size(1) > INT32_MAX) Py_RETURN_NONE;
  const int64_t N = kt->size(1), D = d.p->head_dim, hk = d.p->n_kv_heads;
  const Rows k(a[1], w.device, {d.p->batch, N, hk, D}), v(a[2], w.device, {d.p->batch, N, hk, D});
  Cache c;
  void* pos = dense(a[8], w.device, at::kInt, {d.p->batch, N});
  const Workspace ws(a[9], w.device);
  if (!k.p || !v.p || !c.get(*d.p, w.device, a + 3) || !pos || !ws.p) Py_RETURN_NONE;
  if (a[10] == Py_None) {
    if (a[12] != Py_None || a[13] != Py_None) Py_RETURN_NONE;
    return call([&] {
      return p_append(d.p, (int32_t)N, nullptr, k.p, &k.st, v.p, &v.st, nullptr, nullptr, nullptr, nullptr, i32(pos),
                      i32(c.table), c.k, c.v, c.ks, c.vs, ws.p, ws.bytes, w.stream);
    });
  }
  long table_device;
  Struct<qsa_rope_args> rope(a[10]);
  if (!rope.p || !small_int(a[11], table_device) || table_device != w.device) Py_RETURN_NONE;
  const bool with_q = a[12] != Py_None;
  if (with_q != (a[13] != Py_None)) Py_RETURN_NONE;
  const int64_t hq = d.p->n_q_heads;
  const Rows q = with_q ? Rows(a[12], w.device, {d.p->batch, N, hq, D}) : Rows(nullptr);
  const Rows qo = with_q ? Rows(a[13], w.device, {d.p->batch, N, hq, D}) : Rows(nullptr);
  if (with_q && (!q.p || !qo.p)) Py_RETURN_NONE;
  return call([&] {
    return p_append(d.p, (int32_t)N, rope.p, k.p, &k.st, v.p, &v.st, q.p, &q.st, qo.p, &qo.st, i32(pos), i32(c.table),
                    c.k, c.v, c.ks, c.vs, ws.p, ws.bytes, w.stream);
  });
}

// kv_gather(d, k_cache, v_cache, k_scale, v_scale, page_table, pos, k_out, v_out, ws, stream)
PyObject* fast_gather(PyObject* const* a, Py_ssize_t n) {
  if (n != 11) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[10])) Py_RETURN_NONE;
  Struct<qsa_dims> d(a[0]);
  const at::Tensor* pt = tensor(a[6], w.device, at::kInt);
  if (!d.p || !pt || pt->dim() != 2 || pt->size(1) > INT32_MAX) Py_RETURN_NONE;
  const int64_t N = pt->size(1), D = d.p->head_dim, hk = d.p->n_kv_heads;
  void* pos = dense(a[6], w.device, at::kInt, {d.p->batch, N});
  void* ko = dense(a[7], w.device, at::kBFloat16, {d.p->batch, N, hk, D});
  void* vo = dense(a[8], w.device, at::kBFloat16, {d.p->batch, N, hk, D});
  Cache c;
  const Workspace ws(a[9], w.device);
  if (!pos || !ko || !vo || !c.get(*d.p, w.device, a + 1) || !ws.p) Py_RETURN_NONE;
  return call([&] {
    return p_gather(d.p, (int32_t)N, c.k, c.v, c.ks, c.vs, i32(c.table), i32(pos), ko, vo, ws.p, ws.bytes, w.stream);
  });
}

// paged_attn(d, window, q, k_cache, v_cache, k_scale, v_scale, page_table, q_pos, out, lse, ws, stream)
PyObject* fast_attn(PyObject* const* a, Py_ssize_t n) {
  if (n != 13) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[12])) Py_RETURN_NONE;
  Struct<qsa_dims> d(a[0]);
  long window;
  if (!d.p || !small_int(a[1], window)) Py_RETURN_NONE;
  const int64_t B = d.p->batch, nq = d.p->n_q, H = d.p->n_q_heads, D = d.p->head_dim;
  void* q = dense(a[2], w.device, at::kBFloat16, {B, nq, H, D});
  void* out = dense(a[9], w.device, at::kBFloat16, {B, nq, H, D});
  void* pos = dense(a[8], w.device, at::kInt, {B, nq});
  void* lse = a[10] == Py_None ? nullptr : dense(a[10], w.device, at::kFloat, {B, nq, H});
  Cache c;
  const Workspace ws(a[11], w.device);
  if (!q || !out || !pos || (a[10] != Py_None && !lse) || !c.get(*d.p, w.device, a + 3) || !ws.p) Py_RETURN_NONE;
  return call([&] {
    return p_attn(d.p, (int32_t)window, q, c.k, c.v, c.ks, c.vs, i32(c.table), i32(pos), out,
                  static_cast<float*>(lse), ws.p, ws.bytes, w.stream);
  });
}

// prefix_attn(d, q, k_cache, v_cache, k_scale, v_scale, prefix_table, page_table, q_pos, out, lse, ws, stream)
PyObject* fast_prefix(PyObject* const* a, Py_ssize_t n) {
  if (n != 13) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[12])) Py_RETURN_NONE;
  Struct<qsa_dims> d(a[0]);
  const at::Tensor* xt = tensor(a[6], w.device, at::kInt);
  if (!d.p || !xt || xt->dim() != 1 || xt->size(0) > INT32_MAX) Py_RETURN_NONE;
  const int64_t B = d.p->batch, nq = d.p->n_q, H = d.p->n_q_heads, D = d.p->head_dim, pages = xt->size(0);
  void* shared = dense(a[6], w.device, at::kInt, {pages});
  void* q = dense(a[1], w.device, at::kBFloat16, {B, nq, H, D});
  void* out = dense(a[9], w.device, at::kBFloat16, {B, nq, H, D});
  void* pos = dense(a[8], w.device, at::kInt, {B, nq});
  void* lse = a[10] == Py_None ? nullptr : dense(a[10], w.device, at::kFloat, {B, nq, H});
  Cache c;
  PyObject* const cache[5] = {a[2], a[3], a[4], a[5], a[7]};
  const Workspace ws(a[11], w.device);
  if (!shared || !q || !out || !pos || (a[10] != Py_None && !lse) || !c.get(*d.p, w.device, cache) || !ws.p)
    Py_RETURN_NONE;
  return call([&] {
    return p_prefix(d.p, (int32_t)pages, i32(shared), q, c.k, c.v, c.ks, c.vs, i32(c.table), i32(pos), out,
                    static_cast<float*>(lse), ws.p, ws.bytes, w.stream);
  });
}

// kv_weight(d, decay, q, k_cache, k_scale, page_table, q_pos, lse, weight, ws, stream)
PyObject* fast_weight(PyObject* const* a, Py_ssize_t n) {
  if (n != 11 || !PyFloat_Check(a[1])) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[10])) Py_RETURN_NONE;
  Struct<qsa_dims> d(a[0]);
  if (!d.p) Py_RETURN_NONE;
  const int64_t B = d.p->batch, nq = d.p->n_q, H = d.p->n_q_heads, D = d.p->head_dim, hk = d.p->n_kv_heads;
  const bool fp8 = d.p->kv_dtype == QSA_KV_FP8_E4M3, scaled = fp8 || a[4] != Py_None;
  void* q = dense(a[2], w.device, at::kBFloat16, {B, nq, H, D});
  void* k = dense(a[3], w.device, fp8 ? at::kByte : at::kBFloat16, {d.p->num_pages, hk, d.p->page_size, D});
  void* ks = scaled ? dense(a[4], w.device, at::kFloat, {hk}) : nullptr;
  void* table = dense(a[5], w.device, at::kInt, {B, d.p->max_pages});
  void* pos = dense(a[6], w.device, at::kInt, {B, nq});
  void* lse = dense(a[7], w.device, at::kFloat, {B, nq, H});
  void* weight = dense(a[8], w.device, at::kFloat, {B, (int64_t)d.p->max_pages * d.p->page_size});
  const Workspace ws(a[9], w.device);
  if (!q || !k || (scaled && !ks) || !table || !pos || !lse || !weight || !ws.p) Py_RETURN_NONE;
  const float decay = (float)PyFloat_AS_DOUBLE(a[1]);
  return call([&] {
    return p_weight(d.p, decay, q, k, static_cast<float*>(ks), i32(table), i32(pos), static_cast<float*>(lse),
                    static_cast<float*>(weight), ws.p, ws.bytes, w.stream);
  });
}

// kv_evict(d, k_cache, v_cache, page_table, page_table_out, length, weight, weight_out, kept, new_length, ws, sinks,
//          recent, stream)
PyObject* fast_evict(PyObject* const* a, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[13])) Py_RETURN_NONE;
  Struct<qsa_dims> d(a[0]);
  const at::Tensor *po = tensor(a[4], w.device, at::kInt), *kt = tensor(a[8], w.device, at::kInt);
  long sinks, recent;
  if (!d.p || !po || po->dim() != 2 || !kt || kt->dim() != 2 || !small_int(a[11], sinks) || !small_int(a[12], recent))
    Py_RETURN_NONE;
  const int64_t B = d.p->batch, D = d.p->head_dim, hk = d.p->n_kv_heads, ps = d.p->page_size;
  const int64_t pages = po->size(1), keep = kt->size(1);
  if (pages > INT32_MAX || keep > INT32_MAX) Py_RETURN_NONE;
  const at::ScalarType type = d.p->kv_dtype == QSA_KV_FP8_E4M3 ? at::kByte : at::kBFloat16;
  void* k = dense(a[1], w.device, type, {d.p->num_pages, hk, ps, D});
  void* v = dense(a[2], w.device, type, {d.p->num_pages, hk, ps, D});
  void* table = dense(a[3], w.device, at::kInt, {B, d.p->max_pages});
  void* table_out = dense(a[4], w.device, at::kInt, {B, pages});
  void* len = dense(a[5], w.device, at::kInt, {B});
  void* weight = dense(a[6], w.device, at::kFloat, {B, d.p->max_pages * ps});
  void* weight_out = dense(a[7], w.device, at::kFloat, {B, pages * ps});
  void* kept = dense(a[8], w.device, at::kInt, {B, keep});
  void* new_len = dense(a[9], w.device, at::kInt, {B});
  const Workspace ws(a[10], w.device);
  if (!k || !v || !table || !table_out || !len || !weight || !weight_out || !kept || !new_len || !ws.p) Py_RETURN_NONE;
  return call([&] {
    return p_evict(d.p, (int32_t)keep, (int32_t)sinks, (int32_t)recent, (int32_t)pages, i32(len),
                   static_cast<float*>(weight), i32(table), i32(table_out), k, v, static_cast<float*>(weight_out),
                   static_cast<int32_t*>(kept), static_cast<int32_t*>(new_len), ws.p, ws.bytes, w.stream);
  });
}

// Probabilities [batch][row][vocab] with a contiguous last dimension.
struct Probs {
  const void* p = nullptr;
  qsa_prob_strides st;
  Probs(const at::Tensor* t, int64_t B, int64_t rows, int64_t V) {
    if (t && t->dim() == 3 && t->size(0) == B && t->size(1) == rows && t->size(2) == V &&
        (V <= 1 || t->stride(2) == 1)) {
      p = t->data_ptr();
      st = {t->stride(0), t->stride(1)};
    }
  }
};

// verify_drafts(target, draft, tokens, uniform, accepted, out_tokens, ws, stream)
PyObject* fast_verify(PyObject* const* a, Py_ssize_t n) {
  if (n != 8 || !THPVariable_Check(a[0])) Py_RETURN_NONE;
  Where w;
  if (!w.get(a[7])) Py_RETURN_NONE;
  const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
  const at::Tensor* tt = tensor(a[0], w.device, type);
  if (!tt || tt->dim() != 3) Py_RETURN_NONE;
  const int64_t B = tt->size(0), nd = tt->size(1) - 1, V = tt->size(2);
  if (B > INT32_MAX || nd > INT32_MAX || V > INT32_MAX) Py_RETURN_NONE;
  const bool sampled = a[1] != Py_None;
  const Probs t(tt, B, nd + 1, V), q(sampled ? tensor(a[1], w.device, type) : nullptr, B, nd, V);
  void* tokens = dense(a[2], w.device, at::kInt, {B, nd});
  void* u = dense(a[3], w.device, at::kFloat, {B, nd + 1});
  void* accepted = dense(a[4], w.device, at::kInt, {B});
  void* out = dense(a[5], w.device, at::kInt, {B, nd + 1});
  const Workspace ws(a[6], w.device);
  if (!t.p || (sampled && !q.p) || !tokens || !u || !accepted || !out || !ws.p) Py_RETURN_NONE;
  return call([&] {
    return p_verify((int32_t)B, (int32_t)nd, (int32_t)V, type == at::kFloat ? QSA_PROB_F32 : QSA_PROB_BF16, t.p, &t.st,
                    q.p, &q.st, i32(tokens), static_cast<float*>(u), static_cast<int32_t*>(accepted),
                    static_cast<int32_t*>(out), ws.p, ws.bytes, w.stream);
  });
}

// bind(rope, kv_append, kv_gather, paged_attn, prefix_attn, kv_weight, kv_evict, verify_drafts, current_device,
// raw_stream): the entry points' addresses and torch's two callables
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kPoints = 8;
  if (n != kPoints + 2) {
    PyErr_SetString(PyExc_TypeError, "bind takes 10 arguments");
    return nullptr;
  }
  void* p[kPoints];
  for (int i = 0; i < kPoints; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
      return nullptr;
    }
  }
  p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
  p_append = reinterpret_cast<decltype(p_append)>(p[1]);
  p_gather = reinterpret_cast<decltype(p_gather)>(p[2]);
  p_attn = reinterpret_cast<decltype(p_attn)>(p[3]);
  p_prefix = reinterpret_cast<decltype(p_prefix)>(p[4]);
  p_weight = reinterpret_cast<decltype(p_weight)>(p[5]);
  p_evict = reinterpret_cast<decltype(p_evict)>(p[6]);
  p_verify = reinterpret_cast<decltype(p_verify)>(p[7]);
  Py_XSETREF(g_current_device, Py_NewRef(a[kPoints]));
  Py_XSETREF(g_raw_stream, Py_NewRef(a[kPoints + 1]));
  Py_RETURN_NONE;
}

// A function as Python calls it. What throws on the way (a tensor without
// storage, a sparse one) is not for the fast path either.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (...) {
    if (PyErr_Occurred()) PyErr_Clear();
    Py_RETURN_NONE;
  }
}

#define QSA_METHOD(name, fn) \
  { name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&(fn))), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {QSA_METHOD("bind", bind),
                          QSA_METHOD("rope", guarded<fast_rope>),
                          QSA_METHOD("kv_append", guarded<fast_append>),
                          QSA_METHOD("kv_gather", guarded<fast_gather>),
                          QSA_METHOD("paged_attn", guarded<fast_attn>),
                          QSA_METHOD("prefix_attn", guarded<fast_prefix>),
                          QSA_METHOD("kv_weight", guarded<fast_weight>),
                          QSA_METHOD("kv_evict", guarded<fast_evict>),
                          QSA_METHOD("verify_drafts", guarded<fast_verify>),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&kModule); }

// Native marshalling for the calls of the 4-bit cache and of 16-bit paged serving: checks torch
// tensors and hands their pointers to the C ABI. A decode step runs for a few microseconds; the same
// checks written in Python took about as long again.
//
// Every function takes its arguments by position and returns the call's ATTN_* code, or
// raises TypeError / ValueError for a tensor that does not fit. The C entry points come as
// addresses from the loaded library (bind), so this module links only against torch.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/gqa_attn.h"

namespace {

decltype(&kv_cache_append_q4) c_append;
decltype(&kv_cache_read_q4) c_read;
decltype(&gqa_attn_decode_q4) c_decode;
decltype(&gqa_attn_decode_step_q4) c_step;
decltype(&kv_cache_evict_q4) c_evict;
decltype(&kv_q4_record_bytes) c_record;
decltype(&kv_cache_append_paged) c_append_paged;
decltype(&gqa_attn_decode_paged) c_decode_paged;
decltype(&gqa_attn_decode_shared) c_decode_shared;
decltype(&gqa_attn_prefill_packed) c_prefill_packed;

// Raised inside a call; the Python error is set.
struct Raise {};

[[noreturn]] void fail(PyObject* type, const char* fn, const char* what) {
  PyErr_Format(type, "%s: %s", fn, what);
  throw Raise{};
}

// One call's arguments and the device its tensors must lie on.
struct Args {
  const char* fn;
  PyObject* const* v;
  int device = -1;

  const at::Tensor* tensor(int i, at::ScalarType type, const char* type_name, bool optional) {
    PyObject* o = v[i];
    if (o == Py_None) {
      if (optional) return nullptr;
      fail(PyExc_TypeError, fn, "a required tensor is None");
    }
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, fn, "expected a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type) {
      PyErr_Format(PyExc_TypeError, "%s: expected torch.%s", fn, type_name);
      throw Raise{};
    }
    if (!t.is_cuda()) fail(PyExc_ValueError, fn, "expected CUDA tensors");
    if (device < 0) device = c10::cuda::current_device();
    if (t.get_device() != device)
      fail(PyExc_ValueError, fn, "tensors must lie on the current CUDA device");
    if (!t.is_contiguous()) fail(PyExc_ValueError, fn, "tensors must be contiguous");
    return &t;
  }
  const at::Tensor* f32(int i, bool optional = false) {
    return tensor(i, at::kFloat, "float32", optional);
  }
  const at::Tensor* i32(int i, bool optional = false) {
    return tensor(i, at::kInt, "int32", optional);
  }
  const at::Tensor* u8(int i) { return tensor(i, at::kByte, "uint8", false); }

  long whole(int i) {
    const long x = PyLong_AsLong(v[i]);
    if (x == -1 && PyErr_Occurred()) throw Raise{};
    if (x < INT32_MIN || x > INT32_MAX) fail(PyExc_OverflowError, fn, "integer out of range");
    return x;
  }
  float real(int i) {
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1.0 && PyErr_Occurred()) throw Raise{};
    return static_cast<float>(x);
  }
  // A torch stream, or None: the current one.
  void* stream(int i) {
    if (v[i] == Py_None)
      return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    PyObject* h = PyObject_GetAttrString(v[i], "cuda_stream");
    if (!h) throw Raise{};
    void* s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!s && PyErr_Occurred()) throw Raise{};
    return s;
  }
  // attn_rope_params from the binding's ctypes structure, or None.
  bool rope(int i, attn_rope_params* rp) {
    if (v[i] == Py_None) return false;
    Py_buffer b;
    if (PyObject_GetBuffer(v[i], &b, PyBUF_SIMPLE) != 0) throw Raise{};
    const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(*rp));
    if (fits) *rp = *static_cast<const attn_rope_params*>(b.buf);
    PyBuffer_Release(&b);
    if (!fits) fail(PyExc_TypeError, fn, "params must be RopeParams");
    return true;
  }
  void check(bool ok, const char* what) {
    if (!ok) fail(PyExc_ValueError, fn, what);
  }
  // A 4-bit cache [B, Hkv, capacity, record bytes]; returns its capacity.
  int cache(const at::Tensor* t, int64_t B, int64_t Hkv, int64_t D) {
    check(t->dim() == 4 && t->size(0) == B && t->size(1) == Hkv &&
              t->size(3) == static_cast<int64_t>(c_record(static_cast<int>(D))) &&
              t->size(2) <= INT32_MAX,
          "cache must be [B, Hkv, capacity, kv_q4_record_bytes(D)]");
    return static_cast<int>(t->size(2));
  }
  void rows(const at::Tensor* t, int64_t B) {
    if (t) check(t->numel() == B, "start, pos and lengths hold one value per batch row");
  }
  void status(const at::Tensor* t) {
    if (t) check(t->numel() >= 1, "status holds one value");
  }
  void table(const attn_rope_params* rp, const at::Tensor* t, int64_t D) {
    if (!rp || !t) return;
    const int64_t n = rp->max_positions > 0 ? rp->max_positions : 8192;
    const int64_t R = rp->rope_dim > 0 ? rp->rope_dim : D;
    check(t->numel() >= n * (R / 2) * 2, "table is smaller than attn_rope_table_bytes");
  }
  void norm(const at::Tensor* t, int64_t D) {
    if (t) check(t->numel() == D, "norm weights must have head_dim elements");
  }
  void sizes(const at::Tensor* t) {
    for (int64_t n : t->sizes()) check(n <= INT32_MAX, "a dimension is too large");
  }
};

template <class T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

PyObject* run(const char* fn, PyObject* const* args, Py_ssize_t n, Py_ssize_t want,
              int (*call)(Args&)) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", fn, want, n);
    return nullptr;
  }
  try {
    Args a{fn, args};
    return PyLong_FromLong(call(a));
  } catch (const Raise&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// k, v, cache, start, max_start, params, table, k_norm_w, eps, k_out, pos, max_pos, window,
// status, stream
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("kv_cache_append_q4", args, n, 15, [](Args& a) {
    const at::Tensor *k = a.f32(0), *v = a.f32(1), *cache = a.u8(2), *start = a.i32(3);
    attn_rope_params rp;
    const bool rope = a.rope(5, &rp);
    const at::Tensor *table = a.f32(6, true), *nw = a.f32(7, true), *ko = a.f32(9, true),
                     *pos = a.i32(10, true), *status = a.i32(13, true);
    a.check(k->dim() == 4 && v->sizes() == k->sizes() && (!ko || ko->sizes() == k->sizes()),
            "inconsistent shapes");
    a.sizes(k);
    const int64_t B = k->size(0), Hkv = k->size(1), L = k->size(2), D = k->size(3);
    const int cap = a.cache(cache, B, Hkv, D);
    a.rows(start, B);
    a.rows(pos, B);
    a.status(status);
    a.table(rope ? &rp : nullptr, table, D);
    a.norm(nw, D);
    return c_append(ptr<float>(k), ptr<float>(v), ptr<float>(ko), B, Hkv, L, D,
                    ptr<int32_t>(start), a.whole(4), ptr<int32_t>(pos), a.whole(11),
                    rope ? &rp : nullptr, ptr<float>(table), ptr<float>(nw), a.real(8),
                    ptr<void>(cache), cap, a.whole(12), ptr<int32_t>(status), a.stream(14));
  });
}

// cache, k, v, start, max_start, window, status, stream
PyObject* read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("kv_cache_read_q4", args, n, 8, [](Args& a) {
    const at::Tensor *cache = a.u8(0), *k = a.f32(1), *v = a.f32(2), *start = a.i32(3),
                     *status = a.i32(6, true);
    a.check(k->dim() == 4 && v->sizes() == k->sizes(), "inconsistent shapes");
    a.sizes(k);
    const int64_t B = k->size(0), Hkv = k->size(1), L = k->size(2), D = k->size(3);
    const int cap = a.cache(cache, B, Hkv, D);
    a.rows(start, B);
    a.status(status);
    return c_read(ptr<void>(cache), cap, a.whole(5), ptr<float>(k), ptr<float>(v), B, Hkv, L, D,
                  ptr<int32_t>(start), a.whole(4), ptr<int32_t>(status), a.stream(7));
  });
}

// The workspace argument: any contiguous CUDA tensor of the device.
void workspace(Args& a, int i, void** p, size_t* bytes) {
  if (!THPVariable_Check(a.v[i])) fail(PyExc_TypeError, a.fn, "workspace must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(a.v[i]);
  a.check(t.is_cuda() && t.get_device() == a.device && t.is_contiguous(),
          "workspace must be a contiguous tensor on the current CUDA device");
  *p = t.data_ptr();
  *bytes = t.nbytes();
}

// q, cache, cache_len, max_cache_len, out, weights, window, softcap, scale, workspace,
// status, stream
PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("gqa_attn_decode_q4", args, n, 12, [](Args& a) {
    const at::Tensor *q = a.f32(0), *cache = a.u8(1), *len = a.i32(2), *out = a.f32(4),
                     *w = a.f32(5, true), *status = a.i32(10, true);
    a.check(q->dim() == 4 && q->size(2) == 1 && out->sizes() == q->sizes() && cache->dim() == 4,
            "inconsistent shapes");
    a.sizes(q);
    const int64_t B = q->size(0), H = q->size(1), Hkv = cache->size(1), D = q->size(3);
    const int cap = a.cache(cache, B, Hkv, D);
    a.check(!w || (w->dim() == 3 && w->size(0) == B && w->size(1) == Hkv && w->size(2) == cap),
            "weights must be [B, Hkv, capacity]");
    a.rows(len, B);
    a.status(status);
    void* ws;
    size_t bytes;
    workspace(a, 9, &ws, &bytes);
    return c_decode(ptr<float>(q), ptr<void>(cache), ptr<int32_t>(len), a.whole(3),
                    ptr<float>(out), ptr<float>(w), B, H, Hkv, D, cap, a.whole(6), a.real(7),
                    a.real(8), ws, bytes, ptr<int32_t>(status), a.stream(11));
  });
}

// q, k, v, out, cache, start, max_start, params, table, q_norm_w, k_norm_w, eps, pos,
// max_pos, weights, window, softcap, scale, workspace, status, stream
PyObject* step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("gqa_attn_decode_step_q4", args, n, 21, [](Args& a) {
    const at::Tensor *q = a.f32(0), *k = a.f32(1), *v = a.f32(2), *out = a.f32(3),
                     *cache = a.u8(4), *start = a.i32(5);
    attn_rope_params rp;
    const bool rope = a.rope(7, &rp);
    const at::Tensor *table = a.f32(8, true), *qn = a.f32(9, true), *kn = a.f32(10, true),
                     *pos = a.i32(12, true), *w = a.f32(14, true), *status = a.i32(19, true);
    a.check(q->dim() == 4 && q->size(2) == 1 && out->sizes() == q->sizes() && cache->dim() == 4,
            "inconsistent shapes");
    a.sizes(q);
    const int64_t B = q->size(0), H = q->size(1), Hkv = cache->size(1), D = q->size(3);
    const int cap = a.cache(cache, B, Hkv, D);
    a.check(k->dim() == 4 && k->size(0) == B && k->size(1) == Hkv && k->size(2) == 1 &&
                k->size(3) == D && v->sizes() == k->sizes(),
            "inconsistent shapes");
    a.check(!w || (w->dim() == 3 && w->size(0) == B && w->size(1) == Hkv && w->size(2) == cap),
            "weights must be [B, Hkv, capacity]");
    a.rows(start, B);
    a.rows(pos, B);
    a.status(status);
    a.table(rope ? &rp : nullptr, table, D);
    a.norm(qn, D);
    a.norm(kn, D);
    void* ws;
    size_t bytes;
    workspace(a, 18, &ws, &bytes);
    return c_step(ptr<float>(q), ptr<float>(k), ptr<float>(v), ptr<float>(out), B, H, Hkv, D,
                  ptr<int32_t>(start), a.whole(6), ptr<int32_t>(pos), a.whole(13),
                  rope ? &rp : nullptr, ptr<float>(table), ptr<float>(qn), ptr<float>(kn),
                  a.real(11), ptr<void>(cache), ptr<float>(w), cap, a.whole(15), a.real(16),
                  a.real(17), ws, bytes, ptr<int32_t>(status), a.stream(20));
  });
}

// cache, weights, cache_len, max_cache_len, budget, recent, cache_out, weights_out, index,
// len_out, status, stream
PyObject* evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("kv_cache_evict_q4", args, n, 12, [](Args& a) {
    const at::Tensor *cache = a.u8(0), *w = a.f32(1), *len = a.i32(2), *co = a.u8(6),
                     *wo = a.f32(7), *index = a.i32(8), *lo = a.i32(9), *status = a.i32(10, true);
    a.check(cache->dim() == 4 && co->dim() == 4, "caches must have 4 dims");
    a.sizes(cache);
    const int64_t B = cache->size(0), Hkv = cache->size(1);
    int D = 32;
    while (D <= 256 && static_cast<int64_t>(c_record(D)) != cache->size(3)) D += 32;
    a.check(D <= 256, "cache must be [B, Hkv, capacity, kv_q4_record_bytes(D)]");
    const int cap = a.cache(cache, B, Hkv, D), cap_out = a.cache(co, B, Hkv, D);
    const long budget = a.whole(4);
    a.check(w->dim() == 3 && w->size(0) == B && w->size(1) == Hkv && w->size(2) == cap &&
                wo->dim() == 3 && wo->size(0) == B && wo->size(1) == Hkv &&
                wo->size(2) == cap_out && index->dim() == 3 && index->size(0) == B &&
                index->size(1) == Hkv && index->size(2) == budget,
            "inconsistent shapes");
    a.rows(len, B);
    a.rows(lo, B);
    a.status(status);
    return c_evict(ptr<void>(cache), ptr<float>(w), ptr<int32_t>(len), a.whole(3), budget,
                   a.whole(5), ptr<void>(co), ptr<float>(wo), ptr<int32_t>(index),
                   ptr<int32_t>(lo), B, Hkv, D, cap, cap_out, ptr<int32_t>(status), a.stream(11));
  });
}

// ---------------------------------------------------------------- 16-bit paged serving

// A call's 16-bit tensors: one type, last dim contiguous, on the call's device.
struct Args16 {
  Args& a;
  at::ScalarType type = at::ScalarType::Undefined;

  const at::Tensor* tensor(int i, int dims, bool optional = false) {
    PyObject* o = a.v[i];
    if (o == Py_None) {
      if (optional) return nullptr;
      fail(PyExc_TypeError, a.fn, "a required tensor is None");
    }
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, a.fn, "expected a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (type == at::ScalarType::Undefined) type = t.scalar_type();
    if ((type != at::kHalf && type != at::kBFloat16) || t.scalar_type() != type)
      fail(PyExc_TypeError, a.fn, "expected torch.float16 or torch.bfloat16, one type for all");
    if (!t.is_cuda()) fail(PyExc_ValueError, a.fn, "expected CUDA tensors");
    if (a.device < 0) a.device = c10::cuda::current_device();
    if (t.get_device() != a.device)
      fail(PyExc_ValueError, a.fn, "tensors must lie on the current CUDA device");
    a.check(t.dim() == dims, "a tensor has the wrong number of dims");
    a.sizes(&t);
    a.check(t.size(dims - 1) <= 1 || t.stride(dims - 1) == 1, "the last dim must be contiguous");
    return &t;
  }
  int code() const { return type == at::kHalf ? ATTN_TYPE_FP16 : ATTN_TYPE_BF16; }
};

attn_rows rows16(const at::Tensor* t) {
  if (!t) return attn_rows{nullptr, 0, 0};
  return attn_rows{t->data_ptr(), t->stride(0), t->stride(1)};
}

// Pools [pages, Hkv, page, D]: pages apart as they like, contiguous within, k like v.
attn_paged_kv pools16(Args& a, const at::Tensor* k, const at::Tensor* v, int64_t D) {
  a.check(v->sizes() == k->sizes() && k->size(3) == D, "inconsistent shapes");
  for (const at::Tensor* t : {k, v}) {
    const int64_t page = k->size(2);
    a.check((page <= 1 || t->stride(2) == D) && (k->size(1) <= 1 || t->stride(1) == page * D),
            "a page of the cache must be contiguous");
  }
  a.check(k->size(0) <= 1 || k->stride(0) == v->stride(0), "k_cache and v_cache: one page stride");
  return attn_paged_kv{k->data_ptr(), v->data_ptr(), k->stride(0),
                       static_cast<int32_t>(k->size(0)), static_cast<int32_t>(k->size(2))};
}

const at::Tensor* table16(Args& a, int i, int64_t B) {
  const at::Tensor* t = a.i32(i);
  a.check(t->dim() == 2 && t->size(0) == B, "block_table must be [B, pages of a row]");
  a.sizes(t);
  return t;
}

// k, v, k_cache, v_cache, block_table, start, max_pos, params, table, k_norm_w, eps,
// cu_seqlens, q, q_out, q_norm_w, k_out, status, stream
PyObject* append_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("kv_cache_append_paged", args, n, 18, [](Args& a) {
    Args16 x{a};
    const at::Tensor *k = x.tensor(0, 3), *v = x.tensor(1, 3), *kc = x.tensor(2, 4),
                     *vc = x.tensor(3, 4), *start = a.i32(5);
    attn_rope_params rp;
    const bool rope = a.rope(7, &rp);
    const at::Tensor *table = a.f32(8, true), *kn = a.f32(9, true), *cu = a.i32(11, true),
                     *q = x.tensor(12, 3, true), *qo = x.tensor(13, 3, true),
                     *qn = a.f32(14, true), *ko = x.tensor(15, 3, true), *status = a.i32(16, true);
    const int64_t T = k->size(0), Hkv = k->size(1), D = k->size(2), B = start->numel();
    const int64_t H = q ? q->size(1) : Hkv;
    a.check(v->sizes() == k->sizes() && (!ko || ko->sizes() == k->sizes()) && kc->size(1) == Hkv &&
                (!q || (q->size(0) == T && q->size(2) == D)) && (!q == !qo) &&
                (!q || qo->sizes() == q->sizes()),
            "inconsistent shapes");
    a.check(!cu || cu->numel() == B + 1, "cu_seqlens holds one value more than start");
    const at::Tensor* bt = table16(a, 4, B);
    a.status(status);
    a.table(rope ? &rp : nullptr, table, D);
    a.norm(qn, D);
    a.norm(kn, D);
    const attn_rows rq = rows16(q), rqo = rows16(qo), rk = rows16(k), rko = rows16(ko),
                    rv = rows16(v);
    const attn_paged_kv cache = pools16(a, kc, vc, D);
    return c_append_paged(x.code(), &rq, &rqo, &rk, &rko, &rv, T, B, H, Hkv, D, ptr<int32_t>(cu),
                          ptr<int32_t>(start), a.whole(6), rope ? &rp : nullptr, ptr<float>(table),
                          ptr<float>(qn), ptr<float>(kn), a.real(10), &cache, ptr<int32_t>(bt),
                          bt->size(1), ptr<int32_t>(status), a.stream(17));
  });
}

// q, k_cache, v_cache, block_table, cache_len, max_cache_len, out, window, softcap, scale,
// workspace, status, stream
PyObject* decode_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("gqa_attn_decode_paged", args, n, 13, [](Args& a) {
    Args16 x{a};
    const at::Tensor *q = x.tensor(0, 3), *kc = x.tensor(1, 4), *vc = x.tensor(2, 4),
                     *len = a.i32(4), *out = x.tensor(6, 3), *status = a.i32(11, true);
    const int64_t B = q->size(0), H = q->size(1), D = q->size(2), Hkv = kc->size(1);
    a.check(out->sizes() == q->sizes(), "inconsistent shapes");
    const at::Tensor* bt = table16(a, 3, B);
    a.rows(len, B);
    a.status(status);
    const attn_rows rq = rows16(q), ro = rows16(out);
    const attn_paged_kv cache = pools16(a, kc, vc, D);
    void* ws;
    size_t bytes;
    workspace(a, 10, &ws, &bytes);
    return c_decode_paged(x.code(), &rq, &cache, ptr<int32_t>(bt), bt->size(1), ptr<int32_t>(len),
                          a.whole(5), &ro, B, H, Hkv, D, a.whole(7), a.real(8), a.real(9), ws,
                          bytes, ptr<int32_t>(status), a.stream(12));
  });
}

// q, k_cache, v_cache, prefix_table, prefix_len, block_table, cache_len, max_cache_len, out,
// softcap, scale, workspace, status, stream
PyObject* decode_shared(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("gqa_attn_decode_shared", args, n, 14, [](Args& a) {
    Args16 x{a};
    const at::Tensor *q = x.tensor(0, 3), *kc = x.tensor(1, 4), *vc = x.tensor(2, 4),
                     *pt = a.i32(3), *len = a.i32(6), *out = x.tensor(8, 3),
                     *status = a.i32(12, true);
    const int64_t B = q->size(0), H = q->size(1), D = q->size(2), Hkv = kc->size(1);
    a.check(out->sizes() == q->sizes() && pt->dim() == 1, "inconsistent shapes");
    a.sizes(pt);
    const at::Tensor* bt = table16(a, 5, B);
    a.rows(len, B);
    a.status(status);
    const attn_rows rq = rows16(q), ro = rows16(out);
    const attn_paged_kv cache = pools16(a, kc, vc, D);
    void* ws;
    size_t bytes;
    workspace(a, 11, &ws, &bytes);
    return c_decode_shared(x.code(), &rq, &cache, ptr<int32_t>(pt), pt->size(0), a.whole(4),
                           ptr<int32_t>(bt), bt->size(1), ptr<int32_t>(len), a.whole(7), &ro, B, H,
                           Hkv, D, a.real(9), a.real(10), ws, bytes, ptr<int32_t>(status),
                           a.stream(13));
  });
}

// q, k, v, cu_seqlens, max_len, out, window, softcap, scale, status, stream
PyObject* prefill_packed(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run("gqa_attn_prefill_packed", args, n, 11, [](Args& a) {
    Args16 x{a};
    const at::Tensor *q = x.tensor(0, 3), *k = x.tensor(1, 3), *v = x.tensor(2, 3), *cu = a.i32(3),
                     *out = x.tensor(5, 3), *status = a.i32(9, true);
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2), Hkv = k->size(1);
    a.check(k->size(0) == T && k->size(2) == D && v->sizes() == k->sizes() &&
                out->sizes() == q->sizes(),
            "inconsistent shapes");
    a.check(cu->numel() >= 1 && cu->numel() <= INT32_MAX, "cu_seqlens must hold B + 1 values");
    a.status(status);
    const attn_rows rq = rows16(q), rk = rows16(k), rv = rows16(v), ro = rows16(out);
    return c_prefill_packed(x.code(), &rq, &rk, &rv, ptr<int32_t>(cu), a.whole(4), &ro, T,
                            cu->numel() - 1, H, Hkv, D, a.whole(6), a.real(7), a.real(8),
                            ptr<int32_t>(status), a.stream(10));
  });
}

// Addresses of the C entry points: append, read, decode, step, evict, record bytes; paged
// append, paged decode, shared decode, packed prefill.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int kCalls = 10;
  void* p[kCalls];
  if (n != kCalls) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of addresses");
    return nullptr;
  }
  for (int i = 0; i < kCalls; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  c_append = reinterpret_cast<decltype(c_append)>(p[0]);
  c_read = reinterpret_cast<decltype(c_read)>(p[1]);
  c_decode = reinterpret_cast<decltype(c_decode)>(p[2]);
  c_step = reinterpret_cast<decltype(c_step)>(p[3]);
  c_evict = reinterpret_cast<decltype(c_evict)>(p[4]);
  c_record = reinterpret_cast<decltype(c_record)>(p[5]);
  c_append_paged = reinterpret_cast<decltype(c_append_paged)>(p[6]);
  c_decode_paged = reinterpret_cast<decltype(c_decode_paged)>(p[7]);
  c_decode_shared = reinterpret_cast<decltype(c_decode_shared)>(p[8]);
  c_prefill_packed = reinterpret_cast<decltype(c_prefill_packed)>(p[9]);
  Py_RETURN_NONE;
}

#define NATIVE_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NATIVE_METHOD(append), NATIVE_METHOD(read),  NATIVE_METHOD(decode), NATIVE_METHOD(step),
                         NATIVE_METHOD(evict),  NATIVE_METHOD(bind),
                         NATIVE_METHOD(append_paged), NATIVE_METHOD(decode_paged),
                         NATIVE_METHOD(decode_shared), NATIVE_METHOD(prefill_packed),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gqa_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gqa_binding(void) { return PyModule_Create(&module); }

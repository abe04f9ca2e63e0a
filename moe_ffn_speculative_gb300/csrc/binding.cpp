// The attention side's calls from Python without the cost of looking each
// tensor over there: a small call's GPU time is a few microseconds, and about
// a dozen tensors' types, shapes and strides read one by one in Python take
// longer.  Each function checks everything about its arguments and makes the
// C call; where something is wrong with them it returns None, and ops.py's own
// checks say what.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "moe.h"

namespace {

using at::Tensor;

// An argument that is a tensor or None (null); `ok` falls where it is neither.
const Tensor* tensor(PyObject* o, bool& ok) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    ok = false;
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}
long long integer(PyObject* o, bool& ok) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    ok = false;
  }
  return v;
}
double number(PyObject* o, bool& ok) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    ok = false;
  }
  return v;
}
cudaStream_t stream_of(PyObject* o, bool& ok) { return reinterpret_cast<cudaStream_t>(integer(o, ok)); }

// The current device, on which a call launches; asked for once a call.
thread_local at::DeviceIndex here = -1;
void look_up_device() { here = c10::impl::VirtualGuardImpl(at::kCUDA).getDevice().index(); }
bool gpu(const Tensor& t, at::ScalarType type) {
  return t.is_cuda() && t.device().index() == here && t.scalar_type() == type;
}
// A contiguous tensor of n elements, or none.
bool flat(const Tensor* t, at::ScalarType type, int64_t n) {
  return t == nullptr || (gpu(*t, type) && t->is_contiguous() && t->numel() == n);
}
void* data(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
// [T, h, D] whose rows may lie apart; their distance.
bool heads(const Tensor& t, at::ScalarType type, int64_t T, int64_t h, int64_t D, long long& stride) {
  if (!gpu(t, type) || t.dim() != 3 || t.size(0) != T || t.size(1) != h || t.size(2) != D) return false;
  if (t.numel() != 0 && ((D > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != D))) return false;
  stride = T > 1 ? t.stride(0) : h * D;
  return true;
}
bool rows(const Tensor& t, at::ScalarType type, int64_t m, int64_t n, long long& stride) {
  if (!gpu(t, type) || t.dim() != 2 || t.size(0) != m || t.size(1) != n || (n > 1 && t.stride(1) != 1)) return false;
  stride = m > 1 ? t.stride(0) : n;
  return true;
}
bool type16(const Tensor& t, int& code) {
  code = t.scalar_type() == at::kBFloat16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F16;
  return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf;
}
bool fits(int64_t v) { return v >= 0 && v <= INT32_MAX; }

// (q, k, v, positions, rope, q_weight, k_weight, eps, interleaved, q_out,
//  k_cache, v_cache, slots, workspace address, workspace bytes, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 16;
  if (!ok) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0], ok), *k = tensor(a[1], ok), *v = tensor(a[2], ok), *pos = tensor(a[3], ok),
               *rope = tensor(a[4], ok), *qw = tensor(a[5], ok), *kw = tensor(a[6], ok), *qo = tensor(a[9], ok),
               *kc = tensor(a[10], ok), *vc = tensor(a[11], ok), *slots = tensor(a[12], ok);
  const double eps = number(a[7], ok);
  const bool inter = a[8] == Py_True;
  void* ws = reinterpret_cast<void*>(integer(a[13], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[14], ok));
  const cudaStream_t stream = stream_of(a[15], ok);
  const Tensor* lead = q ? q : k;
  int code = 0;
  if (!ok || !lead || (a[8] != Py_True && a[8] != Py_False) || !type16(*lead, code) || lead->dim() != 3) Py_RETURN_NONE;
  look_up_device();
  const at::ScalarType type = lead->scalar_type();
  const int64_t T = lead->size(0), D = lead->size(2), Hq = q ? q->size(1) : 0;
  long long qs = 0, ks = 0, vs = 0, qos = 0, n_slots = 0;
  int64_t Hkv = 0;
  if (!fits(T) || (q != nullptr) != (qo != nullptr) || (k != nullptr) != (kc != nullptr) ||
      (v != nullptr) != (vc != nullptr) || (v && !k))
    Py_RETURN_NONE;
  if (q && (!heads(*q, type, T, Hq, D, qs) || !heads(*qo, type, T, Hq, D, qos))) Py_RETURN_NONE;
  if (k) {
    if (k->dim() != 3) Py_RETURN_NONE;
    Hkv = k->size(1);
    if (!heads(*k, type, T, Hkv, D, ks) || kc->dim() < 2 || kc->size(-1) != D || kc->size(-2) != Hkv || Hkv * D == 0 ||
        !flat(kc, type, kc->numel()))
      Py_RETURN_NONE;
    n_slots = kc->numel() / (Hkv * D);
    if (v && (!heads(*v, type, T, Hkv, D, vs) || vc->dim() < 2 || vc->size(-1) != D || vc->size(-2) != Hkv ||
              !flat(vc, type, kc->numel())))
      Py_RETURN_NONE;
  }
  if (rope && (rope->dim() != 2 || !fits(rope->size(0)) || !flat(rope, at::kFloat, rope->numel()))) Py_RETURN_NONE;
  if (!flat(pos, at::kInt, T) || !flat(slots, at::kInt, T) || !flat(qw, type, D) || !flat(kw, type, D)) Py_RETURN_NONE;
  const moe_status st = moe_qk_norm_rope(
      data(q), qs, data(k), ks, data(v), vs, static_cast<int>(T), static_cast<int>(Hq), static_cast<int>(Hkv),
      static_cast<int>(D), code, data(qw), data(kw), static_cast<float>(eps), static_cast<const float*>(data(rope)),
      rope ? static_cast<int>(rope->size(1)) : 0, rope ? static_cast<int>(rope->size(0)) : 0, inter ? 1 : 0,
      static_cast<const int32_t*>(data(pos)), data(qo), qos, data(kc), data(vc),
      static_cast<const int32_t*>(data(slots)), n_slots, ws, ws_bytes, stream);
  return PyLong_FromLong(st);
}

// (q, k_cache, v_cache, q_start, prefix_pages, prefix_len, page_table, own_len,
//  causal, scale, out, lse, workspace address, workspace bytes, stream)
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 15;
  if (!ok) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0], ok), *kc = tensor(a[1], ok), *vc = tensor(a[2], ok), *start = tensor(a[3], ok),
               *pp = tensor(a[4], ok), *pl = tensor(a[5], ok), *table = tensor(a[6], ok), *own = tensor(a[7], ok),
               *out = tensor(a[10], ok), *lse = tensor(a[11], ok);
  const double scale = number(a[9], ok);
  void* ws = reinterpret_cast<void*>(integer(a[12], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[13], ok));
  const cudaStream_t stream = stream_of(a[14], ok);
  int code = 0;
  if (!ok || !q || !kc || !vc || !start || !out || (a[8] != Py_True && a[8] != Py_False) || !type16(*q, code) ||
      q->dim() != 3 || kc->dim() != 4)
    Py_RETURN_NONE;
  look_up_device();
  const at::ScalarType type = q->scalar_type();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), B = start->numel() - 1;
  const int64_t pages = kc->size(0), page = kc->size(1), Hkv = kc->size(2);
  const int64_t cap = pp ? pp->numel() : 0, width = table && table->dim() == 2 ? table->size(1) : 0;
  long long qs = 0;
  if (!heads(*q, type, T, Hq, D, qs) || kc->size(3) != D || !flat(kc, type, kc->numel()) ||
      !flat(vc, type, kc->numel()) || vc->sizes() != kc->sizes() || B < 0 || (pp != nullptr) != (pl != nullptr) ||
      (table != nullptr) != (own != nullptr) || (table && (table->dim() != 2 || table->size(0) != B)))
    Py_RETURN_NONE;
  if (!fits(T) || !fits(B) || !fits(pages) || !fits(page) || !fits(cap) || !fits(width) ||
      !flat(start, at::kInt, B + 1) || !flat(pp, at::kInt, cap) || !flat(pl, at::kInt, 1) ||
      !flat(table, at::kInt, B * width) || !flat(own, at::kInt, B) || out->dim() != 3 || out->size(0) != T ||
      out->size(1) != Hq || !flat(out, type, T * Hq * D) || !flat(lse, at::kFloat, T * Hq))
    Py_RETURN_NONE;
  const moe_status st = moe_prefix_attention(
      data(q), qs, static_cast<int>(T), static_cast<int>(B), static_cast<const int32_t*>(data(start)),
      static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D), code, data(kc), data(vc),
      static_cast<int>(pages), static_cast<int>(page), static_cast<const int32_t*>(data(pp)), static_cast<int>(cap),
      static_cast<const int32_t*>(data(pl)), static_cast<const int32_t*>(data(table)), static_cast<int>(width),
      static_cast<const int32_t*>(data(own)), a[8] == Py_True ? 1 : 0, static_cast<float>(scale), data(out),
      static_cast<float*>(data(lse)), ws, ws_bytes, stream);
  return PyLong_FromLong(st);
}

// (x, w, bias, activation code, residual, y, workspace address, workspace
//  bytes, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 9;
  if (!ok) Py_RETURN_NONE;
  const Tensor *x = tensor(a[0], ok), *w = tensor(a[1], ok), *bias = tensor(a[2], ok), *res = tensor(a[4], ok),
               *y = tensor(a[5], ok);
  const long long act = integer(a[3], ok);
  void* ws = reinterpret_cast<void*>(integer(a[6], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[7], ok));
  const cudaStream_t stream = stream_of(a[8], ok);
  int code = 0;
  if (!ok || !x || !w || !y || !type16(*x, code) || x->dim() != 2 || w->dim() != 2) Py_RETURN_NONE;
  look_up_device();
  const at::ScalarType type = x->scalar_type();
  const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
  long long xs = 0, ys = 0, rs = 0;
  if (!fits(M) || !fits(K) || !fits(N) || !fits(act) || !rows(*x, type, M, K, xs) || !flat(w, type, N * K) ||
      !rows(*y, type, M, N, ys) || !flat(bias, type, N) || (res && !rows(*res, type, M, N, rs)))
    Py_RETURN_NONE;
  const moe_status st = moe_linear(data(x), xs, static_cast<int>(M), static_cast<int>(K), data(w), static_cast<int>(N),
                                   code, data(bias), static_cast<int>(act), data(res), rs, data(y), ys, ws, ws_bytes,
                                   stream);
  return PyLong_FromLong(st);
}

// (x, prepared weights, N, K, group, zeros, bias, activation code, residual, y,
//  workspace address, workspace bytes, stream)
PyObject* linear_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 13;
  if (!ok) Py_RETURN_NONE;
  const Tensor *x = tensor(a[0], ok), *w = tensor(a[1], ok), *bias = tensor(a[6], ok), *res = tensor(a[8], ok),
               *y = tensor(a[9], ok);
  const long long N = integer(a[2], ok), K = integer(a[3], ok), group = integer(a[4], ok), act = integer(a[7], ok);
  void* ws = reinterpret_cast<void*>(integer(a[10], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[11], ok));
  const cudaStream_t stream = stream_of(a[12], ok);
  int code = 0;
  if (!ok || !x || !w || !y || (a[5] != Py_True && a[5] != Py_False) || !type16(*x, code) || x->dim() != 2) Py_RETURN_NONE;
  look_up_device();
  const at::ScalarType type = x->scalar_type();
  const int64_t M = x->size(0);
  long long xs = 0, ys = 0, rs = 0;
  if (!fits(M) || !fits(K) || !fits(N) || !fits(act) || !fits(group) || !rows(*x, type, M, K, xs) ||
      !flat(w, at::kByte, w->numel()) || !rows(*y, type, M, N, ys) || !flat(bias, type, N) ||
      (res && !rows(*res, type, M, N, rs)))
    Py_RETURN_NONE;
  const moe_status st = moe_linear_q4(data(x), xs, static_cast<int>(M), static_cast<int>(K), data(w),
                                      static_cast<size_t>(w->numel()), static_cast<int>(N), static_cast<int>(group),
                                      a[5] == Py_True ? 1 : 0, code, data(bias), static_cast<int>(act), data(res), rs,
                                      data(y), ys, ws, ws_bytes, stream);
  return PyLong_FromLong(st);
}

// A kv4 cache uint8 [pages, Hkv, page_size * (D + D / 16)]; its page size.
bool kv4(const Tensor& t, int64_t D, int64_t& page) {
  if (!gpu(t, at::kByte) || t.dim() != 3 || !t.is_contiguous() || D < 16 || D % 16 != 0) return false;
  page = t.size(2) / (D + D / 16);
  return fits(t.size(0)) && fits(t.size(1)) && fits(page) && page * (D + D / 16) == t.size(2);
}

// (k, v, slots, cache, workspace address, workspace bytes, stream)
PyObject* kv4_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 7;
  if (!ok) Py_RETURN_NONE;
  const Tensor *k = tensor(a[0], ok), *v = tensor(a[1], ok), *slots = tensor(a[2], ok), *cache = tensor(a[3], ok);
  void* ws = reinterpret_cast<void*>(integer(a[4], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[5], ok));
  const cudaStream_t stream = stream_of(a[6], ok);
  int code = 0;
  if (!ok || !k || !v || !cache || !type16(*k, code) || k->dim() != 3) Py_RETURN_NONE;
  look_up_device();
  const at::ScalarType type = k->scalar_type();
  const int64_t T = k->size(0), Hkv = k->size(1), D = k->size(2);
  int64_t page = 0;
  long long ks = 0, vs = 0;
  if (!fits(T) || !heads(*k, type, T, Hkv, D, ks) || !heads(*v, type, T, Hkv, D, vs) || !kv4(*cache, D, page) ||
      cache->size(1) != Hkv || !flat(slots, at::kInt, T))
    Py_RETURN_NONE;
  return PyLong_FromLong(moe_kv4_write(data(k), ks, data(v), vs, static_cast<int>(T), static_cast<int>(Hkv),
                                       static_cast<int>(D), code, static_cast<const int32_t*>(data(slots)),
                                       data(cache), static_cast<int>(cache->size(0)), static_cast<int>(page), ws,
                                       ws_bytes, stream));
}

// (cache, head size, pages, k, v, workspace address, workspace bytes, stream)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 8;
  if (!ok) Py_RETURN_NONE;
  const Tensor *cache = tensor(a[0], ok), *pages = tensor(a[2], ok), *k = tensor(a[3], ok), *v = tensor(a[4], ok);
  const long long D = integer(a[1], ok);
  void* ws = reinterpret_cast<void*>(integer(a[5], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[6], ok));
  const cudaStream_t stream = stream_of(a[7], ok);
  int code = 0;
  if (!ok || !cache || !k || !v || !type16(*k, code)) Py_RETURN_NONE;
  look_up_device();
  int64_t page = 0;
  if (!kv4(*cache, D, page)) Py_RETURN_NONE;
  const int64_t Hkv = cache->size(1), count = pages ? pages->numel() : cache->size(0);
  const auto shaped = [&](const Tensor& t) {
    return t.dim() == 4 && t.size(0) == count && t.size(1) == page && t.size(2) == Hkv && t.size(3) == D &&
           flat(&t, k->scalar_type(), t.numel());
  };
  if (!fits(count) || !flat(pages, at::kInt, count) || !shaped(*k) || !shaped(*v)) Py_RETURN_NONE;
  return PyLong_FromLong(moe_kv4_read(data(cache), static_cast<int>(cache->size(0)), static_cast<int>(page),
                                      static_cast<int>(Hkv), static_cast<int>(D),
                                      static_cast<const int32_t*>(data(pages)), static_cast<int>(count), data(k),
                                      data(v), code, ws, ws_bytes, stream));
}

// (q, cache, q_start, prefix_pages, prefix_len, page_table, own_len, causal,
//  scale, out, lse, workspace address, workspace bytes, stream)
PyObject* prefix_attention_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 14;
  if (!ok) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0], ok), *cache = tensor(a[1], ok), *start = tensor(a[2], ok), *pp = tensor(a[3], ok),
               *pl = tensor(a[4], ok), *table = tensor(a[5], ok), *own = tensor(a[6], ok), *out = tensor(a[9], ok),
               *lse = tensor(a[10], ok);
  const double scale = number(a[8], ok);
  void* ws = reinterpret_cast<void*>(integer(a[11], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[12], ok));
  const cudaStream_t stream = stream_of(a[13], ok);
  int code = 0;
  if (!ok || !q || !cache || !start || !out || (a[7] != Py_True && a[7] != Py_False) || !type16(*q, code) ||
      q->dim() != 3)
    Py_RETURN_NONE;
  look_up_device();
  const at::ScalarType type = q->scalar_type();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), B = start->numel() - 1;
  const int64_t cap = pp ? pp->numel() : 0, width = table && table->dim() == 2 ? table->size(1) : 0;
  int64_t page = 0;
  long long qs = 0;
  if (!heads(*q, type, T, Hq, D, qs) || !kv4(*cache, D, page) || B < 0 || (pp != nullptr) != (pl != nullptr) ||
      (table != nullptr) != (own != nullptr) || (table && (table->dim() != 2 || table->size(0) != B)))
    Py_RETURN_NONE;
  if (!fits(T) || !fits(B) || !fits(cap) || !fits(width) || !flat(start, at::kInt, B + 1) || !flat(pp, at::kInt, cap) ||
      !flat(pl, at::kInt, 1) || !flat(table, at::kInt, B * width) || !flat(own, at::kInt, B) || out->dim() != 3 ||
      out->size(0) != T || out->size(1) != Hq || !flat(out, type, T * Hq * D) || !flat(lse, at::kFloat, T * Hq))
    Py_RETURN_NONE;
  const moe_status st = moe_prefix_attention_kv4(
      data(q), qs, static_cast<int>(T), static_cast<int>(B), static_cast<const int32_t*>(data(start)),
      static_cast<int>(Hq), static_cast<int>(cache->size(1)), static_cast<int>(D), code, data(cache),
      static_cast<int>(cache->size(0)), static_cast<int>(page), static_cast<const int32_t*>(data(pp)),
      static_cast<int>(cap), static_cast<const int32_t*>(data(pl)), static_cast<const int32_t*>(data(table)),
      static_cast<int>(width), static_cast<const int32_t*>(data(own)), a[7] == Py_True ? 1 : 0,
      static_cast<float>(scale), data(out), static_cast<float*>(data(lse)), ws, ws_bytes, stream);
  return PyLong_FromLong(st);
}

// The pools of a page call, of n_pages pages each: [n_pages, page_size, ...] rows
// of any type, or a kv4 cache (uint8 of three dimensions).
bool pools_of(PyObject* o, int64_t n_pages, int64_t page, moe_page_pool* out, int& n) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) > MOE_MAX_POOLS || page < 1) return false;
  n = static_cast<int>(PyTuple_GET_SIZE(o));
  for (int i = 0; i < n; ++i) {
    bool ok = true;
    const Tensor* t = tensor(PyTuple_GET_ITEM(o, i), ok);
    if (!ok || !t || !t->is_cuda() || t->device().index() != here || t->dim() < 3 || !t->is_contiguous() ||
        t->size(0) != n_pages)
      return false;
    moe_page_pool& p = out[i];
    p = moe_page_pool{t->data_ptr(), MOE_POOL_ROWS, 0, 0, 0};
    if (t->scalar_type() == at::kByte && t->dim() == 3) {
      if (t->size(2) % page != 0 || t->size(2) / page * 16 % 17 != 0 || !fits(t->size(1))) return false;
      p.format = MOE_POOL_KV4;
      p.heads = static_cast<int32_t>(t->size(1));
      p.head_dim = static_cast<int32_t>(t->size(2) / page * 16 / 17);
    } else {
      if (t->size(1) != page) return false;
      p.row_bytes = t->element_size();
      for (int64_t d = 2; d < t->dim(); ++d) p.row_bytes *= t->size(d);
    }
  }
  return true;
}

// (refs, page_table, own_len, new_len, page_size, pools, workspace address,
//  workspace bytes, stream)
PyObject* pages_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 9;
  if (!ok) Py_RETURN_NONE;
  const Tensor *refs = tensor(a[0], ok), *table = tensor(a[1], ok), *own = tensor(a[2], ok), *now = tensor(a[3], ok);
  const long long page = integer(a[4], ok);
  void* ws = reinterpret_cast<void*>(integer(a[6], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[7], ok));
  const cudaStream_t stream = stream_of(a[8], ok);
  if (!ok || !refs || !table || !own || !now || table->dim() != 2 || !fits(page)) Py_RETURN_NONE;
  look_up_device();
  const int64_t B = table->size(0), width = table->size(1), pages = refs->numel();
  moe_page_pool pools[MOE_MAX_POOLS];
  int n_pools = 0;
  if (!fits(B) || !fits(width) || !fits(pages) || !flat(refs, at::kInt, pages) || !flat(table, at::kInt, B * width) ||
      !flat(own, at::kInt, B) || !flat(now, at::kInt, B) || !pools_of(a[5], pages, page, pools, n_pools))
    Py_RETURN_NONE;
  return PyLong_FromLong(moe_pages_resize(static_cast<int32_t*>(data(refs)), static_cast<int>(pages),
                                          static_cast<int32_t*>(data(table)), static_cast<int>(B),
                                          static_cast<int>(width), static_cast<int>(page),
                                          static_cast<int32_t*>(data(own)), static_cast<const int32_t*>(data(now)),
                                          pools, n_pools, ws, ws_bytes, stream));
}

// (refs, page_table, own_len, src, dst, page_size, pools, workspace address,
//  workspace bytes, stream)
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 10;
  if (!ok) Py_RETURN_NONE;
  const Tensor *refs = tensor(a[0], ok), *table = tensor(a[1], ok), *own = tensor(a[2], ok), *src = tensor(a[3], ok),
               *dst = tensor(a[4], ok);
  const long long page = integer(a[5], ok);
  void* ws = reinterpret_cast<void*>(integer(a[7], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[8], ok));
  const cudaStream_t stream = stream_of(a[9], ok);
  if (!ok || !refs || !table || !own || !src || !dst || table->dim() != 2 || !fits(page)) Py_RETURN_NONE;
  look_up_device();
  const int64_t B = table->size(0), width = table->size(1), pages = refs->numel(), pairs = src->numel();
  moe_page_pool pools[MOE_MAX_POOLS];
  int n_pools = 0;
  if (!fits(B) || !fits(width) || !fits(pages) || !fits(pairs) || !flat(refs, at::kInt, pages) ||
      !flat(table, at::kInt, B * width) || !flat(own, at::kInt, B) || !flat(src, at::kInt, pairs) ||
      !flat(dst, at::kInt, pairs) || !pools_of(a[6], pages, page, pools, n_pools))
    Py_RETURN_NONE;
  return PyLong_FromLong(moe_pages_fork(
      static_cast<int32_t*>(data(refs)), static_cast<int>(pages), static_cast<int32_t*>(data(table)),
      static_cast<int>(B), static_cast<int>(width), static_cast<int>(page), static_cast<int32_t*>(data(own)),
      static_cast<const int32_t*>(data(src)), static_cast<const int32_t*>(data(dst)), static_cast<int>(pairs), pools,
      n_pools, ws, ws_bytes, stream));
}

// (page_table, base, keep, page_size, pages of the pools, pools, new_len,
//  workspace address, workspace bytes, stream)
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  bool ok = n == 10;
  if (!ok) Py_RETURN_NONE;
  const Tensor *table = tensor(a[0], ok), *base = tensor(a[1], ok), *keep = tensor(a[2], ok), *now = tensor(a[6], ok);
  const long long page = integer(a[3], ok), pages = integer(a[4], ok);
  void* ws = reinterpret_cast<void*>(integer(a[7], ok));
  const size_t ws_bytes = static_cast<size_t>(integer(a[8], ok));
  const cudaStream_t stream = stream_of(a[9], ok);
  if (!ok || !table || !base || !keep || table->dim() != 2 || keep->dim() != 2 || !fits(page) || !fits(pages))
    Py_RETURN_NONE;
  look_up_device();
  const int64_t B = table->size(0), width = table->size(1), block = keep->size(1);
  moe_page_pool pools[MOE_MAX_POOLS];
  int n_pools = 0;
  if (!fits(B) || !fits(width) || !fits(block) || keep->size(0) != B || !flat(table, at::kInt, B * width) ||
      !flat(base, at::kInt, B) || !flat(keep, at::kInt, B * block) || !flat(now, at::kInt, B) ||
      !pools_of(a[5], pages, page, pools, n_pools))
    Py_RETURN_NONE;
  return PyLong_FromLong(moe_pages_compact(static_cast<const int32_t*>(data(table)), static_cast<int>(pages),
                                           static_cast<int>(B), static_cast<int>(width), static_cast<int>(page),
                                           static_cast<const int32_t*>(data(base)),
                                           static_cast<const int32_t*>(data(keep)), static_cast<int>(block), pools,
                                           n_pools, static_cast<int32_t*>(data(now)), ws, ws_bytes, stream));
}

// No C++ exception leaves for the interpreter (a sparse tensor's layout throws
// where its strides are asked for).
typedef PyObject* Fast(PyObject*, PyObject* const*, Py_ssize_t);
template <Fast* F>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    Py_RETURN_NONE;
  }
}
#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<f>))
PyMethodDef methods[] = {{"qk_norm_rope", FAST(qk_norm_rope), METH_FASTCALL, nullptr},
                         {"prefix_attention", FAST(prefix_attention), METH_FASTCALL, nullptr},
                         {"linear", FAST(linear), METH_FASTCALL, nullptr},
                         {"linear_q4", FAST(linear_q4), METH_FASTCALL, nullptr},
                         {"kv4_write", FAST(kv4_write), METH_FASTCALL, nullptr},
                         {"kv4_read", FAST(kv4_read), METH_FASTCALL, nullptr},
                         {"prefix_attention_kv4", FAST(prefix_attention_kv4), METH_FASTCALL, nullptr},
                         {"pages_resize", FAST(pages_resize), METH_FASTCALL, nullptr},
                         {"pages_fork", FAST(pages_fork), METH_FASTCALL, nullptr},
                         {"pages_compact", FAST(pages_compact), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // what it was compiled against, for the loader to compare
  if (m && (PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0 ||
            PyModule_AddIntConstant(m, "python_version", PY_VERSION_HEX >> 16) != 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

// Python module _marshal: the serving calls' arguments from torch tensors to
// the C ABI.
//
// These calls are made once per layer and token; with ctypes the marshalling
// of one took 11 us on the host, longer than most of the kernels behind it.
// The module reads what it needs from each tensor through its Python
// interface (dtype, shape, stride, data_ptr, get_device), checks what the C
// side cannot see, and calls the C function whose address the package gives it
// (the library itself is loaded by ctypes, once). It keeps nothing between
// calls and links to nothing but Python.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../../include/rtp.h"

namespace {

constexpr int kHeadDim = 128;
constexpr int kMaxDims = 4;

// Interned names and what setup() was given.
PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device;
PyObject *g_error, *g_check, *g_bf16, *g_f16, *g_f32, *g_i32, *g_raw_stream, *g_current_device;

decltype(&rtp_attn_packed) f_packed;
decltype(&rtp_attn_key_weights) f_weights;
decltype(&rtp_paged_append) f_append;
decltype(&rtp_paged_attn_decode) f_decode;
decltype(&rtp_cache_evict) f_evict;
decltype(&rtp_workspace_size_paged_attn_decode) f_decode_ws;

bool refuse(const char* fmt, ...) {
  char text[256];
  va_list args;
  va_start(args, fmt);
  vsnprintf(text, sizeof text, fmt, args);
  va_end(args);
  PyErr_SetString(g_error, text);
  return false;
}

struct Tensor {
  void* p = nullptr;
  int dev = -1, dims = 0;
  int64_t shape[kMaxDims], stride[kMaxDims];
  PyObject* dtype = nullptr;   // borrowed: torch's dtypes live as long as torch
  bool contiguous() const {
    for (int d = 0; d < dims; ++d)
      if (shape[d] == 0) return true;   // no element: strides say nothing
    int64_t want = 1;
    for (int d = dims - 1; d >= 0; --d) {
      if (shape[d] != 1 && stride[d] != want) return false;
      want *= shape[d];
    }
    return true;
  }
  bool is(int64_t a, int64_t b = -1, int64_t c = -1) const {
    const int64_t want[3] = {a, b, c};
    const int n = b < 0 ? 1 : (c < 0 ? 2 : 3);
    if (dims != n) return false;
    for (int d = 0; d < n; ++d)
      if (shape[d] != want[d]) return false;
    return true;
  }
};

// The items of a tuple of ints (a torch.Size is one).
bool read_ints(PyObject* t, int64_t* to, int* n) {
  if (!t) return false;
  bool ok = PyTuple_Check(t);
  if (!ok) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
  } else {
    const Py_ssize_t len = PyTuple_GET_SIZE(t);
    *n = (int)len;
    for (Py_ssize_t i = 0; ok && i < len && i < kMaxDims; ++i) {
      to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
      ok = !(to[i] == -1 && PyErr_Occurred());
    }
  }
  Py_DECREF(t);
  return ok;
}

bool read_int(PyObject* v, int64_t* to) {
  if (!v) return false;
  *to = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return !(*to == -1 && PyErr_Occurred());
}

// Reads a tensor; `dev` (-1: not known yet) has to be its device.
bool read(const char* what, PyObject* o, Tensor* t, int* dev) {
  int64_t x;
  if (!read_int(PyObject_CallMethodNoArgs(o, s_get_device), &x)) return false;
  t->dev = (int)x;
  if (t->dev < 0) return refuse("%s: CUDA tensors only", what);
  if (*dev < 0) *dev = t->dev;
  if (t->dev != *dev) return refuse("%s: tensors on different devices", what);
  PyObject* dtype = PyObject_GetAttr(o, s_dtype);
  if (!dtype) return false;
  t->dtype = dtype;
  Py_DECREF(dtype);
  int n_stride = 0;
  if (!read_ints(PyObject_GetAttr(o, s_shape), t->shape, &t->dims) ||
      !read_ints(PyObject_CallMethodNoArgs(o, s_stride), t->stride, &n_stride))
    return false;
  if (t->dims > kMaxDims) return refuse("%s: too many dimensions", what);
  PyObject* p = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!p) return false;
  t->p = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

bool read_f32(const char* what, PyObject* o, Tensor* t, int* dev, int64_t a, int64_t b, int64_t c = -1) {
  if (o == Py_None) return true;
  if (!read(what, o, t, dev)) return false;
  if (t->dtype != g_f32 || !t->is(a, b, c) || !t->contiguous())
    return c < 0 ? refuse("%s: expected contiguous float32 (%lld, %lld)", what, (long long)a, (long long)b)
                 : refuse("%s: expected contiguous float32 (%lld, %lld, %lld)", what, (long long)a, (long long)b,
                          (long long)c);
  return true;
}

bool read_i32(const char* what, PyObject* o, Tensor* t, int* dev, int64_t n) {
  if (!read(what, o, t, dev)) return false;
  if (t->dtype != g_i32 || t->dims != 1 || (n >= 0 && t->shape[0] != n) || !t->contiguous())
    return refuse("%s: a contiguous int32 vector%s", what, n >= 0 ? " as long as the batch" : "");
  return true;
}

// cu_seqlens: S + 1 bounds
bool read_bounds(PyObject* o, Tensor* t, int* dev) {
  if (!read_i32("cu_seqlens", o, t, dev, -1)) return false;
  return t->shape[0] >= 2 || refuse("cu_seqlens: at least two bounds");
}

// Packed rows [rows, heads, 128] of `dtype`, D contiguous.
bool read_rows(const char* what, PyObject* o, Tensor* t, int* dev, int64_t rows, int64_t heads, PyObject* dtype) {
  if (!read(what, o, t, dev)) return false;
  if (t->dtype != dtype || !t->is(rows, heads, kHeadDim))
    return refuse("%s: expected (%lld, %lld, %d) of the call's type", what, (long long)rows, (long long)heads,
                  kHeadDim);
  if (t->stride[2] != 1) return refuse("%s: the last dimension must be contiguous", what);
  return true;
}

rtp_strides rows_strides(const Tensor& t) { return rtp_strides{t.stride[0], t.stride[0], t.stride[1]}; }

bool dtype_code(const Tensor& t, rtp_dtype* code) {
  *code = t.dtype == g_f16 ? RTP_F16 : RTP_BF16;
  return t.dtype == g_f16 || t.dtype == g_bf16;
}

bool as_int(PyObject* o, int* to, const char* what) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) return false;
  if (x > INT32_MAX || x < INT32_MIN) return refuse("%s: out of range", what);
  *to = (int)x;
  return true;
}

// None: `otherwise`.
bool as_int_or(PyObject* o, int* to, int otherwise, const char* what) {
  *to = otherwise;
  return o == Py_None || as_int(o, to, what);
}

bool as_scale(PyObject* o, float* to) {
  *to = 0.08838834764831845f;   // 1 / sqrt(128)
  if (o == Py_None) return true;
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) return false;
  *to = (float)x;
  return true;
}

// Whether `dev` is the current device (1), is not (0), or an error (-1).
int is_current(int dev) {
  int64_t now;
  if (!read_int(PyObject_CallNoArgs(g_current_device), &now)) return -1;
  return now == dev;
}

// The raw stream: the given int, or (None) the device's current stream.
bool as_stream(PyObject* o, int dev, rtp_stream_t* to) {
  if (o != Py_None) {
    *to = (rtp_stream_t)PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  PyObject* d = PyLong_FromLong(dev);
  PyObject* s = d ? PyObject_CallOneArg(g_raw_stream, d) : nullptr;
  Py_XDECREF(d);
  if (!s) return false;
  *to = (rtp_stream_t)PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

// A head list: a bytes object of int32 values.
bool as_heads(PyObject* o, const int32_t** to, int* n) {
  if (!PyBytes_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "heads: packed int32 bytes");
    return false;
  }
  *to = reinterpret_cast<const int32_t*>(PyBytes_AS_STRING(o));
  *n = (int)(PyBytes_GET_SIZE(o) / 4);
  return true;
}

bool as_workspace(PyObject* o, Tensor* t, int* dev, size_t* bytes, size_t item) {
  if (!read("ws", o, t, dev)) return false;
  if (!t->contiguous()) return refuse("ws: a contiguous tensor");
  size_t n = item;
  for (int d = 0; d < t->dims; ++d) n *= (size_t)t->shape[d];
  *bytes = n;
  return true;
}

PyObject* done(rtp_status s, const char* what) {
  if (s == RTP_OK) Py_RETURN_TRUE;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)s, what);   // raises
  Py_XDECREF(r);
  return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_RuntimeError, "%s: status %d", what, (int)s);
}

bool want(Py_ssize_t n, Py_ssize_t m) {
  if (n == m) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", m, n);
  return false;
}

// A PagedCache, checked: bytes that the calls below take.
struct Cache {
  rtp_paged_cache c;
  int64_t B;
  int dev;
  rtp_dtype dtype;
};
const Cache* as_cache(PyObject* o) {
  if (PyBytes_Check(o) && PyBytes_GET_SIZE(o) == (Py_ssize_t)sizeof(Cache))
    return reinterpret_cast<const Cache*>(PyBytes_AS_STRING(o));
  PyErr_SetString(PyExc_TypeError, "expected a packed PagedCache");
  return nullptr;
}

// cache(k, v, table, weights) -> bytes
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 4)) return nullptr;
  Tensor k, v, table, w;
  int dev = -1;
  Cache c = {};
  if (!read("PagedCache: k", a[0], &k, &dev) || !read("PagedCache: v", a[1], &v, &dev)) return nullptr;
  bool ok = dtype_code(k, &c.dtype) && k.dims == 4 && k.shape[3] == kHeadDim && v.dtype == k.dtype && v.dims == 4;
  for (int d = 0; ok && d < 4; ++d) ok = v.shape[d] == k.shape[d];
  if (!ok) {
    refuse("PagedCache: k and v [num_pages, page_size, Hkv, %d], bf16 or fp16 alike", kHeadDim);
    return nullptr;
  }
  if (k.stride[3] != 1 || v.stride[3] != 1) {
    refuse("PagedCache: D must be contiguous");
    return nullptr;
  }
  if (!read("PagedCache: table", a[2], &table, &dev)) return nullptr;
  if (table.dtype != g_i32 || table.dims != 2 || (table.shape[1] > 1 && table.stride[1] != 1)) {
    refuse("PagedCache: table int32 [B, max_pages] with contiguous rows");
    return nullptr;
  }
  if (!read_f32("PagedCache: weights", a[3], &w, &dev, k.shape[0], k.shape[2], k.shape[1])) return nullptr;
  for (int64_t x : {k.shape[0], k.shape[1], k.shape[2], table.shape[1]})
    if (x > INT32_MAX) {
      refuse("PagedCache: too large");
      return nullptr;
    }
  c.c.k = k.p;
  c.c.v = v.p;
  c.c.ks = rtp_strides{k.stride[0], k.stride[1], k.stride[2]};
  c.c.vs = rtp_strides{v.stride[0], v.stride[1], v.stride[2]};
  c.c.weights = static_cast<float*>(w.p);
  c.c.table = static_cast<const int32_t*>(table.p);
  c.c.table_stride = table.shape[0] > 1 ? table.stride[0] : (table.shape[1] > 1 ? table.shape[1] : 1);
  c.c.num_pages = (int32_t)k.shape[0];
  c.c.page_size = (int32_t)k.shape[1];
  c.c.max_pages = (int32_t)table.shape[1];
  c.c.Hkv = (int32_t)k.shape[2];
  c.B = table.shape[0];
  c.dev = dev;
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&c), sizeof c);
}

// attn_packed(q, k, v, o, heads, cu, window, scale, lse, ws, stream) -> True,
// or False where the tensors' device is not the current one
PyObject* attn_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 11)) return nullptr;
  Tensor q, k, v, o, cu, lse, ws;
  int dev = -1, n_heads, window;
  const int32_t* heads;
  float scale;
  size_t bytes;
  rtp_dtype dtype;
  rtp_stream_t stream;
  if (!read("q", a[0], &q, &dev) || !read("k", a[1], &k, &dev)) return nullptr;
  if (!dtype_code(q, &dtype) || q.dims != 3 || k.dims != 3 || q.shape[2] != kHeadDim || q.stride[2] != 1 ||
      q.shape[0] > INT32_MAX || q.shape[1] > INT32_MAX || k.shape[1] > INT32_MAX) {
    refuse("attn_packed: q [T, Hq, %d] and k [T, Hkv, %d], bf16 or fp16, D contiguous", kHeadDim, kHeadDim);
    return nullptr;
  }
  const int64_t T = q.shape[0], Hq = q.shape[1], Hkv = k.shape[1];
  if (k.dtype != q.dtype || !k.is(T, Hkv, kHeadDim) || k.stride[2] != 1) {
    refuse("attn_packed: k [T, Hkv, %d] like q, D contiguous", kHeadDim);
    return nullptr;
  }
  if (!read_rows("v", a[2], &v, &dev, T, Hkv, q.dtype) || !read_rows("o", a[3], &o, &dev, T, Hq, q.dtype) ||
      !as_heads(a[4], &heads, &n_heads) || !read_bounds(a[5], &cu, &dev) ||
      !as_int_or(a[6], &window, INT32_MAX, "window") || !as_scale(a[7], &scale) ||
      !read_f32("lse", a[8], &lse, &dev, n_heads, T) || !as_workspace(a[9], &ws, &dev, &bytes, 1) ||
      !as_stream(a[10], dev, &stream))
    return nullptr;
  const int current = is_current(dev);
  if (current < 0) return nullptr;
  if (!current) Py_RETURN_FALSE;
  return done(f_packed(q.p, rows_strides(q), k.p, rows_strides(k), v.p, rows_strides(v), o.p, rows_strides(o), dtype,
                       (int)T, (int)Hq, (int)Hkv, heads, n_heads, static_cast<const int32_t*>(cu.p),
                       (int)(cu.shape[0] - 1), window, scale, static_cast<float*>(lse.p), ws.p, bytes, stream),
              "rtp_attn_packed");
}

// attn_key_weights(q, k, lse, weights, heads, cu, n_obs, window, scale, ws, stream)
PyObject* attn_key_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 11)) return nullptr;
  Tensor q, k, lse, w, cu, ws;
  int dev = -1, n_heads, n_obs, window;
  const int32_t* heads;
  float scale;
  size_t bytes;
  rtp_dtype dtype;
  rtp_stream_t stream;
  if (!read("q", a[0], &q, &dev) || !read("k", a[1], &k, &dev)) return nullptr;
  if (!dtype_code(q, &dtype) || q.dims != 3 || k.dims != 3 || q.shape[2] != kHeadDim || q.stride[2] != 1 ||
      k.dtype != q.dtype || !k.is(q.shape[0], k.shape[1], kHeadDim) || k.stride[2] != 1 || q.shape[0] > INT32_MAX ||
      q.shape[1] > INT32_MAX || k.shape[1] > INT32_MAX) {
    refuse("attn_key_weights: q [T, Hq, %d] and k [T, Hkv, %d], bf16 or fp16, D contiguous", kHeadDim, kHeadDim);
    return nullptr;
  }
  const int64_t T = q.shape[0], Hq = q.shape[1], Hkv = k.shape[1];
  if (!as_heads(a[4], &heads, &n_heads)) return nullptr;
  if (a[2] == Py_None || a[3] == Py_None) {
    refuse("attn_key_weights: lse and weights are needed");
    return nullptr;
  }
  if (!read_f32("lse", a[2], &lse, &dev, n_heads, T) || !read_f32("weights", a[3], &w, &dev, Hkv, T) ||
      !read_bounds(a[5], &cu, &dev) || !as_int_or(a[6], &n_obs, INT32_MAX, "n_obs") ||
      !as_int_or(a[7], &window, INT32_MAX, "window") || !as_scale(a[8], &scale) ||
      !as_workspace(a[9], &ws, &dev, &bytes, 1) || !as_stream(a[10], dev, &stream))
    return nullptr;
  const int current = is_current(dev);
  if (current < 0) return nullptr;
  if (!current) Py_RETURN_FALSE;
  return done(f_weights(q.p, rows_strides(q), k.p, rows_strides(k), dtype, (int)T, (int)Hq, (int)Hkv, heads, n_heads,
                        static_cast<const int32_t*>(cu.p), (int)(cu.shape[0] - 1), static_cast<const float*>(lse.p),
                        n_obs, window, scale, static_cast<float*>(w.p), ws.p, bytes, stream),
              "rtp_attn_key_weights");
}

// paged_append(cache, k, v, cu, pos, weights, stream)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 7)) return nullptr;
  const Cache* c = as_cache(a[0]);
  if (!c) return nullptr;
  Tensor k, v, cu, pos, w;
  int dev = c->dev;
  rtp_stream_t stream;
  PyObject* dtype = c->dtype == RTP_F16 ? g_f16 : g_bf16;
  if (!read("k", a[1], &k, &dev)) return nullptr;
  if (k.dims != 3 || k.dtype != dtype || !k.is(k.shape[0], c->c.Hkv, kHeadDim) || k.stride[2] != 1 ||
      k.shape[0] > INT32_MAX) {
    refuse("paged_append: k [T, Hkv, %d] of the cache's type and heads, D contiguous", kHeadDim);
    return nullptr;
  }
  const int64_t T = k.shape[0];
  if (!read_rows("v", a[2], &v, &dev, T, c->c.Hkv, dtype) || !read_bounds(a[3], &cu, &dev)) return nullptr;
  const int64_t S = cu.shape[0] - 1;
  if (S > c->B) {
    refuse("paged_append: more sequences than table rows");
    return nullptr;
  }
  if (!read_i32("pos", a[4], &pos, &dev, S) || !read_f32("weights", a[5], &w, &dev, c->c.Hkv, T) ||
      !as_stream(a[6], dev, &stream))
    return nullptr;
  const int current = is_current(dev);
  if (current < 0) return nullptr;
  if (!current) Py_RETURN_FALSE;
  return done(f_append(&c->c, k.p, rows_strides(k), v.p, rows_strides(v), static_cast<const float*>(w.p), (int)T,
                       static_cast<const int32_t*>(cu.p), (int)S, static_cast<const int32_t*>(pos.p), stream),
              "rtp_paged_append");
}

// paged_attn_decode(q, cache, lens, o, heads, window, sink, scale, max_len, lse, weights_out, ws, stream)
PyObject* paged_attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 13)) return nullptr;
  const Cache* c = as_cache(a[1]);
  if (!c) return nullptr;
  Tensor q, lens, o, lse, w, ws;
  int dev = c->dev, n_heads, window, sink, max_len;
  const int32_t* heads;
  float scale;
  size_t bytes;
  rtp_stream_t stream;
  PyObject* dtype = c->dtype == RTP_F16 ? g_f16 : g_bf16;
  if (!read("q", a[0], &q, &dev)) return nullptr;
  if (q.dims != 3 || q.dtype != dtype || q.shape[2] != kHeadDim || q.stride[2] != 1 || q.shape[1] > INT32_MAX) {
    refuse("paged_attn_decode: q [B, Hq, %d] of the cache's type, D contiguous", kHeadDim);
    return nullptr;
  }
  const int64_t B = q.shape[0], Hq = q.shape[1];
  if (B > c->B) {
    refuse("paged_attn_decode: more sequences than table rows");
    return nullptr;
  }
  if (!read_i32("lens", a[2], &lens, &dev, B) || !read_rows("o", a[3], &o, &dev, B, Hq, dtype) ||
      !as_heads(a[4], &heads, &n_heads) || !as_int_or(a[5], &window, INT32_MAX, "window") ||
      !as_int(a[6], &sink, "sink") || !as_scale(a[7], &scale) || !as_int(a[8], &max_len, "max_len") ||
      !read_f32("lse", a[9], &lse, &dev, B, n_heads) ||
      !read_f32("weights_out", a[10], &w, &dev, c->c.num_pages, c->c.Hkv, c->c.page_size) ||
      !as_workspace(a[11], &ws, &dev, &bytes, 1) || !as_stream(a[12], dev, &stream))
    return nullptr;
  const int current = is_current(dev);
  if (current < 0) return nullptr;
  if (!current) Py_RETURN_FALSE;
  return done(f_decode(q.p, rows_strides(q), &c->c, static_cast<const int32_t*>(lens.p), max_len, o.p,
                       rows_strides(o), c->dtype, (int)B, (int)Hq, heads, n_heads, window, sink, scale,
                       static_cast<float*>(lse.p), static_cast<float*>(w.p), ws.p, bytes, stream),
              "rtp_paged_attn_decode");
}

// decode_workspace_size(B, max_len, n_heads, window, sink, with_weights) -> int
PyObject* decode_workspace_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 6)) return nullptr;
  int B, max_len, n_heads, window, sink;
  const int weights = PyObject_IsTrue(a[5]);
  if (weights < 0 || !as_int(a[0], &B, "B") || !as_int(a[1], &max_len, "max_len") ||
      !as_int(a[2], &n_heads, "n_heads") || !as_int_or(a[3], &window, INT32_MAX, "window") ||
      !as_int(a[4], &sink, "sink"))
    return nullptr;
  return PyLong_FromSize_t(f_decode_ws(B, max_len, n_heads, window, sink, weights));
}

// cache_evict(cache, out, lens, budget, sink, recent, idx, new_lens, max_len, stream)
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 10)) return nullptr;
  const Cache *c = as_cache(a[0]), *to = c ? as_cache(a[1]) : nullptr;
  if (!to) return nullptr;
  Tensor lens, idx, new_lens;
  int dev = c->dev, budget, sink, recent, max_len;
  rtp_stream_t stream;
  if (to->dev != c->dev || to->dtype != c->dtype) {
    refuse("cache_evict: caches of different types or devices");
    return nullptr;
  }
  if (!read_i32("lens", a[2], &lens, &dev, -1) || !as_int(a[3], &budget, "budget") || !as_int(a[4], &sink, "sink") ||
      !as_int(a[5], &recent, "recent") || !as_int(a[8], &max_len, "max_len") || !read("idx", a[6], &idx, &dev))
    return nullptr;
  const int64_t B = lens.shape[0];
  if (B > c->B || B > to->B) {
    refuse("cache_evict: more sequences than table rows");
    return nullptr;
  }
  if (idx.dtype != g_i32 || !idx.is(B, c->c.Hkv, budget < 0 ? 0 : budget) || !idx.contiguous()) {
    refuse("idx: expected contiguous int32 (%lld, %d, %d)", (long long)B, (int)c->c.Hkv, budget);
    return nullptr;
  }
  if (!read_i32("new_lens", a[7], &new_lens, &dev, B) || !as_stream(a[9], dev, &stream)) return nullptr;
  const int current = is_current(dev);
  if (current < 0) return nullptr;
  if (!current) Py_RETURN_FALSE;
  return done(f_evict(&c->c, &to->c, (int)B, static_cast<const int32_t*>(lens.p), max_len, budget, sink, recent,
                      static_cast<int32_t*>(idx.p), static_cast<int32_t*>(new_lens.p), stream),
              "rtp_cache_evict");
}

// setup(error, check, bf16, f16, f32, i32, raw_stream, current_device, packed,
// weights, append, decode, evict, decode_ws): the last six are function addresses
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 14)) return nullptr;
  PyObject** to[] = {&g_error, &g_check, &g_bf16, &g_f16, &g_f32, &g_i32, &g_raw_stream, &g_current_device};
  for (int i = 0; i < 8; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*to[i], a[i]);
  }
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[8 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_packed = reinterpret_cast<decltype(f_packed)>(f[0]);
  f_weights = reinterpret_cast<decltype(f_weights)>(f[1]);
  f_append = reinterpret_cast<decltype(f_append)>(f[2]);
  f_decode = reinterpret_cast<decltype(f_decode)>(f[3]);
  f_evict = reinterpret_cast<decltype(f_evict)>(f[4]);
  f_decode_ws = reinterpret_cast<decltype(f_decode_ws)>(f[5]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(setup), FAST(cache), FAST(attn_packed), FAST(attn_key_weights), FAST(paged_append),
                         FAST(paged_attn_decode), FAST(decode_workspace_size), FAST(cache_evict),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Arguments of the serving calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device) return nullptr;
  return PyModule_Create(&module);
}

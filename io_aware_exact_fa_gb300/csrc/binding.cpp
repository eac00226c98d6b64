/* Argument checks and calls of the paged operators' entry points, for the case that
 * a serving step makes over and over: tensors that fit, on the current device and
 * its current stream. Every function returns NotImplemented for anything else
 * (another device or stream, a tensor that does not fit, no workspace), and the
 * Python code beside it, which says what is wrong or makes what is missing, takes
 * the same arguments. What both accept they pass on alike. (Asked through Python for
 * its type, device, shape, strides and address a tensor costs 0.35 us, a call has up to
 * twelve, and a new one 0.9 us: a decode step 8 us in place of 12, append and read
 * back 12.6 in place of 20.)
 *
 * A function that made its call returns (status, results). No C++ exception leaves them; where a result could not be
 * allocated they return NULL with Python's exception set. */
#define PY_SSIZE_T_CLEAN
#ifdef FA_TORCH_CUDA
#include <ATen/cuda/EmptyTensor.h>
#else
#include <ATen/ops/empty_strided.h>
#endif
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "fa.h"

static PyObject *g_stream, *g_device;

static struct {
  fa_status (*append_fp4)(const void*, const void*, const void*, void*, void*, void*, void*, uint8_t*, uint8_t*, const int*,
                          int64_t, const int*, const int*, const int*, const int64_t*, const void*, const void*,
                          const int64_t*, int, int, int, int, int, int, int, int, int, int, float, float, int, void*);
  fa_status (*decode_fp4)(const void*, const int64_t*, const void*, const void*, const uint8_t*, const uint8_t*, const int*,
                          int64_t, const int*, void*, const int64_t*, float*, int, int, int, int, int, int, int, int, float,
                          int, void*, size_t, void*);
  fa_status (*read)(const void*, const void*, const void*, const void*, int, const int*, int64_t, const int*, const int*,
                    void*, void*, const int64_t*, int, int, int, int, int, int, int, void*);
  fa_status (*weigh)(const void*, const int64_t*, const float*, const void*, const void*, int, const int*, int64_t,
                     const int*, float*, int64_t, int, int, int, int, int, int, int, int, float, void*);
  fa_status (*evict)(const float*, int64_t, void*, void*, void*, void*, int, const int*, int64_t, const int*, const int*,
                     const int*, int64_t, int*, int*, int*, float*, int64_t, int, int, int, int, int, int, int, int, int,
                     int, void*);
} g_fn;

/* An address, as whatever pointer a call takes. */
struct Address {
  void* p;
  Address(void* x = NULL) : p(x) {}
  template <class T>
  operator T*() const {
    return static_cast<T*>(p);
  }
};

#define MAX_DIM 4
typedef struct {
  at::ScalarType dtype;
  int dev, dims;
  int64_t shape[MAX_DIM], stride[MAX_DIM];
  Address ptr;
} Tensor;

/* 1: a CUDA tensor with elements. Leaves no exception set. */
static int tensor_of(PyObject* o, Tensor* t) {
  if (!THPVariable_Check(o)) return 0;
  try { /* (tensors without strides, sizes or memory of their own throw) */
    const at::Tensor& x = THPVariable_Unpack(o);
    if (!x.is_cuda() || x.layout() != at::kStrided || x.dim() > MAX_DIM) return 0;
    t->dtype = x.scalar_type();
    t->dev = x.get_device();
    t->dims = (int)x.dim();
    for (int i = 0; i < t->dims; ++i) {
      t->shape[i] = x.size(i), t->stride[i] = x.stride(i);
      if (t->shape[i] < 1 || t->shape[i] > INT32_MAX || t->stride[i] < 0) return 0;
    }
    t->ptr = x.data_ptr();
    return t->ptr.p != NULL;
  } catch (...) {
    return 0;
  }
}

static int whole(const Tensor* t) {
  int64_t step = 1;
  for (int i = t->dims - 1; i >= 0; --i) {
    if (t->shape[i] > 1 && t->stride[i] != step) return 0;
    step *= t->shape[i];
  }
  return 1;
}

/* A contiguous tensor of one or more dimensions, the first of which may be -1 (any). */
static int vec(PyObject* o, Tensor* t, at::ScalarType dtype, int dev, int dims, int64_t a, int64_t b, int64_t c) {
  const int64_t want[3] = {a, b, c};
  if (!tensor_of(o, t) || t->dtype != dtype || t->dev != dev || t->dims != dims || !whole(t)) return 0;
  for (int i = 0; i < dims; ++i)
    if (want[i] >= 0 && t->shape[i] != want[i]) return 0;
  return 1;
}

/* bf16 [.., d] with contiguous d. */
static int heads(PyObject* o, Tensor* t, int dims) {
  return tensor_of(o, t) && t->dtype == at::kBFloat16 && t->dims == dims && t->stride[dims - 1] == 1;
}

/* Bytes, or pairs of 4-bit values (by name: older torch has no such type). */
static int fp4_bytes(at::ScalarType t) { return t == at::kByte || strcmp(c10::toString(t), "Float4_e2m1fn_x2") == 0; }

typedef struct {
  Address p, s;
  int kind, pages, Hkv, page, d;
} Pool;

static int pool_of(PyObject* pages, PyObject* scale, int dev, Pool* x) {
  Tensor p, s;
  if (!tensor_of(pages, &p) || p.dev != dev || p.dims != 4 || !whole(&p)) return 0;
  x->p = p.ptr, x->s = NULL;
  x->pages = (int)p.shape[0], x->Hkv = (int)p.shape[1], x->page = (int)p.shape[2], x->d = (int)p.shape[3];
  if (scale == Py_None) {
    x->kind = FA_PAGES_BF16;
    return p.dtype == at::kBFloat16;
  }
  if (!tensor_of(scale, &s) || s.dev != dev || !whole(&s) || s.shape[0] != p.shape[0] || s.shape[1] != p.shape[1]) return 0;
  x->s = s.ptr;
  if (s.dtype == at::kByte) {
    if (p.shape[3] > 1024) return 0;
    x->kind = FA_PAGES_FP4, x->d *= 2;
    return fp4_bytes(p.dtype) && s.dims == 4 && s.shape[2] == p.shape[2] && s.shape[3] == x->d / 16;
  }
  x->kind = FA_PAGES_E4M3;
  return s.dtype == at::kFloat && s.dims == 2 && (p.dtype == at::kFloat8_e4m3fn || p.dtype == at::kByte);
}

static int same_pool(const Pool* a, const Pool* b) {
  return a->kind == b->kind && a->pages == b->pages && a->Hkv == b->Hkv && a->page == b->page && a->d == b->d;
}

/* int32 [B, width] with contiguous rows; B < 0: any. */
static int table_of(PyObject* o, Tensor* t, int dev, int64_t B) {
  return tensor_of(o, t) && t->dtype == at::kInt && t->dev == dev && t->dims == 2 && (t->shape[1] == 1 || t->stride[1] == 1) &&
         (B < 0 || t->shape[0] == B);
}

/* fp32 [B, Hkv, width], rows contiguous and evenly apart. */
static int weights_of(PyObject* o, Tensor* t, int dev, int64_t B, int64_t Hkv, int64_t* step) {
  if (!tensor_of(o, t) || t->dtype != at::kFloat || t->dev != dev || t->dims != 3 || t->shape[0] != B || t->shape[1] != Hkv ||
      (t->stride[2] != 1 && t->shape[2] > 1))
    return 0;
  *step = Hkv > 1 ? t->stride[1] : B > 1 ? t->stride[0] : t->shape[2];
  return !((B > 1 && t->stride[0] != Hkv * *step) || (B * Hkv > 1 && *step < t->shape[2]));
}

/* The current stream of `dev`, if that is the current device. */
static int stream_of(int dev, PyObject* given, void** out) {
  if (given != Py_None) return 0;
  PyObject* x = PyObject_CallNoArgs(g_device);
  const long here = x == NULL ? -1 : PyLong_AsLong(x);
  Py_XDECREF(x);
  if (here == dev && (x = PyLong_FromLong(dev)) != NULL) {
    PyObject* y = PyObject_CallOneArg(g_stream, x);
    Py_DECREF(x);
    if (y != NULL) {
      *out = PyLong_AsVoidPtr(y);
      Py_DECREF(y);
      if (*out != NULL || !PyErr_Occurred()) return 1;
    }
  }
  PyErr_Clear();
  return 0;
}

/* A new tensor on device `dev`; its address in *ptr. */
static PyObject* make(int dims, const int64_t* shape, const int64_t* stride, at::ScalarType dtype, int dev, void** ptr) {
  HANDLE_TH_ERRORS
  const at::IntArrayRef sizes(shape, dims), steps(stride, dims);
  const at::Device where(at::kCUDA, (c10::DeviceIndex)dev);
#ifdef FA_TORCH_CUDA /* (the dispatcher before it takes as long as the rest) */
  at::Tensor t = at::detail::empty_strided_cuda(sizes, steps, dtype, where);
#else
  at::Tensor t = at::empty_strided(sizes, steps, at::TensorOptions().dtype(dtype).device(where));
#endif
  *ptr = t.data_ptr();
  return THPVariable_Wrap(std::move(t));
  END_HANDLE_TH_ERRORS
}
static PyObject* make3(int64_t a, int64_t b, int64_t c, at::ScalarType dtype, int dev, void** ptr) {
  const int64_t shape[3] = {a, b, c}, stride[3] = {b * c, c, 1};
  return make(3, shape, stride, dtype, dev, ptr);
}

/* An integer in [lo, hi], or for None the default, where that lies in the range. */
static int int_of(PyObject* o, int64_t lo, int64_t hi, int64_t none, int* out) {
  int64_t x = none;
  if (o != Py_None) {
    if (!PyLong_CheckExact(o)) return 0;
    x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return 0;
    }
  }
  if (x < lo || x > hi) return 0;
  *out = (int)x;
  return 1;
}
static int float_of(PyObject* o, double none, float* out) { /* a default of NaN: None does not do */
  if (o == Py_None) {
    if (isnan(none)) return 0;
    *out = (float)none;
  } else {
    if (!PyFloat_CheckExact(o)) return 0;
    *out = (float)PyFloat_AS_DOUBLE(o);
  }
  return 1;
}

static PyObject* answer(fa_status st, PyObject* results) {
  PyObject* r;
  if (results == NULL) return NULL;
  r = Py_BuildValue("iN", (int)st, results);
  return r;
}
#define FALL_BACK \
  do {            \
    Py_RETURN_NOTIMPLEMENTED; \
  } while (0)

/* q, lse, k_pages, block_table, seqlens_k, weights, k_scale, scale, max_len, stream */
static PyObject* b_weigh(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, lse, table, lens, w;
  Pool k;
  int64_t step;
  int max_len;
  float scale;
  void* stream;
  fa_status st;
  if (n != 10 || !heads(a[0], &q, 4) || !vec(a[1], &lse, at::kFloat, q.dev, 3, q.shape[0], q.shape[1], q.shape[2]) ||
      !pool_of(a[2], a[6], q.dev, &k) || k.d != q.shape[3] || !table_of(a[3], &table, q.dev, q.shape[0]) ||
      !vec(a[4], &lens, at::kInt, q.dev, 1, q.shape[0], 0, 0) || !weights_of(a[5], &w, q.dev, q.shape[0], k.Hkv, &step))
    FALL_BACK;
  {
    const int64_t rows = table.shape[1] * k.page, most = w.shape[2] < rows ? w.shape[2] : rows;
    if (!int_of(a[8], 0, most < INT32_MAX ? most : INT32_MAX, most, &max_len) ||
        !float_of(a[7], 1.0 / sqrt((double)k.d), &scale) || !stream_of(q.dev, a[9], &stream))
      FALL_BACK;
  }
  Py_BEGIN_ALLOW_THREADS
  st = g_fn.weigh(q.ptr, q.stride, lse.ptr, k.p, k.s, k.kind, table.ptr, table.stride[0], lens.ptr, w.ptr, step,
                  (int)q.shape[0], (int)q.shape[1], k.Hkv, (int)q.shape[2], k.d, k.pages, k.page, max_len, scale, stream);
  Py_END_ALLOW_THREADS
  return answer(st, Py_NewRef(a[5]));
}

/* q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, scale, max_len, num_splits, workspace, out, lse, with_lse,
 * stream */
static PyObject* b_decode_fp4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, table, lens, ws, o, l;
  Pool k, v;
  int max_len, splits;
  int64_t os[4], bytes = 1;
  float scale;
  void* stream;
  Address op, lp;
  PyObject *out = NULL, *lse = NULL;
  fa_status st;
  if (n != 15 || !heads(a[0], &q, 4) || !pool_of(a[1], a[3], q.dev, &k) ||
      !pool_of(a[2], a[4], q.dev, &v) || !same_pool(&k, &v) || k.kind != FA_PAGES_FP4 || k.d != q.shape[3] ||
      !table_of(a[5], &table, q.dev, q.shape[0]) || !vec(a[6], &lens, at::kInt, q.dev, 1, q.shape[0], 0, 0) ||
      !tensor_of(a[10], &ws) || ws.dtype != at::kByte || ws.dev != q.dev || !whole(&ws))
    FALL_BACK;
  for (int i = 0; i < ws.dims; ++i) bytes *= ws.shape[i];
  {
    const int64_t rows = table.shape[1] * k.page;
    if (!int_of(a[8], 0, rows < INT32_MAX ? rows : INT32_MAX, rows, &max_len) || !int_of(a[9], 0, INT32_MAX, -1, &splits) ||
        !float_of(a[7], 1.0 / sqrt((double)k.d), &scale))
      FALL_BACK;
  }
  if (a[11] != Py_None) {
    if (!heads(a[11], &o, 4) || o.dev != q.dev) FALL_BACK;
    for (int i = 0; i < 4; ++i)
      if (o.shape[i] != q.shape[i]) FALL_BACK;
  }
  if (a[12] != Py_None && !vec(a[12], &l, at::kFloat, q.dev, 3, q.shape[0], q.shape[1], q.shape[2])) FALL_BACK;
  if (!PyBool_Check(a[13]) || !stream_of(q.dev, a[14], &stream)) FALL_BACK;
  if (a[11] != Py_None) {
    out = Py_NewRef(a[11]);
    op = o.ptr;
    for (int i = 0; i < 3; ++i) os[i] = o.stride[i];
  } else { /* laid out like q where that is token-major, else contiguous */
    const int64_t H = q.shape[1], Nq = q.shape[2], d = q.shape[3];
    const int major = q.stride[1] == d && q.stride[2] == H * d;
    os[0] = H * Nq * d, os[1] = major ? d : Nq * d, os[2] = major ? H * d : d, os[3] = 1;
    out = make(4, q.shape, os, at::kBFloat16, q.dev, &op.p);
    if (out == NULL) return NULL;
  }
  if (a[12] != Py_None) {
    lse = Py_NewRef(a[12]);
    lp = l.ptr;
  } else if (a[13] == Py_True) {
    lse = make3(q.shape[0], q.shape[1], q.shape[2], at::kFloat, q.dev, &lp.p);
    if (lse == NULL) {
      Py_DECREF(out);
      return NULL;
    }
  } else {
    lse = Py_NewRef(Py_None);
  }
  Py_BEGIN_ALLOW_THREADS
  st = g_fn.decode_fp4(q.ptr, q.stride, k.p, v.p, k.s, v.s, table.ptr, table.stride[0], lens.ptr, op, os, lp,
                       (int)q.shape[0], (int)q.shape[1], k.Hkv, (int)q.shape[2], k.d, k.pages, k.page, max_len, scale,
                       splits, ws.ptr, (size_t)bytes, stream);
  Py_END_ALLOW_THREADS
  return answer(st, Py_BuildValue("NN", out, lse));
}

/* q, k, v, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, cu_seqlens, max_new, turns, interleaved, rot_scale,
 * q_weight, k_weight, eps, offsets, q_out, k_out, with_k, stream */
static PyObject* b_append_fp4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, k, v, table, lens, cu, turns, qw, kw, off, qo, ko;
  Pool kp, vp;
  int64_t st10[10], T, H, Hkv, d, B;
  int max_new, rot = 0, inter;
  float rot_scale, eps;
  void* stream;
  Address qop, kop;
  PyObject *q_out = NULL, *k_out = NULL;
  fa_status st;
  if (n != 22 || !heads(a[0], &q, 3) || !heads(a[1], &k, 3) || !heads(a[2], &v, 3) || k.dev != q.dev ||
      v.dev != q.dev)
    FALL_BACK;
  T = q.shape[0], H = q.shape[1], d = q.shape[2], Hkv = k.shape[1];
  if (k.shape[0] != T || k.shape[2] != d || v.shape[0] != T || v.shape[1] != Hkv || v.shape[2] != d ||
      !pool_of(a[3], a[5], q.dev, &kp) || !pool_of(a[4], a[6], q.dev, &vp) || !same_pool(&kp, &vp) ||
      kp.kind != FA_PAGES_FP4 || kp.Hkv != Hkv || kp.d != d || !table_of(a[7], &table, q.dev, -1))
    FALL_BACK;
  B = table.shape[0];
  if (!vec(a[8], &lens, at::kInt, q.dev, 1, B, 0, 0) || (a[9] != Py_None && !vec(a[9], &cu, at::kInt, q.dev, 1, B + 1, 0, 0)) ||
      !int_of(a[10], 0, INT32_MAX, -1, &max_new) || (a[11] != Py_None && !vec(a[11], &turns, at::kLong, q.dev, 1, -1, 0, 0)) ||
      !PyBool_Check(a[12]) || !float_of(a[13], NAN, &rot_scale) ||
      (a[14] != Py_None && !vec(a[14], &qw, at::kBFloat16, q.dev, 1, d, 0, 0)) ||
      (a[15] != Py_None && !vec(a[15], &kw, at::kBFloat16, q.dev, 1, d, 0, 0)) || !float_of(a[16], NAN, &eps) ||
      (a[17] != Py_None && !vec(a[17], &off, at::kInt, q.dev, 1, B, 0, 0)) || !PyBool_Check(a[20]))
    FALL_BACK;
  inter = a[12] == Py_True;
  if (a[11] != Py_None) {
    if (turns.shape[0] > 1024) FALL_BACK;
    rot = 2 * (int)turns.shape[0];
  }
  if (a[18] != Py_None && (!heads(a[18], &qo, 3) || qo.dev != q.dev || qo.shape[0] != T || qo.shape[1] != H || qo.shape[2] != d))
    FALL_BACK;
  if (a[19] != Py_None && (!heads(a[19], &ko, 3) || ko.dev != q.dev || ko.shape[0] != T || ko.shape[1] != Hkv || ko.shape[2] != d))
    FALL_BACK;
  if (!stream_of(q.dev, a[21], &stream)) FALL_BACK;
  st10[0] = q.stride[0], st10[1] = q.stride[1], st10[2] = k.stride[0], st10[3] = k.stride[1];
  st10[4] = v.stride[0], st10[5] = v.stride[1], st10[6] = H * d, st10[7] = d, st10[8] = Hkv * d, st10[9] = d;
  if (a[18] != Py_None) {
    q_out = Py_NewRef(a[18]);
    qop = qo.ptr, st10[6] = qo.stride[0], st10[7] = qo.stride[1];
  } else {
    q_out = make3(T, H, d, at::kBFloat16, q.dev, &qop.p);
    if (q_out == NULL) return NULL;
  }
  if (a[19] != Py_None) {
    k_out = Py_NewRef(a[19]);
    kop = ko.ptr, st10[8] = ko.stride[0], st10[9] = ko.stride[1];
  } else if (a[20] == Py_True) {
    k_out = make3(T, Hkv, d, at::kBFloat16, q.dev, &kop.p);
    if (k_out == NULL) {
      Py_DECREF(q_out);
      return NULL;
    }
  } else {
    k_out = Py_NewRef(Py_None);
    st10[8] = st10[9] = 0;
  }
  Py_BEGIN_ALLOW_THREADS
  st = g_fn.append_fp4(q.ptr, k.ptr, v.ptr, qop, kop, kp.p, vp.p, kp.s, vp.s, table.ptr, table.stride[0], lens.ptr,
                       a[9] == Py_None ? Address() : cu.ptr, a[17] == Py_None ? Address() : off.ptr,
                       a[11] == Py_None ? Address() : turns.ptr, a[14] == Py_None ? Address() : qw.ptr,
                       a[15] == Py_None ? Address() : kw.ptr, st10, (int)B, (int)T, (int)H, (int)Hkv, (int)d, kp.pages, kp.page,
                       (int)table.shape[1], rot, inter, rot_scale, eps, max_new, stream);
  Py_END_ALLOW_THREADS
  return answer(st, Py_BuildValue("NN", q_out, k_out));
}

/* k_pages, v_pages, block_table, seqlens_k, cu_seqlens, total, k_scale, v_scale, k_out, v_out, stream */
static PyObject* b_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor first, table, lens, cu, o[2];
  Pool k, v;
  int total, dev;
  int64_t st4[4];
  void* stream;
  Address op[2];
  PyObject* out[2] = {NULL, NULL};
  fa_status st;
  if (n != 11 || !tensor_of(a[3], &first)) FALL_BACK;
  dev = first.dev;
  if (!pool_of(a[0], a[6], dev, &k) || !pool_of(a[1], a[7], dev, &v) || !same_pool(&k, &v) ||
      !table_of(a[2], &table, dev, -1) || !vec(a[3], &lens, at::kInt, dev, 1, table.shape[0], 0, 0) ||
      !vec(a[4], &cu, at::kInt, dev, 1, table.shape[0] + 1, 0, 0) || !int_of(a[5], 1, INT32_MAX, -1, &total))
    FALL_BACK;
  for (int i = 0; i < 2; ++i)
    if (a[8 + i] != Py_None && (!heads(a[8 + i], &o[i], 3) || o[i].dev != dev || o[i].shape[0] != total ||
                                o[i].shape[1] != k.Hkv || o[i].shape[2] != k.d))
      FALL_BACK;
  if (!stream_of(dev, a[10], &stream)) FALL_BACK;
  for (int i = 0; i < 2; ++i) {
    if (a[8 + i] != Py_None) {
      out[i] = Py_NewRef(a[8 + i]);
      op[i] = o[i].ptr, st4[2 * i] = o[i].stride[0], st4[2 * i + 1] = o[i].stride[1];
    } else {
      out[i] = make3(total, k.Hkv, k.d, at::kBFloat16, dev, &op[i].p);
      if (out[i] == NULL) {
        Py_XDECREF(out[0]);
        return NULL;
      }
      st4[2 * i] = (int64_t)k.Hkv * k.d, st4[2 * i + 1] = k.d;
    }
  }
  Py_BEGIN_ALLOW_THREADS
  st = g_fn.read(k.p, v.p, k.s, v.s, k.kind, table.ptr, table.stride[0], lens.ptr, cu.ptr, op[0], op[1], st4,
                 (int)table.shape[0], total, k.Hkv, k.d, k.pages, k.page, (int)table.shape[1], stream);
  Py_END_ALLOW_THREADS
  return answer(st, Py_BuildValue("NN", out[0], out[1]));
}

/* weights, k_pages, v_pages, block_table, seqlens_k, new_table, keep, first, recent, k_scale, v_scale, offsets, max_len,
 * new_weights, stream */
static PyObject* b_evict(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor head, w, table, lens, nt, off, nw;
  Pool k, v;
  int dev, keep, first, recent, max_len, B;
  int64_t step, nstep, one = 1, b64;
  void* stream;
  Address kept_p, lens_p, off_p, nw_p;
  PyObject *kept = NULL, *nl = NULL, *no = NULL, *nwt = NULL;
  fa_status st;
  if (n != 15 || !tensor_of(a[4], &head)) FALL_BACK;
  dev = head.dev;
  if (!pool_of(a[1], a[9], dev, &k) || !pool_of(a[2], a[10], dev, &v) || !same_pool(&k, &v) || !table_of(a[3], &table, dev, -1) ||
      !vec(a[4], &lens, at::kInt, dev, 1, table.shape[0], 0, 0) || !table_of(a[5], &nt, dev, table.shape[0]) ||
      !weights_of(a[0], &w, dev, table.shape[0], k.Hkv, &step) ||
      (a[11] != Py_None && !vec(a[11], &off, at::kInt, dev, 1, table.shape[0], 0, 0)) || !int_of(a[6], 1, 1 << 30, -1, &keep) ||
      !int_of(a[7], 0, INT32_MAX, -1, &first) || !int_of(a[8], 0, INT32_MAX, -1, &recent))
    FALL_BACK;
  B = (int)table.shape[0], b64 = B;
  {
    const int64_t rows = table.shape[1] * k.page, most = w.shape[2] < rows ? w.shape[2] : rows;
    if (!int_of(a[12], 0, most < INT32_MAX ? most : INT32_MAX, most, &max_len) ||
        (keep < max_len ? keep : max_len) > nt.shape[1] * k.page)
      FALL_BACK;
  }
  if (a[13] != Py_None && !weights_of(a[13], &nw, dev, B, k.Hkv, &nstep)) FALL_BACK;
  if (!stream_of(dev, a[14], &stream)) FALL_BACK;
  kept = make3(B, k.Hkv, keep, at::kInt, dev, &kept_p.p);
  nl = kept == NULL ? NULL : make(1, &b64, &one, at::kInt, dev, &lens_p.p);
  no = nl == NULL ? NULL : make(1, &b64, &one, at::kInt, dev, &off_p.p);
  if (a[13] != Py_None) {
    nwt = Py_NewRef(a[13]);
    nw_p = nw.ptr;
  } else if (no != NULL) {
    nwt = make3(B, k.Hkv, keep, at::kFloat, dev, &nw_p.p);
    nw.shape[2] = nstep = keep;
  }
  if (no == NULL || nwt == NULL) {
    Py_XDECREF(kept);
    Py_XDECREF(nl);
    Py_XDECREF(no);
    Py_XDECREF(nwt);
    return NULL;
  }
  Py_BEGIN_ALLOW_THREADS
  st = g_fn.evict(w.ptr, step, k.p, v.p, k.s, v.s, k.kind, table.ptr, table.stride[0], lens.ptr,
                  a[11] == Py_None ? Address() : off.ptr, nt.ptr, nt.stride[0], kept_p, lens_p, off_p, nw_p, nstep,
                  (int)nw.shape[2], B, k.Hkv, k.d, k.pages, k.page, max_len, keep, first, recent, stream);
  Py_END_ALLOW_THREADS
  return answer(st, Py_BuildValue("NNNN", kept, nl, nwt, no));
}

/* setup(callables, addresses): (raw stream of a device, current device), (append_fp4, decode_fp4, read, weigh, evict) */
static PyObject* b_setup(PyObject* self, PyObject* args) {
  PyObject* x[2];
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "(OO)(KKKKK)", &x[0], &x[1], &f[0], &f[1], &f[2], &f[3], &f[4])) return NULL;
  Py_XSETREF(g_stream, Py_NewRef(x[0]));
  Py_XSETREF(g_device, Py_NewRef(x[1]));
  *(void**)&g_fn.append_fp4 = (void*)(uintptr_t)f[0];
  *(void**)&g_fn.decode_fp4 = (void*)(uintptr_t)f[1];
  *(void**)&g_fn.read = (void*)(uintptr_t)f[2];
  *(void**)&g_fn.weigh = (void*)(uintptr_t)f[3];
  *(void**)&g_fn.evict = (void*)(uintptr_t)f[4];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", b_setup, METH_VARARGS, "types, callables and addresses that the calls use"},
    {"append_fp4", (PyCFunction)(void (*)(void))b_append_fp4, METH_FASTCALL, "fa_append_paged_fp4"},
    {"decode_fp4", (PyCFunction)(void (*)(void))b_decode_fp4, METH_FASTCALL, "fa_decode_paged_fp4"},
    {"read", (PyCFunction)(void (*)(void))b_read, METH_FASTCALL, "fa_read_paged"},
    {"weigh", (PyCFunction)(void (*)(void))b_weigh, METH_FASTCALL, "fa_weigh_paged"},
    {"evict", (PyCFunction)(void (*)(void))b_evict, METH_FASTCALL, "fa_evict_paged"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Checks and calls of the paged operators.", -1, methods};

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }

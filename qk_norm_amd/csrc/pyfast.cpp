/* Python entry points of the QK-Norm C ABI with no argument-conversion layer.
 *
 * Two kinds of call, both argument marshalling only (every step of the work
 * runs in libqknorm.so):
 * - per_head, layerwise, partial_sumsq, apply_scalar, the qkv_proj_per_head
 *   calls (plain, _ws, _noalloc), quant_rows, qkv_proj_quant and the kv calls take the C ABI's arguments as Python ints and floats
 *   (pointers as ints, 0 or None for NULL), convert them to C values and call the library's
 *   extern "C" function, returning its int status.  They replace ctypes,
 *   whose per-call conversion of eleven or more arguments costs about a
 *   microsecond, a third of a decode-sized launch.
 * - per_head_t, layerwise_t and the other _t calls take the binding's own arguments (torch
 *   tensors) and read from them what the binding's Python path would, through
 *   torch's C++ tensor API (no Python-level attribute calls, each of which
 *   costs about 0.1 us): the common case only, and None for anything else
 *   (see below).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qknorm.h"

static int as_ptr(PyObject* o, void** out) {
  if (o == Py_None) {
    *out = NULL;
    return 0;
  }
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) return -1;
  *out = (void*)(uintptr_t)v;
  return 0;
}

static int as_i64(PyObject* o, int64_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *out = (int64_t)v;
  return 0;
}

static int as_i32(PyObject* o, int32_t* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit a 32-bit int");
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

static int as_f32(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)v;
  return 0;
}

static int nargs_ok(Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, n);
  return 0;
}

/* per_head(qkv, T, ld, hq, hkv, head_dim, gamma_q, gamma_k, eps, dtype, stream) -> int */
static PyObject* f_per_head(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *qkv, *gq, *gk, *st;
  int64_t T, ld;
  int32_t hq, hkv, d, dt;
  float eps;
  if (!nargs_ok(n, 11, "per_head")) return NULL;
  if (as_ptr(a[0], &qkv) || as_i64(a[1], &T) || as_i64(a[2], &ld) || as_i32(a[3], &hq) ||
      as_i32(a[4], &hkv) || as_i32(a[5], &d) || as_ptr(a[6], &gq) || as_ptr(a[7], &gk) ||
      as_f32(a[8], &eps) || as_i32(a[9], &dt) || as_ptr(a[10], &st))
    return NULL;
  return PyLong_FromLong(qknorm_per_head(qkv, T, ld, hq, hkv, d, gq, gk, eps, dt, st));
}

/* layerwise(qkv, T, ld, wq, wk, gamma_q, gamma_k, eps, nshards, dtype, stream) -> int */
static PyObject* f_layerwise(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *qkv, *gq, *gk, *st;
  int64_t T, ld, wq, wk;
  int32_t ns, dt;
  float eps;
  if (!nargs_ok(n, 11, "layerwise")) return NULL;
  if (as_ptr(a[0], &qkv) || as_i64(a[1], &T) || as_i64(a[2], &ld) || as_i64(a[3], &wq) ||
      as_i64(a[4], &wk) || as_ptr(a[5], &gq) || as_ptr(a[6], &gk) || as_f32(a[7], &eps) ||
      as_i32(a[8], &ns) || as_i32(a[9], &dt) || as_ptr(a[10], &st))
    return NULL;
  return PyLong_FromLong(qknorm_layerwise(qkv, T, ld, wq, wk, gq, gk, eps, ns, dt, st));
}

/* partial_sumsq(qkv, T, ld, wq, wk, nshards, part_q, part_k, dtype, stream) -> int */
static PyObject* f_partial_sumsq(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *qkv, *pq, *pk, *st;
  int64_t T, ld, wq, wk;
  int32_t ns, dt;
  if (!nargs_ok(n, 10, "partial_sumsq")) return NULL;
  if (as_ptr(a[0], &qkv) || as_i64(a[1], &T) || as_i64(a[2], &ld) || as_i64(a[3], &wq) ||
      as_i64(a[4], &wk) || as_i32(a[5], &ns) || as_ptr(a[6], &pq) || as_ptr(a[7], &pk) ||
      as_i32(a[8], &dt) || as_ptr(a[9], &st))
    return NULL;
  return PyLong_FromLong(qknorm_partial_sumsq(qkv, T, ld, wq, wk, ns, (float*)pq, (float*)pk, dt, st));
}

/* apply_scalar(qkv, T, ld, wq, wk, part_q, part_k, nparts, norm_wq, norm_wk, gamma_q, gamma_k,
 *              eps, dtype, stream) -> int */
static PyObject* f_apply_scalar(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *qkv, *pq, *pk, *gq, *gk, *st;
  int64_t T, ld, wq, wk, nwq, nwk;
  int32_t np, dt;
  float eps;
  if (!nargs_ok(n, 15, "apply_scalar")) return NULL;
  if (as_ptr(a[0], &qkv) || as_i64(a[1], &T) || as_i64(a[2], &ld) || as_i64(a[3], &wq) ||
      as_i64(a[4], &wk) || as_ptr(a[5], &pq) || as_ptr(a[6], &pk) || as_i32(a[7], &np) ||
      as_i64(a[8], &nwq) || as_i64(a[9], &nwk) || as_ptr(a[10], &gq) || as_ptr(a[11], &gk) ||
      as_f32(a[12], &eps) || as_i32(a[13], &dt) || as_ptr(a[14], &st))
    return NULL;
  return PyLong_FromLong(qknorm_apply_scalar(qkv, T, ld, wq, wk, (const float*)pq, (const float*)pk,
                                             np, nwq, nwk, gq, gk, eps, dt, st));
}

/* qkv_proj_per_head(x, ldx, w, ldw, qkv, ld, T, hidden, hq, hkv, head_dim, gamma_q, gamma_k, eps,
 *                   flags, dtype, stream) -> int */
static PyObject* f_qkv_proj_per_head(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *x, *w, *qkv, *gq, *gk, *st;
  int64_t ldx, ldw, ld, T, hidden;
  int32_t hq, hkv, d, fl, dt;
  float eps;
  if (!nargs_ok(n, 17, "qkv_proj_per_head")) return NULL;
  if (as_ptr(a[0], &x) || as_i64(a[1], &ldx) || as_ptr(a[2], &w) || as_i64(a[3], &ldw) ||
      as_ptr(a[4], &qkv) || as_i64(a[5], &ld) || as_i64(a[6], &T) || as_i64(a[7], &hidden) ||
      as_i32(a[8], &hq) || as_i32(a[9], &hkv) || as_i32(a[10], &d) || as_ptr(a[11], &gq) ||
      as_ptr(a[12], &gk) || as_f32(a[13], &eps) || as_i32(a[14], &fl) || as_i32(a[15], &dt) ||
      as_ptr(a[16], &st))
    return NULL;
  return PyLong_FromLong(
      qknorm_qkv_proj_per_head(x, ldx, w, ldw, qkv, ld, T, hidden, hq, hkv, d, gq, gk, eps, fl, dt, st));
}

/* qkv_proj_per_head_noalloc: the arguments of qkv_proj_per_head -> int */
static PyObject* f_qkv_proj_per_head_noalloc(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *x, *w, *qkv, *gq, *gk, *st;
  int64_t ldx, ldw, ld, T, hidden;
  int32_t hq, hkv, d, fl, dt;
  float eps;
  if (!nargs_ok(n, 17, "qkv_proj_per_head_noalloc")) return NULL;
  if (as_ptr(a[0], &x) || as_i64(a[1], &ldx) || as_ptr(a[2], &w) || as_i64(a[3], &ldw) ||
      as_ptr(a[4], &qkv) || as_i64(a[5], &ld) || as_i64(a[6], &T) || as_i64(a[7], &hidden) ||
      as_i32(a[8], &hq) || as_i32(a[9], &hkv) || as_i32(a[10], &d) || as_ptr(a[11], &gq) ||
      as_ptr(a[12], &gk) || as_f32(a[13], &eps) || as_i32(a[14], &fl) || as_i32(a[15], &dt) ||
      as_ptr(a[16], &st))
    return NULL;
  return PyLong_FromLong(qknorm_qkv_proj_per_head_noalloc(x, ldx, w, ldw, qkv, ld, T, hidden, hq, hkv,
                                                          d, gq, gk, eps, fl, dt, st));
}

/* qkv_proj_per_head_ws(x, ldx, w, ldw, qkv, ld, T, hidden, hq, hkv, head_dim, gamma_q, gamma_k,
 *                      eps, flags, dtype, workspace, workspace_bytes, stream) -> int */
static PyObject* f_qkv_proj_per_head_ws(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *x, *w, *qkv, *gq, *gk, *ws, *st;
  int64_t ldx, ldw, ld, T, hidden, wsb;
  int32_t hq, hkv, d, fl, dt;
  float eps;
  if (!nargs_ok(n, 19, "qkv_proj_per_head_ws")) return NULL;
  if (as_ptr(a[0], &x) || as_i64(a[1], &ldx) || as_ptr(a[2], &w) || as_i64(a[3], &ldw) ||
      as_ptr(a[4], &qkv) || as_i64(a[5], &ld) || as_i64(a[6], &T) || as_i64(a[7], &hidden) ||
      as_i32(a[8], &hq) || as_i32(a[9], &hkv) || as_i32(a[10], &d) || as_ptr(a[11], &gq) ||
      as_ptr(a[12], &gk) || as_f32(a[13], &eps) || as_i32(a[14], &fl) || as_i32(a[15], &dt) ||
      as_ptr(a[16], &ws) || as_i64(a[17], &wsb) || as_ptr(a[18], &st))
    return NULL;
  return PyLong_FromLong(qknorm_qkv_proj_per_head_ws(x, ldx, w, ldw, qkv, ld, T, hidden, hq, hkv, d, gq,
                                                     gk, eps, fl, dt, ws, wsb, st));
}

/* quant_rows(x, ldx, q, ldq, scale_p, T, width, dt, st) -> int */
static PyObject* f_quant_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *x, *q, *scale_p, *st;
  int64_t ldx, ldq, T, width;
  int32_t dt;
  if (!nargs_ok(n, 9, "quant_rows")) return NULL;
  if (as_ptr(a[0], &x) ||
      as_i64(a[1], &ldx) ||
      as_ptr(a[2], &q) ||
      as_i64(a[3], &ldq) ||
      as_ptr(a[4], &scale_p) ||
      as_i64(a[5], &T) ||
      as_i64(a[6], &width) ||
      as_i32(a[7], &dt) ||
      as_ptr(a[8], &st))
    return NULL;
  return PyLong_FromLong(qknorm_quant_rows(x, ldx, q, ldq, (float*)scale_p, T, width, dt, st));
}

/* qkv_proj_quant(x, ldx, x_scale, w, ldw, w_scale, qkv, ld, T, hidden, hq, hkv, d, gq, gk, eps, fl, dt, ws, wsb, st) -> int */
static PyObject* f_qkv_proj_quant(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *x, *x_scale, *w, *w_scale, *qkv, *gq, *gk, *ws, *st;
  int64_t ldx, ldw, ld, T, hidden, wsb;
  int32_t hq, hkv, d, fl, dt;
  float eps;
  if (!nargs_ok(n, 21, "qkv_proj_quant")) return NULL;
  if (as_ptr(a[0], &x) ||
      as_i64(a[1], &ldx) ||
      as_ptr(a[2], &x_scale) ||
      as_ptr(a[3], &w) ||
      as_i64(a[4], &ldw) ||
      as_ptr(a[5], &w_scale) ||
      as_ptr(a[6], &qkv) ||
      as_i64(a[7], &ld) ||
      as_i64(a[8], &T) ||
      as_i64(a[9], &hidden) ||
      as_i32(a[10], &hq) ||
      as_i32(a[11], &hkv) ||
      as_i32(a[12], &d) ||
      as_ptr(a[13], &gq) ||
      as_ptr(a[14], &gk) ||
      as_f32(a[15], &eps) ||
      as_i32(a[16], &fl) ||
      as_i32(a[17], &dt) ||
      as_ptr(a[18], &ws) ||
      as_i64(a[19], &wsb) ||
      as_ptr(a[20], &st))
    return NULL;
  return PyLong_FromLong(qknorm_qkv_proj_quant(x, ldx, (const float*)x_scale, w, ldw, (const float*)w_scale, qkv, ld, T, hidden, hq, hkv, d, gq, gk, eps, fl, dt, ws, wsb, st));
}

/* kv_append(qkv, T, ld, hq, hkv, d, cache, pages, stride, slots, dt, st) -> int */
static PyObject* f_kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *qkv, *cache, *slots, *st;
  int64_t T, ld, pages, stride;
  int32_t hq, hkv, d, dt;
  if (!nargs_ok(n, 12, "kv_append")) return NULL;
  if (as_ptr(a[0], &qkv) ||
      as_i64(a[1], &T) ||
      as_i64(a[2], &ld) ||
      as_i32(a[3], &hq) ||
      as_i32(a[4], &hkv) ||
      as_i32(a[5], &d) ||
      as_ptr(a[6], &cache) ||
      as_i64(a[7], &pages) ||
      as_i64(a[8], &stride) ||
      as_ptr(a[9], &slots) ||
      as_i32(a[10], &dt) ||
      as_ptr(a[11], &st))
    return NULL;
  return PyLong_FromLong(qknorm_kv_append(qkv, T, ld, hq, hkv, d, cache, pages, stride, (const int64_t*)slots, dt, st));
}

/* kv_gather(cache, pages, stride, slots, T, hkv, d, k, ldk, v, ldv, dt, st) -> int */
static PyObject* f_kv_gather(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *cache, *slots, *k, *v, *st;
  int64_t pages, stride, T, ldk, ldv;
  int32_t hkv, d, dt;
  if (!nargs_ok(n, 13, "kv_gather")) return NULL;
  if (as_ptr(a[0], &cache) ||
      as_i64(a[1], &pages) ||
      as_i64(a[2], &stride) ||
      as_ptr(a[3], &slots) ||
      as_i64(a[4], &T) ||
      as_i32(a[5], &hkv) ||
      as_i32(a[6], &d) ||
      as_ptr(a[7], &k) ||
      as_i64(a[8], &ldk) ||
      as_ptr(a[9], &v) ||
      as_i64(a[10], &ldv) ||
      as_i32(a[11], &dt) ||
      as_ptr(a[12], &st))
    return NULL;
  return PyLong_FromLong(qknorm_kv_gather(cache, pages, stride, (const int64_t*)slots, T, hkv, d, k, ldk, v, ldv, dt, st));
}

/* kv_attention(qkv, T, ld, cache, pages, stride, table, ldt, width, lens, starts, B, out, ldo, lse, hq, hkv, d, scale, window, dt, ws, wsb, st) -> int */
static PyObject* f_kv_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *qkv, *cache, *table, *lens, *starts, *out, *lse, *ws, *st;
  int64_t T, ld, pages, stride, ldt, width, B, ldo, wsb;
  int32_t hq, hkv, d, window, dt;
  float scale;
  if (!nargs_ok(n, 24, "kv_attention")) return NULL;
  if (as_ptr(a[0], &qkv) ||
      as_i64(a[1], &T) ||
      as_i64(a[2], &ld) ||
      as_ptr(a[3], &cache) ||
      as_i64(a[4], &pages) ||
      as_i64(a[5], &stride) ||
      as_ptr(a[6], &table) ||
      as_i64(a[7], &ldt) ||
      as_i64(a[8], &width) ||
      as_ptr(a[9], &lens) ||
      as_ptr(a[10], &starts) ||
      as_i64(a[11], &B) ||
      as_ptr(a[12], &out) ||
      as_i64(a[13], &ldo) ||
      as_ptr(a[14], &lse) ||
      as_i32(a[15], &hq) ||
      as_i32(a[16], &hkv) ||
      as_i32(a[17], &d) ||
      as_f32(a[18], &scale) ||
      as_i32(a[19], &window) ||
      as_i32(a[20], &dt) ||
      as_ptr(a[21], &ws) ||
      as_i64(a[22], &wsb) ||
      as_ptr(a[23], &st))
    return NULL;
  return PyLong_FromLong(qknorm_kv_attention(qkv, T, ld, cache, pages, stride, (const int32_t*)table, ldt, width, (const int32_t*)lens, (const int32_t*)starts, B, out, ldo, (float*)lse, hq, hkv, d, scale, window, dt, ws, wsb, st));
}

/* ------------------------------------------------------------------------
 * The common case of the binding's marshalling, on torch tensors: qkv a
 * contiguous [T, ...] GPU torch.Tensor (T > 0; not a subclass) of a dtype the
 * library takes, gamma None or a contiguous torch.Tensor on the same GPU in
 * the dtype that goes with qkv's.  The same facts the Python binding reads
 * (device, dtype, contiguity, rows, data pointer), read from the tensor's
 * C++ object.  Anything else returns None, and the binding's Python path
 * handles it (views with a row pitch, and every error, with its message).
 * `setup` hands over torch's current-raw-stream function and the
 * torch.Tensor type. */

static PyObject* g_tensor;          /* torch.Tensor: only that exact type takes the C++ path */
static PyObject* g_raw_stream;      /* torch._C._cuda_getCurrentRawStream; set last, so that
                                       its presence means the rest is ready */

static PyObject* f_setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 2, "setup")) return NULL;
  if (!PyType_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "setup(raw_stream, tensor_type)");
    return NULL;
  }
  Py_XSETREF(g_tensor, Py_NewRef(a[1]));
  Py_XSETREF(g_raw_stream, Py_NewRef(a[0]));
  Py_RETURN_NONE;
}

/* The tensor inside o when o is exactly a torch.Tensor, else NULL. */
static const at::Tensor* tensor_of(PyObject* o) {
  if ((PyObject*)Py_TYPE(o) != g_tensor) return NULL;
  return &THPVariable_Unpack(o);
}

/* The library's dtype code of a tensor, or -1 for another dtype. */
static int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case c10::ScalarType::Float: return QKNORM_F32;
    case c10::ScalarType::BFloat16: return QKNORM_BF16;
    case c10::ScalarType::Half: return QKNORM_F16;
    case c10::ScalarType::Float8_e4m3fn: return QKNORM_FP8_E4M3;
    default: return -1;
  }
}

/* qkv: 1 and (T, ld, dev, ptr, code) for the common case, 0 otherwise */
static int qkv_rows(PyObject* o, int64_t* T, int64_t* ld, int64_t* dev, void** ptr, int* code) {
  const at::Tensor* t = tensor_of(o);
  if (!t || !t->is_cuda() || (*code = dtype_code(*t)) < 0 || !t->is_contiguous() || t->dim() < 2) return 0;
  *T = t->size(0);
  if (*T <= 0) return 0;
  *ld = t->numel() / *T;
  *dev = t->get_device();
  *ptr = t->data_ptr();
  return 1;
}

/* gamma: 1 and its pointer (NULL for None) for the common case, 0 otherwise;
 * the dtype that goes with qkv's is its own, bf16 for FP8 */
static int gamma_ptr(PyObject* g, int code, int64_t dev, void** ptr) {
  if (g == Py_None) {
    *ptr = NULL;
    return 1;
  }
  const at::Tensor* t = tensor_of(g);
  const int want = code == QKNORM_FP8_E4M3 ? QKNORM_BF16 : code;
  if (!t || dtype_code(*t) != want || !t->is_contiguous() || !t->is_cuda() || t->get_device() != dev)
    return 0;
  *ptr = t->data_ptr();
  return 1;
}

/* the stream handle: torch's current raw stream on `dev` for None, else
 * `stream.cuda_stream` or the int itself */
static int stream_ptr(PyObject* s, int64_t dev, void** out) {
  PyObject* v;
  if (s == Py_None) {
    PyObject* d = PyLong_FromLongLong(dev);
    if (!d) return -1;
    v = PyObject_CallOneArg(g_raw_stream, d);
    Py_DECREF(d);
  } else if (PyLong_Check(s)) {
    v = Py_NewRef(s);
  } else {
    v = PyObject_GetAttrString(s, "cuda_stream");
  }
  if (!v) return -1;
  const int r = as_ptr(v, out);
  Py_DECREF(v);
  return r;
}

/* per_head_t(qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, stream) -> int or None */
static PyObject* f_per_head_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 8, "per_head_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t T, ld, dev;
  void *qkv, *gq, *gk, *st;
  int code;
  int32_t hq, hkv, d;
  float eps;
  if (!qkv_rows(a[0], &T, &ld, &dev, &qkv, &code) || !gamma_ptr(a[4], code, dev, &gq) ||
      !gamma_ptr(a[5], code, dev, &gk))
    Py_RETURN_NONE;
  if (as_i32(a[1], &hq) || as_i32(a[2], &hkv) || as_i32(a[3], &d) || as_f32(a[6], &eps) ||
      stream_ptr(a[7], dev, &st))
    return NULL;
  return PyLong_FromLong(qknorm_per_head(qkv, T, ld, hq, hkv, d, gq, gk, eps, code, st));
}

/* layerwise_t(qkv, wq, wk, gamma_q, gamma_k, eps, nshards, stream) -> int or None */
static PyObject* f_layerwise_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 8, "layerwise_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t T, ld, dev, wq, wk;
  void *qkv, *gq, *gk, *st;
  int code;
  int32_t ns;
  float eps;
  if (!qkv_rows(a[0], &T, &ld, &dev, &qkv, &code) || !gamma_ptr(a[3], code, dev, &gq) ||
      !gamma_ptr(a[4], code, dev, &gk))
    Py_RETURN_NONE;
  if (as_i64(a[1], &wq) || as_i64(a[2], &wk) || as_f32(a[5], &eps) || as_i32(a[6], &ns) ||
      stream_ptr(a[7], dev, &st))
    return NULL;
  return PyLong_FromLong(qknorm_layerwise(qkv, T, ld, wq, wk, gq, gk, eps, ns, code, st));
}

/* ---- the 8-bit and 4-bit operators on torch tensors (common case) --------
 * Each reads what the binding's Python path would and returns None for
 * anything it would not take as it is: that path then answers, with its
 * messages. */

/* a GPU tensor on dev (dev < 0: any, which becomes dev) */
static const at::Tensor* gpu_tensor(PyObject* o, int64_t* dev) {
  const at::Tensor* t = tensor_of(o);
  if (!t || !t->is_cuda()) return NULL;
  if (*dev < 0) *dev = t->get_device();
  return t->get_device() == *dev ? t : NULL;
}

/* whether dev is the current device (kernels are launched there) */
static int is_current(int64_t dev) {
  return c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index() == dev;
}

/* [T, ...] with packed rows: 1 and (T, row width, pitch, ptr), 0 otherwise */
static int rows_of(PyObject* o, int64_t* dev, const at::Tensor** tensor, int64_t* T, int64_t* width, int64_t* ld,
                   void** ptr) {
  const at::Tensor* t = gpu_tensor(o, dev);
  if (!t || t->dim() < 2) return 0;
  *T = t->size(0);
  if (*T <= 0) return 0;
  int64_t row = 1;
  for (int64_t i = t->dim() - 1; i > 0; --i) {
    if (t->size(i) != 1 && t->stride(i) != row) return 0;
    row *= t->size(i);
  }
  *width = row;
  *ld = *T > 1 || t->stride(0) > row ? t->stride(0) : row;
  *ptr = t->data_ptr();
  *tensor = t;
  return 1;
}

/* a contiguous tensor of n values (n < 0: any number) of a type */
static int vector_of(PyObject* o, int64_t* dev, c10::ScalarType type, int64_t n, void** ptr) {
  const at::Tensor* t = gpu_tensor(o, dev);
  if (!t || t->scalar_type() != type || !t->is_contiguous() || (n >= 0 && t->numel() != n)) return 0;
  *ptr = t->data_ptr();
  return 1;
}

/* None or a contiguous tensor, as bytes (none: NULL) */
static int space_of(PyObject* o, int64_t* dev, void** ptr, int64_t* bytes) {
  *ptr = NULL;
  *bytes = 0;
  if (o == Py_None) return 1;
  const at::Tensor* t = gpu_tensor(o, dev);
  if (!t || !t->is_contiguous()) return 0;
  *bytes = t->numel() * (int64_t)t->element_size();
  if (*bytes) *ptr = t->data_ptr();
  return 1;
}

/* whether gamma is of no use, None, or n values */
static int values_or_none(PyObject* o, int unused, int64_t n) {
  if (unused || o == Py_None) return 1;
  const at::Tensor* t = tensor_of(o);
  return t && t->numel() == n;
}

/* quant_rows_t(x, q, scale, stream) -> int or None */
static PyObject* f_quant_rows_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 4, "quant_rows_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t dev = -1, T, w, ldx, Tq, wq, ldq;
  void *x, *q, *sc, *st;
  const at::Tensor *tx, *tq;
  if (!rows_of(a[0], &dev, &tx, &T, &w, &ldx, &x) || !rows_of(a[1], &dev, &tq, &Tq, &wq, &ldq, &q) || tx->dim() != 2 ||
      tq->dim() != 2 || tq->scalar_type() != c10::ScalarType::Char || Tq != T || wq != w ||
      !vector_of(a[2], &dev, c10::ScalarType::Float, T, &sc) || !is_current(dev))
    Py_RETURN_NONE;
  const int code = dtype_code(*tx);
  if (code < 0) Py_RETURN_NONE;
  if (stream_ptr(a[3], dev, &st)) return NULL;
  return PyLong_FromLong(qknorm_quant_rows(x, ldx, q, ldq, (float*)sc, T, w, code, st));
}

/* qkv_proj_quant_t(x, x_scale, w, w_scale, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, plain, workspace, stream) */
static PyObject* f_qkv_proj_quant_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 14, "qkv_proj_quant_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t dev = -1, T, K, ldx, N, Kw, ldw, To, wo, ldo, bytes;
  void *x, *xs, *w, *ws, *out, *gq = NULL, *gk = NULL, *work, *st;
  const at::Tensor *to, *tx, *tw;
  int32_t hq, hkv, d;
  float eps;
  if (!rows_of(a[4], &dev, &to, &To, &wo, &ldo, &out) || !rows_of(a[0], &dev, &tx, &T, &K, &ldx, &x) ||
      !rows_of(a[2], &dev, &tw, &N, &Kw, &ldw, &w) || to->dim() != 2 || tx->dim() != 2 || tw->dim() != 2 ||
      tx->scalar_type() != c10::ScalarType::Char || tw->scalar_type() != c10::ScalarType::Char || To != T || Kw != K ||
      !vector_of(a[1], &dev, c10::ScalarType::Float, T, &xs) || !vector_of(a[3], &dev, c10::ScalarType::Float, N, &ws) ||
      !space_of(a[12], &dev, &work, &bytes) || (a[11] != Py_True && a[11] != Py_False) || !is_current(dev))
    Py_RETURN_NONE;
  const int code = dtype_code(*to), plain = a[11] == Py_True;
  if (code < 0 || (!plain && (!gamma_ptr(a[8], code, dev, &gq) || !gamma_ptr(a[9], code, dev, &gk)))) Py_RETURN_NONE;
  if (as_i32(a[5], &hq) || as_i32(a[6], &hkv) || as_i32(a[7], &d) || as_f32(a[10], &eps)) return NULL;
  if (N != ((int64_t)hq + 2 * (int64_t)hkv) * d || wo < N || !values_or_none(a[8], plain, d) ||
      !values_or_none(a[9], plain, d))
    Py_RETURN_NONE;
  if (stream_ptr(a[13], dev, &st)) return NULL;
  return PyLong_FromLong(qknorm_qkv_proj_quant(x, ldx, (const float*)xs, w, ldw, (const float*)ws, out, ldo, T, K, hq, hkv, d,
                                               gq, gk, eps, plain ? QKNORM_PROJ_PLAIN : 0, code, work, bytes, st));
}

/* the cache: uint8 [pages, ...] of pages of hkv heads of d */
static int cache_of(PyObject* o, int64_t* dev, int32_t hkv, int32_t d, int64_t* pages, int64_t* stride, void** ptr) {
  const at::Tensor* t;
  int64_t w;
  return rows_of(o, dev, &t, pages, &w, stride, ptr) && t->scalar_type() == c10::ScalarType::Byte &&
         w == (int64_t)hkv * (64 * (int64_t)d + 256);
}

/* kv_append_t(qkv, hq, hkv, head_dim, cache, slots, stream) -> int or None */
static PyObject* f_kv_append_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 7, "kv_append_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t dev = -1, T, w, ld, pages, stride;
  void *qkv, *cache, *slots, *st;
  const at::Tensor* t;
  int32_t hq, hkv, d;
  if (as_i32(a[1], &hq) || as_i32(a[2], &hkv) || as_i32(a[3], &d)) return NULL;
  if (!rows_of(a[0], &dev, &t, &T, &w, &ld, &qkv) || dtype_code(*t) < 0 ||
      w < ((int64_t)hq + 2 * (int64_t)hkv) * d || !cache_of(a[4], &dev, hkv, d, &pages, &stride, &cache) ||
      !vector_of(a[5], &dev, c10::ScalarType::Long, T, &slots) || !is_current(dev))
    Py_RETURN_NONE;
  const int code = dtype_code(*t);
  if (stream_ptr(a[6], dev, &st)) return NULL;
  return PyLong_FromLong(qknorm_kv_append(qkv, T, ld, hq, hkv, d, cache, pages, stride, (const int64_t*)slots, code, st));
}

/* kv_gather_t(cache, slots, k, v, hkv, head_dim, stream) -> int or None */
static PyObject* f_kv_gather_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 7, "kv_gather_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t dev = -1, T, wk, ldk, Tv, wv, ldv, pages, stride;
  void *cache, *slots, *k, *v, *st;
  const at::Tensor *tk, *tv;
  int32_t hkv, d;
  if (as_i32(a[4], &hkv) || as_i32(a[5], &d)) return NULL;
  if (!cache_of(a[0], &dev, hkv, d, &pages, &stride, &cache) || !rows_of(a[2], &dev, &tk, &T, &wk, &ldk, &k) ||
      !rows_of(a[3], &dev, &tv, &Tv, &wv, &ldv, &v) || Tv != T || wk != (int64_t)hkv * d || wv != wk ||
      tk->scalar_type() != tv->scalar_type() || dtype_code(*tk) < 0 ||
      !vector_of(a[1], &dev, c10::ScalarType::Long, T, &slots) || !is_current(dev))
    Py_RETURN_NONE;
  const int code = dtype_code(*tk);
  if (stream_ptr(a[6], dev, &st)) return NULL;
  return PyLong_FromLong(
      qknorm_kv_gather(cache, pages, stride, (const int64_t*)slots, T, hkv, d, k, ldk, v, ldv, code, st));
}

/* kv_attention_t(qkv, cache, page_table, seq_lens, out, hq, hkv, head_dim, scale, q_starts, window, lse, workspace,
 *                stream) -> int or None */
static PyObject* f_kv_attention_t(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!nargs_ok(n, 14, "kv_attention_t")) return NULL;
  if (!g_raw_stream) Py_RETURN_NONE;
  int64_t dev = -1, T, w, ld, pages, stride, B, wt, ldt, To, wo, ldo, bytes;
  void *qkv, *cache, *table, *lens, *starts = NULL, *out, *lse = NULL, *work, *st;
  const at::Tensor *tq, *tt, *to;
  int32_t hq, hkv, d, window;
  float scale;
  if (as_i32(a[5], &hq) || as_i32(a[6], &hkv) || as_i32(a[7], &d) || as_i32(a[10], &window) || as_f32(a[8], &scale))
    return NULL;
  if (!rows_of(a[0], &dev, &tq, &T, &w, &ld, &qkv) || dtype_code(*tq) < 0 ||
      !cache_of(a[1], &dev, hkv, d, &pages, &stride, &cache) || !rows_of(a[2], &dev, &tt, &B, &wt, &ldt, &table) ||
      tt->dim() != 2 || tt->scalar_type() != c10::ScalarType::Int ||
      !vector_of(a[3], &dev, c10::ScalarType::Int, B, &lens) || !rows_of(a[4], &dev, &to, &To, &wo, &ldo, &out) ||
      To != T || to->scalar_type() != tq->scalar_type() || wo < (int64_t)hq * d || w < (int64_t)hq * d ||
      (a[9] != Py_None && !vector_of(a[9], &dev, c10::ScalarType::Int, B + 1, &starts)) ||
      (a[11] != Py_None && !vector_of(a[11], &dev, c10::ScalarType::Float, T * hq, &lse)) ||
      !space_of(a[12], &dev, &work, &bytes) || !is_current(dev))
    Py_RETURN_NONE;
  const int code = dtype_code(*tq);
  if (stream_ptr(a[13], dev, &st)) return NULL;
  return PyLong_FromLong(qknorm_kv_attention(qkv, T, ld, cache, pages, stride, (const int32_t*)table, ldt, wt,
                                             (const int32_t*)lens, (const int32_t*)starts, B, out, ldo, (float*)lse, hq, hkv,
                                             d, scale, window, code, work, bytes, st));
}

static PyMethodDef kMethods[] = {
    {"setup", (PyCFunction)(void (*)(void))f_setup, METH_FASTCALL,
     "hand over torch's current-raw-stream function and the torch.Tensor type"},
    {"per_head_t", (PyCFunction)(void (*)(void))f_per_head_t, METH_FASTCALL,
     "qknorm_per_head on torch tensors (common case; None: use the Python path)"},
    {"layerwise_t", (PyCFunction)(void (*)(void))f_layerwise_t, METH_FASTCALL,
     "qknorm_layerwise on torch tensors (common case; None: use the Python path)"},
    {"quant_rows_t", (PyCFunction)(void (*)(void))f_quant_rows_t, METH_FASTCALL,
     "qknorm_quant_rows on torch tensors (common case; None: use the Python path)"},
    {"qkv_proj_quant_t", (PyCFunction)(void (*)(void))f_qkv_proj_quant_t, METH_FASTCALL,
     "qknorm_qkv_proj_quant on torch tensors (common case; None: use the Python path)"},
    {"kv_append_t", (PyCFunction)(void (*)(void))f_kv_append_t, METH_FASTCALL,
     "qknorm_kv_append on torch tensors (common case; None: use the Python path)"},
    {"kv_gather_t", (PyCFunction)(void (*)(void))f_kv_gather_t, METH_FASTCALL,
     "qknorm_kv_gather on torch tensors (common case; None: use the Python path)"},
    {"kv_attention_t", (PyCFunction)(void (*)(void))f_kv_attention_t, METH_FASTCALL,
     "qknorm_kv_attention on torch tensors (common case; None: use the Python path)"},
    {"per_head", (PyCFunction)(void (*)(void))f_per_head, METH_FASTCALL, "qknorm_per_head"},
    {"layerwise", (PyCFunction)(void (*)(void))f_layerwise, METH_FASTCALL, "qknorm_layerwise"},
    {"partial_sumsq", (PyCFunction)(void (*)(void))f_partial_sumsq, METH_FASTCALL, "qknorm_partial_sumsq"},
    {"apply_scalar", (PyCFunction)(void (*)(void))f_apply_scalar, METH_FASTCALL, "qknorm_apply_scalar"},
    {"qkv_proj_per_head", (PyCFunction)(void (*)(void))f_qkv_proj_per_head, METH_FASTCALL,
     "qknorm_qkv_proj_per_head"},
    {"qkv_proj_per_head_ws", (PyCFunction)(void (*)(void))f_qkv_proj_per_head_ws, METH_FASTCALL,
     "qknorm_qkv_proj_per_head_ws"},
    {"qkv_proj_per_head_noalloc", (PyCFunction)(void (*)(void))f_qkv_proj_per_head_noalloc,
     METH_FASTCALL, "qknorm_qkv_proj_per_head_noalloc"},
    {"quant_rows", (PyCFunction)(void (*)(void))f_quant_rows, METH_FASTCALL, "qknorm_quant_rows"},
    {"qkv_proj_quant", (PyCFunction)(void (*)(void))f_qkv_proj_quant, METH_FASTCALL, "qknorm_qkv_proj_quant"},
    {"kv_append", (PyCFunction)(void (*)(void))f_kv_append, METH_FASTCALL, "qknorm_kv_append"},
    {"kv_gather", (PyCFunction)(void (*)(void))f_kv_gather, METH_FASTCALL, "qknorm_kv_gather"},
    {"kv_attention", (PyCFunction)(void (*)(void))f_kv_attention, METH_FASTCALL, "qknorm_kv_attention"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_qknorm_fast",
                                     "Direct calls of the QK-Norm C ABI (see qk_norm_amd).", -1,
                                     kMethods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qknorm_fast(void) { return PyModule_Create(&kModule); }

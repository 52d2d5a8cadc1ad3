/* binding.c -- Python calls of the paged-cache entry points.
 *
 * Marshalling only, like the ctypes binding of the other entry points: reads each
 * torch.Tensor's data pointer, dtype, device, shape and strides into a gqa_tensor
 * and calls the library, which does every check.  It is compiled because a decode
 * step makes these calls once per layer, on tensors whose kernels run for a few
 * microseconds: filling a descriptor from Python takes 1.6 us, ten of them longer
 * than the kernel; from here it is about 0.25 us.  No torch header is needed: the
 * attributes are read through the Python objects.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/gqa.h"

static PyTypeObject* g_tensor;         /* torch.Tensor */
static PyObject* g_raw_stream;         /* device index -> cudaStream_t of its current stream */
static PyObject *g_dtypes[8];          /* torch dtypes ... */
static int32_t g_codes[8];             /* ... and their gqa_dtype */
static int g_n_dtypes;
/* The library's entry points, in the order in which setup() gets them. */
static __typeof__(&gqa_paged_append_t) g_append;
static __typeof__(&nvfp4_paged_append_t) g_nvfp4_append;
static __typeof__(&gqa_paged_window_attn_t) g_attn;
static __typeof__(&gqa_paged_norm_append_t) g_norm_append;
static __typeof__(&nvfp4_paged_norm_append_t) g_nvfp4_norm_append;
static __typeof__(&gqa_tree_mask_t) g_tree_mask;
static __typeof__(&gqa_paged_keep_t) g_keep;
static __typeof__(&gqa_paged_tree_attn_t) g_tree_attn;
static void** const g_entries[] = {(void**)&g_append,           (void**)&g_nvfp4_append, (void**)&g_attn, (void**)&g_norm_append,
                                   (void**)&g_nvfp4_norm_append, (void**)&g_tree_mask,    (void**)&g_keep,
                                   (void**)&g_tree_attn};
enum { kEntries = sizeof(g_entries) / sizeof(g_entries[0]) };
/* torch.Tensor's own descriptors, looked up once: methods and attributes */
static PyObject *m_data_ptr, *m_get_device, *m_stride, *a_dtype, *a_shape;

static PyObject* call(PyObject* method, PyObject* t) {
  PyObject* args[2] = {NULL, t};
  return PyObject_Vectorcall(method, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}
static PyObject* get(PyObject* attribute, PyObject* t) {
  return Py_TYPE(attribute)->tp_descr_get(attribute, t, (PyObject*)Py_TYPE(t));
}

static int read_ints(PyObject* tuple, int64_t* out, int n) {
  for (int i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return 0;
}

/* Fills a descriptor; *ref is NULL for None.  -1 with an exception set on failure. */
static int fill(PyObject* t, const char* name, gqa_tensor* d, gqa_tensor** ref) {
  *ref = NULL;
  if (t == Py_None) return 0;
  if (!PyObject_TypeCheck(t, g_tensor)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return -1;
  }
  PyObject *shape = NULL, *stride = NULL, *x = NULL;
  int rc = -1;
  if (!(x = call(m_data_ptr, t))) goto done;
  d->data = PyLong_AsVoidPtr(x);
  if (!d->data && PyErr_Occurred()) goto done;
  Py_CLEAR(x);
  if (!(x = get(a_dtype, t))) goto done;
  d->dtype = 0;
  for (int i = 0; i < g_n_dtypes; ++i)
    if (x == g_dtypes[i]) d->dtype = g_codes[i];
  Py_CLEAR(x);
  if (!(x = call(m_get_device, t))) goto done;
  d->device = (int32_t)PyLong_AsLong(x);
  if (d->device == -1 && PyErr_Occurred()) goto done;
  if (!(shape = get(a_shape, t)) || !(stride = call(m_stride, t))) goto done;
  if (!PyTuple_Check(shape) || !PyTuple_Check(stride) || PyTuple_GET_SIZE(shape) != PyTuple_GET_SIZE(stride)) {
    PyErr_Format(PyExc_TypeError, "%s: shape and strides are not tuples of one length", name);
    goto done;
  }
  if (PyTuple_GET_SIZE(shape) > 6) {
    PyErr_Format(PyExc_ValueError, "%s has more than 6 dimensions", name);
    goto done;
  }
  d->ndim = (int32_t)PyTuple_GET_SIZE(shape);
  if (read_ints(shape, d->shape, d->ndim) || read_ints(stride, d->strides, d->ndim)) goto done;
  *ref = d;
  rc = 0;
done:
  Py_XDECREF(x);
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  return rc;
}

static int fill_all(PyObject* const* args, const char* const* names, int n, gqa_tensor* d, gqa_tensor** refs) {
  for (int i = 0; i < n; ++i)
    if (fill(args[i], names[i], &d[i], &refs[i])) return -1;
  return 0;
}

/* The current stream of a tensor's device (the default stream for host tensors: the
 * library refuses them). */
static int stream_of(const gqa_tensor* t, gqa_stream_t* stream) {
  *stream = NULL;
  if (!t || t->device < 0) return 0;
  PyObject* i = PyLong_FromLong(t->device);
  if (!i) return -1;
  PyObject* s = PyObject_CallOneArg(g_raw_stream, i);
  Py_DECREF(i);
  if (!s) return -1;
  *stream = (gqa_stream_t)PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return PyErr_Occurred() ? -1 : 0;
}

static int expect(Py_ssize_t have, Py_ssize_t want) {
  if (have == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments; expected %zd", have, want);
  return -1;
}

static int as_float(PyObject* x, float* out) {
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)v;
  return 0;
}

static int as_int(PyObject* x, int* out) {
  const long v = PyLong_AsLong(x);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "a number does not fit 32 bits");
    return -1;
  }
  *out = (int)v;
  return 0;
}

/* append(q, k, v, k_pages, v_pages, block_table, kv_lens, qo_indptr, rope, q_out, positions, q_norm, k_norm, interleaved,
 * norm_eps, k_scale, v_scale) -> status */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[13] = {"q",         "k",    "v",     "k_pages",   "v_pages", "block_table", "kv_lens",
                                        "qo_indptr", "rope", "q_out", "positions", "q_norm",  "k_norm"};
  gqa_tensor d[13];
  gqa_tensor* r[13];
  float eps, ks, vs;
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 17) || fill_all(a, names, 13, d, r)) return NULL;
  const int inter = PyObject_IsTrue(a[13]);
  if (inter < 0 || as_float(a[14], &eps) || as_float(a[15], &ks) || as_float(a[16], &vs) || stream_of(r[1], &stream)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  if (r[10] || r[11] || r[12])
    st = g_norm_append(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[10], r[11], r[12], r[9], inter, eps, ks, vs, stream);
  else
    st = g_append(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], inter, ks, vs, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* nvfp4_append(q, k, v, k_fp4, k_sf, v_fp4, v_sf, block_table, qo_indptr, kv_lens, rope, q_out, positions, q_norm, k_norm,
 * interleaved, norm_eps, q_scale) -> status */
static PyObject* py_nvfp4_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[15] = {"q",           "k",         "v",       "k_fp4", "k_sf",  "v_fp4",     "v_sf",
                                        "block_table", "qo_indptr", "kv_lens", "rope",  "q_out", "positions", "q_norm", "k_norm"};
  gqa_tensor d[15];
  gqa_tensor* r[15];
  float eps, qs;
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 18) || fill_all(a, names, 15, d, r)) return NULL;
  const int inter = PyObject_IsTrue(a[15]);
  if (inter < 0 || as_float(a[16], &eps) || as_float(a[17], &qs) || stream_of(r[1], &stream)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  if (r[12] || r[13] || r[14])
    st = g_nvfp4_norm_append(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[12], r[13], r[14], r[11], inter,
                             eps, qs, stream);
  else
    st = g_nvfp4_append(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], inter, qs, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* A workspace tensor's memory; none for NULL.  -1 with an exception set if it is no dense row of bytes. */
static int workspace_of(const gqa_tensor* t, void** ws, int64_t* bytes) {
  *ws = NULL;
  *bytes = 0;
  if (!t) return 0;
  if (t->dtype != GQA_U8 || t->ndim != 1 || (t->shape[0] > 1 && t->strides[0] != 1)) {
    PyErr_SetString(PyExc_ValueError, "workspace must be a dense 1-d uint8 tensor");
    return -1;
  }
  *ws = t->data;
  *bytes = t->shape[0];
  return 0;
}

/* attn(q, k_pages, v_pages, block_table, seq_lens, out, lse, workspace, q_scale, k_scale, v_scale, window, softcap[, sinks]) -> status */
static PyObject* py_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[8] = {"q", "k_pages", "v_pages", "block_table", "seq_lens", "out", "lse", "workspace"};
  gqa_tensor d[8];
  gqa_tensor* r[8];
  float qs, ks, vs, cap;
  int window, sinks = 0;
  gqa_stream_t stream;
  (void)self;
  if ((n != 14 && expect(n, 13)) || fill_all(a, names, 8, d, r)) return NULL;
  if (as_float(a[8], &qs) || as_float(a[9], &ks) || as_float(a[10], &vs) || as_int(a[11], &window) || as_float(a[12], &cap) ||
      (n == 14 && as_int(a[13], &sinks)) || stream_of(r[0], &stream))
    return NULL;
  void* ws;
  int64_t bytes;
  if (workspace_of(r[7], &ws, &bytes)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_attn(r[0], r[1], r[2], r[3], r[4], r[5], r[6], qs, ks, vs, window, sinks, cap, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* tree_mask(parents, qo_indptr, kv_lens, mask, positions, window, sinks) -> status */
static PyObject* py_tree_mask(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[5] = {"parents", "qo_indptr", "kv_lens", "mask", "positions"};
  gqa_tensor d[5];
  gqa_tensor* r[5];
  int window, sinks;
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 7) || fill_all(a, names, 5, d, r)) return NULL;
  if (as_int(a[5], &window) || as_int(a[6], &sinks) || stream_of(r[0], &stream)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_tree_mask(r[0], r[1], r[2], r[3], r[4], window, sinks, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* tree_attn(q, k_pages, v_pages, block_table, qo_indptr, kv_lens, mask, positions, out, lse, workspace, q_scale, k_scale,
 * v_scale, window, sinks, softcap) -> status */
static PyObject* py_tree_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[11] = {"q",    "k_pages",   "v_pages", "block_table", "qo_indptr", "kv_lens",
                                        "mask", "positions", "out",     "lse",         "workspace"};
  gqa_tensor d[11];
  gqa_tensor* r[11];
  float qs, ks, vs, cap;
  int window, sinks;
  gqa_stream_t stream;
  void* ws;
  int64_t bytes;
  (void)self;
  if (expect(n, 17) || fill_all(a, names, 11, d, r)) return NULL;
  if (as_float(a[11], &qs) || as_float(a[12], &ks) || as_float(a[13], &vs) || as_int(a[14], &window) || as_int(a[15], &sinks) ||
      as_float(a[16], &cap) || stream_of(r[0], &stream) || workspace_of(r[10], &ws, &bytes))
    return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_tree_attn(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], qs, ks, vs, window, sinks, cap, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* keep((pages, ...), block_table, qo_indptr, kv_lens, kept, num_kept, new_lens) -> status */
static PyObject* py_keep(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[6] = {"block_table", "qo_indptr", "kv_lens", "kept", "num_kept", "new_lens"};
  static const char* const page_names[4] = {"pages[0]", "pages[1]", "pages[2]", "pages[3]"};
  gqa_tensor d[6], pd[4];
  gqa_tensor *r[6], *pr[4] = {NULL, NULL, NULL, NULL};
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 7)) return NULL;
  if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) > 4) {
    PyErr_SetString(PyExc_TypeError, "pages must be a tuple of up to 4 tensors");
    return NULL;
  }
  const int count = (int)PyTuple_GET_SIZE(a[0]);
  for (int i = 0; i < count; ++i)
    if (fill(PyTuple_GET_ITEM(a[0], i), page_names[i], &pd[i], &pr[i])) return NULL;
  if (fill_all(a + 1, names, 6, d, r) || stream_of(r[2], &stream)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_keep((const gqa_tensor* const*)pr, count, r[0], r[1], r[2], r[3], r[4], r[5], stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* setup(torch.Tensor, current raw stream function, ((dtype, code), ...), (the entry points' addresses)) */
static PyObject* py_setup(PyObject* self, PyObject* args) {
  PyObject *tensor, *stream, *dtypes, *addr;
  (void)self;
  if (!PyArg_ParseTuple(args, "O!OO!O!", &PyType_Type, &tensor, &stream, &PyTuple_Type, &dtypes, &PyTuple_Type, &addr)) return NULL;
  const Py_ssize_t n = PyTuple_GET_SIZE(dtypes);
  if (n > 8 || PyTuple_GET_SIZE(addr) != kEntries) {
    PyErr_Format(PyExc_ValueError, "setup: up to 8 dtypes and %d addresses", (int)kEntries);
    return NULL;
  }
  void* f[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addr, i));
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: a null address");
      return NULL;
    }
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* dt;
    int code;
    if (!PyArg_ParseTuple(PyTuple_GET_ITEM(dtypes, i), "Oi", &dt, &code)) return NULL;
    Py_INCREF(dt);
    g_dtypes[i] = dt;
    g_codes[i] = code;
  }
  g_n_dtypes = (int)n;
  if (!(m_data_ptr = PyObject_GetAttrString(tensor, "data_ptr")) || !(m_get_device = PyObject_GetAttrString(tensor, "get_device")) ||
      !(m_stride = PyObject_GetAttrString(tensor, "stride")) || !(a_dtype = PyObject_GetAttrString(tensor, "dtype")) ||
      !(a_shape = PyObject_GetAttrString(tensor, "shape")))
    return NULL;
  if (!Py_TYPE(a_dtype)->tp_descr_get || !Py_TYPE(a_shape)->tp_descr_get) {
    PyErr_SetString(PyExc_TypeError, "setup: torch.Tensor.dtype and shape are no descriptors");
    return NULL;
  }
  Py_INCREF(tensor);
  g_tensor = (PyTypeObject*)tensor;
  Py_INCREF(stream);
  g_raw_stream = stream;
  for (int i = 0; i < kEntries; ++i) *g_entries[i] = f[i];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
                                {"nvfp4_append", (PyCFunction)(void (*)(void))py_nvfp4_append, METH_FASTCALL, NULL},
                                {"attn", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, NULL},
                                {"tree_mask", (PyCFunction)(void (*)(void))py_tree_mask, METH_FASTCALL, NULL},
                                {"tree_attn", (PyCFunction)(void (*)(void))py_tree_attn, METH_FASTCALL, NULL},
                                {"keep", (PyCFunction)(void (*)(void))py_keep, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  return PyModule_Create(&module);
}

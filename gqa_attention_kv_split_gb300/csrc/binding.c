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
static gqa_status (*g_append)(const gqa_tensor*, const gqa_tensor*, const gqa_tensor*, gqa_tensor*, gqa_tensor*,
                              const gqa_tensor*, const gqa_tensor*, const gqa_tensor*, const gqa_tensor*, gqa_tensor*, int,
                              float, float, gqa_stream_t);
static gqa_status (*g_nvfp4_append)(const gqa_tensor*, const gqa_tensor*, const gqa_tensor*, gqa_tensor*, gqa_tensor*,
                                    gqa_tensor*, gqa_tensor*, const gqa_tensor*, const gqa_tensor*, const gqa_tensor*,
                                    const gqa_tensor*, gqa_tensor*, int, float, gqa_stream_t);
static gqa_status (*g_attn)(const gqa_tensor*, const gqa_tensor*, const gqa_tensor*, const gqa_tensor*, const gqa_tensor*,
                            gqa_tensor*, gqa_tensor*, float, float, float, int, float, void*, int64_t, gqa_stream_t);
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
    PyErr_SetString(PyExc_OverflowError, "window does not fit 32 bits");
    return -1;
  }
  *out = (int)v;
  return 0;
}

/* append(q, k, v, k_pages, v_pages, block_table, kv_lens, qo_indptr, rope, q_out, interleaved, k_scale, v_scale) -> status */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[10] = {"q", "k", "v", "k_pages", "v_pages", "block_table", "kv_lens", "qo_indptr", "rope", "q_out"};
  gqa_tensor d[10];
  gqa_tensor* r[10];
  float ks, vs;
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 13) || fill_all(a, names, 10, d, r)) return NULL;
  const int inter = PyObject_IsTrue(a[10]);
  if (inter < 0 || as_float(a[11], &ks) || as_float(a[12], &vs) || stream_of(r[1], &stream)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_append(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], inter, ks, vs, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* nvfp4_append(q, k, v, k_fp4, k_sf, v_fp4, v_sf, block_table, qo_indptr, kv_lens, rope, q_out, interleaved, q_scale) -> status */
static PyObject* py_nvfp4_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[12] = {"q",           "k",         "v",       "k_fp4", "k_sf", "v_fp4", "v_sf",
                                        "block_table", "qo_indptr", "kv_lens", "rope",  "q_out"};
  gqa_tensor d[12];
  gqa_tensor* r[12];
  float qs;
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 14) || fill_all(a, names, 12, d, r)) return NULL;
  const int inter = PyObject_IsTrue(a[12]);
  if (inter < 0 || as_float(a[13], &qs) || stream_of(r[1], &stream)) return NULL;
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_nvfp4_append(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], inter, qs, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* attn(q, k_pages, v_pages, block_table, seq_lens, out, lse, workspace, q_scale, k_scale, v_scale, window, softcap) -> status */
static PyObject* py_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[8] = {"q", "k_pages", "v_pages", "block_table", "seq_lens", "out", "lse", "workspace"};
  gqa_tensor d[8];
  gqa_tensor* r[8];
  float qs, ks, vs, cap;
  int window;
  gqa_stream_t stream;
  (void)self;
  if (expect(n, 13) || fill_all(a, names, 8, d, r)) return NULL;
  if (as_float(a[8], &qs) || as_float(a[9], &ks) || as_float(a[10], &vs) || as_int(a[11], &window) || as_float(a[12], &cap) ||
      stream_of(r[0], &stream))
    return NULL;
  void* ws = NULL;
  int64_t bytes = 0;
  if (r[7]) {
    if (r[7]->dtype != GQA_U8 || r[7]->ndim != 1 || (r[7]->shape[0] > 1 && r[7]->strides[0] != 1)) {
      PyErr_SetString(PyExc_ValueError, "workspace must be a dense 1-d uint8 tensor");
      return NULL;
    }
    ws = r[7]->data;
    bytes = r[7]->shape[0];
  }
  gqa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_attn(r[0], r[1], r[2], r[3], r[4], r[5], r[6], qs, ks, vs, window, cap, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* setup(torch.Tensor, current raw stream function, ((dtype, code), ...), (three entry points' addresses)) */
static PyObject* py_setup(PyObject* self, PyObject* args) {
  PyObject *tensor, *stream, *dtypes, *addr;
  (void)self;
  if (!PyArg_ParseTuple(args, "O!OO!O!", &PyType_Type, &tensor, &stream, &PyTuple_Type, &dtypes, &PyTuple_Type, &addr)) return NULL;
  const Py_ssize_t n = PyTuple_GET_SIZE(dtypes);
  if (n > 8 || PyTuple_GET_SIZE(addr) != 3) {
    PyErr_SetString(PyExc_ValueError, "setup: up to 8 dtypes and 3 addresses");
    return NULL;
  }
  void* f[3];
  for (int i = 0; i < 3; ++i) {
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
  *(void**)&g_append = f[0];
  *(void**)&g_nvfp4_append = f[1];
  *(void**)&g_attn = f[2];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, NULL},
                                {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
                                {"nvfp4_append", (PyCFunction)(void (*)(void))py_nvfp4_append, METH_FASTCALL, NULL},
                                {"attn", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  return PyModule_Create(&module);
}

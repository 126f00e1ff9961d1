/*
 * _hgcall: a CPython object that holds the marshalled arguments of one
 * hg_gather call (handle, shard and output pointer arrays, row count, stream)
 * and makes the call when invoked.
 *
 * It exists for the host cost per call only. Through ctypes, every call
 * converts five arguments and costs about 1 us of interpreter time on top of
 * the C entry point; a decode loop that issues one gather per step pays that
 * on every step. This object calls the entry point directly from tp_call.
 *
 * It computes nothing: the pointers come from the Python binding, which has
 * already checked the tensors, and the C entry point validates them again.
 * The entry point's address is passed in by the binding (from the loaded
 * libhg), so this module does not link against libhg itself.
 *
 * vocab_embed, vocab_embed_grad, vocab_loss and vocab_loss_grad do the same for
 * the vocabulary operators: they check the tensors, collect their data
 * pointers and call the entry point, and answer its status, or None where a
 * check failed (the binding then says which). In Python the checks and ctypes
 * cost an embedding call of eight shards 14 us on a Grace core, of which the
 * entry point, launch included, takes 3.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <stdlib.h>
#include <string.h>

typedef int (*gather_fn)(void *h, const void *const *shards, void *const *outs, int M,
                         void *stream);

typedef struct {
  PyObject_HEAD
  gather_fn fn;
  PyObject *handle;   /* the binding's Handle: its `ptr` attribute is read at each call */
  const void **shards;
  void **outs;
  int M;
  void *stream;
  PyObject *keep;     /* keeps the tensors behind the pointers alive */
  PyObject *on_error; /* called with the status when the call fails; raises */
} CallObject;

static PyObject *g_ptr_name; /* interned "ptr" */
/* The same for what is asked of a tensor. */
static PyObject *g_is_cuda, *g_dtype, *g_shape, *g_stride, *g_is_contiguous, *g_data_ptr,
    *g_get_device;

static int read_ptrs(PyObject *seq, void ***out, Py_ssize_t *n) {
  PyObject *fast = PySequence_Fast(seq, "pointer list must be a sequence of ints");
  if (!fast) return -1;
  *n = PySequence_Fast_GET_SIZE(fast);
  *out = (void **)calloc((size_t)(*n > 0 ? *n : 1), sizeof(void *));
  if (!*out) {
    Py_DECREF(fast);
    PyErr_NoMemory();
    return -1;
  }
  for (Py_ssize_t i = 0; i < *n; ++i) {
    void *p = PyLong_AsVoidPtr(PySequence_Fast_GET_ITEM(fast, i));
    if (!p && PyErr_Occurred()) {
      Py_DECREF(fast);
      return -1;
    }
    (*out)[i] = p;
  }
  Py_DECREF(fast);
  return 0;
}

static void call_dealloc(CallObject *self) {
  free((void *)self->shards);
  free(self->outs);
  Py_XDECREF(self->handle);
  Py_XDECREF(self->keep);
  Py_XDECREF(self->on_error);
  Py_TYPE(self)->tp_free((PyObject *)self);
}

/* Call(fn_address, handle, shard_ptrs, out_ptrs, M, stream, keep, on_error) */
static PyObject *call_new(PyTypeObject *type, PyObject *args, PyObject *kwds) {
  PyObject *fn_obj, *handle, *shard_seq, *out_seq, *stream_obj, *keep, *on_error;
  int M;
  if (kwds && PyDict_Size(kwds) > 0) {
    PyErr_SetString(PyExc_TypeError, "Call takes positional arguments only");
    return NULL;
  }
  if (!PyArg_ParseTuple(args, "OOOOiOOO", &fn_obj, &handle, &shard_seq, &out_seq, &M,
                        &stream_obj, &keep, &on_error))
    return NULL;
  if (!PyCallable_Check(on_error)) {
    PyErr_SetString(PyExc_TypeError, "on_error must be callable");
    return NULL;
  }
  void *fn = PyLong_AsVoidPtr(fn_obj);
  if (!fn) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address");
    return NULL;
  }
  void *stream = PyLong_AsVoidPtr(stream_obj);
  if (!stream && PyErr_Occurred()) return NULL;
  CallObject *self = (CallObject *)type->tp_alloc(type, 0);
  if (!self) return NULL;
  Py_ssize_t ns = 0, no = 0;
  void **shards = NULL;
  if (read_ptrs(shard_seq, &shards, &ns) != 0 || read_ptrs(out_seq, &self->outs, &no) != 0) {
    free(shards);
    Py_DECREF(self);
    return NULL;
  }
  self->shards = (const void **)shards;
  if (ns != no) {
    Py_DECREF(self);
    PyErr_SetString(PyExc_ValueError, "shard and output lists differ in length");
    return NULL;
  }
  self->fn = (gather_fn)fn;
  self->M = M;
  self->stream = stream;
  Py_INCREF(handle);
  self->handle = handle;
  Py_INCREF(keep);
  self->keep = keep;
  Py_INCREF(on_error);
  self->on_error = on_error;
  return (PyObject *)self;
}

static PyObject *call_call(PyObject *obj, PyObject *args, PyObject *kwds) {
  CallObject *self = (CallObject *)obj;
  if ((args && PyTuple_GET_SIZE(args) != 0) || (kwds && PyDict_Size(kwds) != 0)) {
    PyErr_SetString(PyExc_TypeError, "a gather call takes no arguments");
    return NULL;
  }
  /* A closed handle has ptr 0 (None is taken the same way): pass NULL, which
     the library rejects. */
  PyObject *p = PyObject_GetAttr(self->handle, g_ptr_name);
  if (!p) return NULL;
  void *h = p == Py_None ? NULL : PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  if (!h && PyErr_Occurred()) return NULL;
  const int st = self->fn(h, self->shards, (void *const *)self->outs, self->M, self->stream);
  if (st != 0) {
    PyObject *r = PyObject_CallFunction(self->on_error, "i", st);
    if (!r) return NULL;
    Py_DECREF(r);
    PyErr_Format(PyExc_RuntimeError, "hg_gather failed with status %d", st);
    return NULL;
  }
  Py_RETURN_NONE;
}

/* What the binding's VocabHandle packs into its `desc` (struct module, "Pqqqq"):
 * the handle, the shards, their sizes and their device. */
typedef struct {
  void *h;
  long long tp, cols, hidden, device;
} VocabDesc;

#define MAX_SHARDS 32 /* HG_MAX_TP */

typedef int (*embed_fn)(void *h, const void *tokens, int id_bytes, int N, void *const *table,
                        float scale, void *out, size_t ld, void *stream);
typedef int (*embed_grad_fn)(void *h, const void *tokens, int id_bytes, int N, const void *grad,
                             size_t ld, void *const *table, float scale, int accumulate,
                             void *stream);
typedef int (*loss_fn)(void *h, const void *hidden, size_t ld, void *const *weight,
                       const void *targets, int id_bytes, int N, float scale, void *loss,
                       void *lse, void *stream);
typedef int (*loss_grad_fn)(void *h, const void *hidden, size_t ld, void *const *weight,
                            const void *targets, int id_bytes, const void *lse,
                            const void *grad_loss, int N, float scale, void *grad_hidden,
                            size_t ld_grad, void *const *grad_weight, int accumulate,
                            void *stream);

static void *g_entry[4]; /* the four entry points, in the order above */
static PyObject *g_int32, *g_int64, *g_float32, *g_raw_stream; /* torch's */

/* Checks below: 1: as wanted; 0: not; -1: an exception is set. */

static int is_true_attr(PyObject *t, PyObject *name) {
  PyObject *x = PyObject_GetAttr(t, name);
  if (!x) return -1;
  Py_DECREF(x);
  return x == Py_True;
}

static int is_true_call(PyObject *t, PyObject *name) {
  PyObject *x = PyObject_CallMethodNoArgs(t, name);
  if (!x) return -1;
  Py_DECREF(x);
  return x == Py_True;
}

/* A CUDA tensor of the handle's device: its type, and its data. */
static int cuda_tensor(PyObject *t, const VocabDesc *d, PyObject **dtype, void **ptr) {
  int ok = is_true_attr(t, g_is_cuda);
  if (ok != 1) return ok;
  PyObject *x = PyObject_CallMethodNoArgs(t, g_get_device);
  if (!x) return -1;
  ok = PyLong_AsLongLong(x) == d->device;
  Py_DECREF(x);
  if (PyErr_Occurred()) return -1;
  if (!ok) return 0;
  x = PyObject_GetAttr(t, g_dtype);
  if (!x) return -1;
  Py_DECREF(x); /* torch's types live as long as torch */
  *dtype = x;
  x = PyObject_CallMethodNoArgs(t, g_data_ptr);
  if (!x) return -1;
  *ptr = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return PyErr_Occurred() ? -1 : 1;
}

/* The sizes or strides in tuple `x` (a new reference, released here). */
static int read_sizes(PyObject *x, long long *out, Py_ssize_t n) {
  if (!x) return -1;
  int ok = PyTuple_Check(x) && PyTuple_GET_SIZE(x) == n;
  for (Py_ssize_t i = 0; ok && i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(x, i));
  Py_DECREF(x);
  return PyErr_Occurred() ? -1 : ok;
}

static int shard_list(PyObject *seq, const VocabDesc *d, PyObject *want, void **ptrs) {
  if (!PyList_Check(seq) && !PyTuple_Check(seq)) return 0;
  if (PySequence_Fast_GET_SIZE(seq) != d->tp || d->tp > MAX_SHARDS) return 0;
  for (Py_ssize_t i = 0; i < (Py_ssize_t)d->tp; ++i) {
    PyObject *t = PySequence_Fast_GET_ITEM(seq, i), *dtype = NULL;
    long long size[2];
    int ok = cuda_tensor(t, d, &dtype, &ptrs[i]);
    if (ok == 1) ok = dtype == want;
    if (ok == 1) ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 2);
    if (ok == 1) ok = size[0] == d->cols && size[1] == d->hidden;
    if (ok == 1) ok = is_true_call(t, g_is_contiguous);
    if (ok != 1) return ok;
  }
  return 1;
}

static int id_tensor(PyObject *t, const VocabDesc *d, void **ptr, int *bytes, int *n) {
  PyObject *dtype = NULL;
  long long size[1];
  int ok = cuda_tensor(t, d, &dtype, ptr);
  if (ok == 1) ok = dtype == g_int64 || dtype == g_int32;
  if (ok == 1) ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 1);
  if (ok == 1) ok = size[0] <= 0x7fffffffLL;
  if (ok == 1) ok = is_true_call(t, g_is_contiguous);
  if (ok != 1) return ok;
  *bytes = dtype == g_int64 ? 8 : 4;
  *n = (int)size[0];
  return 1;
}

static int row_tensor(PyObject *t, const VocabDesc *d, PyObject *want, int n, void **ptr,
                      size_t *ld) {
  PyObject *dtype = NULL;
  long long size[2], stride[2];
  int ok = cuda_tensor(t, d, &dtype, ptr);
  if (ok == 1) ok = dtype == want;
  if (ok == 1) ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 2);
  if (ok == 1) ok = size[0] == n && size[1] == d->hidden;
  if (ok == 1) ok = read_sizes(PyObject_CallMethodNoArgs(t, g_stride), stride, 2);
  if (ok == 1) ok = d->hidden == 1 || stride[1] == 1;
  if (ok == 1) ok = n <= 1 || stride[0] >= d->hidden;
  if (ok != 1) return ok;
  *ld = (size_t)(n <= 1 ? d->hidden : stride[0]);
  return 1;
}

static int float_tensor(PyObject *t, const VocabDesc *d, int n, void **ptr) {
  PyObject *dtype = NULL;
  long long size[1];
  int ok = cuda_tensor(t, d, &dtype, ptr);
  if (ok == 1) ok = dtype == g_float32;
  if (ok == 1) ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 1);
  if (ok == 1) ok = size[0] == n;
  if (ok == 1) ok = is_true_call(t, g_is_contiguous);
  return ok;
}

/* The raw stream: an int, or None for the current one of the handle's device. */
static int raw_stream(PyObject *stream, const VocabDesc *d, void **out) {
  PyObject *x = NULL;
  if (stream == Py_None) {
    PyObject *device = PyLong_FromLongLong(d->device);
    if (!device) return -1;
    x = PyObject_CallOneArg(g_raw_stream, device);
    Py_DECREF(device);
  } else {
    x = PyNumber_Long(stream);
  }
  if (!x) return -1;
  *out = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return PyErr_Occurred() ? -1 : 1;
}

/* Arguments that every call starts with: desc, dtype. */
static int read_desc(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, VocabDesc *d) {
  if (n != want || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) != sizeof *d) {
    PyErr_SetString(PyExc_TypeError, "wrong arguments");
    return -1;
  }
  if (!g_entry[0]) {
    PyErr_SetString(PyExc_RuntimeError, "bind_vocab has not been called");
    return -1;
  }
  memcpy(d, PyBytes_AS_STRING(args[0]), sizeof *d);
  return 1;
}

static PyObject *answer(int ok, int status) {
  if (ok < 0) return NULL;
  if (ok == 0) Py_RETURN_NONE;
  return PyLong_FromLong(status);
}

/* vocab_embed(desc, dtype, tokens, table, out, scale, stream) */
static PyObject *vocab_embed(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *ids, *out, *shards[MAX_SHARDS], *stream;
  int bytes = 0, N = 0, st = 0;
  size_t ld = 0;
  int ok = read_desc(a, n, 7, &d);
  if (ok == 1) ok = id_tensor(a[2], &d, &ids, &bytes, &N);
  if (ok == 1) ok = shard_list(a[3], &d, a[1], shards);
  if (ok == 1) ok = row_tensor(a[4], &d, a[1], N, &out, &ld);
  if (ok == 1) ok = raw_stream(a[6], &d, &stream);
  if (ok == 1) {
    const double scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) return NULL;
    st = ((embed_fn)g_entry[0])(d.h, ids, bytes, N, shards, (float)scale, out, ld, stream);
  }
  return answer(ok, st);
}

/* vocab_embed_grad(desc, dtype, tokens, grad_out, grad_table, scale, accumulate, stream) */
static PyObject *vocab_embed_grad(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *ids, *grad, *shards[MAX_SHARDS], *stream;
  int bytes = 0, N = 0, st = 0;
  size_t ld = 0;
  int ok = read_desc(a, n, 8, &d);
  if (ok == 1) ok = id_tensor(a[2], &d, &ids, &bytes, &N);
  if (ok == 1) ok = row_tensor(a[3], &d, a[1], N, &grad, &ld);
  if (ok == 1) ok = shard_list(a[4], &d, a[1], shards);
  if (ok == 1) ok = raw_stream(a[7], &d, &stream);
  if (ok == 1) {
    const double scale = PyFloat_AsDouble(a[5]);
    const int add = PyObject_IsTrue(a[6]);
    if (PyErr_Occurred()) return NULL;
    st = ((embed_grad_fn)g_entry[1])(d.h, ids, bytes, N, grad, ld, shards, (float)scale, add,
                                     stream);
  }
  return answer(ok, st);
}

/* vocab_loss(desc, dtype, hidden, weight, targets, loss, lse, scale, stream) */
static PyObject *vocab_loss(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *hidden, *ids, *loss, *lse, *shards[MAX_SHARDS], *stream;
  int bytes = 0, N = 0, st = 0;
  size_t ld = 0;
  int ok = read_desc(a, n, 9, &d);
  if (ok == 1) ok = id_tensor(a[4], &d, &ids, &bytes, &N);
  if (ok == 1) ok = row_tensor(a[2], &d, a[1], N, &hidden, &ld);
  if (ok == 1) ok = shard_list(a[3], &d, a[1], shards);
  if (ok == 1) ok = float_tensor(a[5], &d, N, &loss);
  if (ok == 1) ok = float_tensor(a[6], &d, N, &lse);
  if (ok == 1) ok = raw_stream(a[8], &d, &stream);
  if (ok == 1) {
    const double scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return NULL;
    st = ((loss_fn)g_entry[2])(d.h, hidden, ld, shards, ids, bytes, N, (float)scale, loss, lse,
                               stream);
  }
  return answer(ok, st);
}

/* vocab_loss_grad(desc, dtype, hidden, weight, targets, lse, grad_loss, grad_hidden or
 * None, grad_weight or None, scale, accumulate, stream) */
static PyObject *vocab_loss_grad(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *hidden, *ids, *lse, *up, *grad = NULL, *shards[MAX_SHARDS], *grads[MAX_SHARDS], *stream;
  int bytes = 0, N = 0, st = 0;
  size_t ld = 0, ld_grad = 0;
  int ok = read_desc(a, n, 12, &d);
  if (ok == 1) ok = id_tensor(a[4], &d, &ids, &bytes, &N);
  if (ok == 1) ok = row_tensor(a[2], &d, a[1], N, &hidden, &ld);
  if (ok == 1) ok = shard_list(a[3], &d, a[1], shards);
  if (ok == 1) ok = float_tensor(a[5], &d, N, &lse);
  if (ok == 1) ok = float_tensor(a[6], &d, N, &up);
  if (ok == 1 && a[7] != Py_None) ok = row_tensor(a[7], &d, a[1], N, &grad, &ld_grad);
  if (ok == 1 && a[8] != Py_None) ok = shard_list(a[8], &d, a[1], grads);
  if (ok == 1) ok = raw_stream(a[11], &d, &stream);
  if (ok == 1) {
    const double scale = PyFloat_AsDouble(a[9]);
    const int add = PyObject_IsTrue(a[10]);
    if (PyErr_Occurred()) return NULL;
    st = ((loss_grad_fn)g_entry[3])(d.h, hidden, ld, shards, ids, bytes, lse, up, N, (float)scale,
                                    grad, ld_grad, a[8] == Py_None ? NULL : grads, add, stream);
  }
  return answer(ok, st);
}

/* bind_vocab(embed, embed_grad, loss, loss_grad addresses, int32, int64, float32,
 * raw stream getter) */
static PyObject *bind_vocab(PyObject *m, PyObject *args) {
  PyObject *p[4], *i32, *i64, *f32, *getter;
  void *entry[4];
  (void)m;
  if (!PyArg_ParseTuple(args, "OOOOOOOO", &p[0], &p[1], &p[2], &p[3], &i32, &i64, &f32, &getter))
    return NULL;
  for (int i = 0; i < 4; ++i) {
    entry[i] = PyLong_AsVoidPtr(p[i]);
    if (!entry[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address");
      return NULL;
    }
  }
  memcpy(g_entry, entry, sizeof entry);
  Py_INCREF(i32);
  Py_XSETREF(g_int32, i32);
  Py_INCREF(i64);
  Py_XSETREF(g_int64, i64);
  Py_INCREF(f32);
  Py_XSETREF(g_float32, f32);
  Py_INCREF(getter);
  Py_XSETREF(g_raw_stream, getter);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef hgcall_methods[] = {
    {"bind_vocab", bind_vocab, METH_VARARGS, NULL},
    FAST(vocab_embed),
    FAST(vocab_embed_grad),
    FAST(vocab_loss),
    FAST(vocab_loss_grad),
    {NULL, NULL, 0, NULL},
};

static PyTypeObject CallType = {
    PyVarObject_HEAD_INIT(NULL, 0)
    .tp_name = "_hgcall.Call",
    .tp_basicsize = sizeof(CallObject),
    .tp_dealloc = (destructor)call_dealloc,
    .tp_call = call_call,
    .tp_flags = Py_TPFLAGS_DEFAULT,
    .tp_doc = "Marshalled arguments of one hg_gather call; calling it makes the call.",
    .tp_new = call_new,
};

static struct PyModuleDef hgcall_module = {
    PyModuleDef_HEAD_INIT, "_hgcall", "Direct hg_gather calls for the Python binding.", -1,
    hgcall_methods, NULL /* slots */, NULL /* traverse */, NULL /* clear */, NULL /* free */,
};

PyMODINIT_FUNC PyInit__hgcall(void) {
  if (PyType_Ready(&CallType) < 0) return NULL;
  g_ptr_name = PyUnicode_InternFromString("ptr");
  g_is_cuda = PyUnicode_InternFromString("is_cuda");
  g_dtype = PyUnicode_InternFromString("dtype");
  g_shape = PyUnicode_InternFromString("shape");
  g_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_stride = PyUnicode_InternFromString("stride");
  g_get_device = PyUnicode_InternFromString("get_device");
  if (!g_ptr_name || !g_is_cuda || !g_dtype || !g_shape || !g_stride || !g_is_contiguous ||
      !g_data_ptr || !g_get_device)
    return NULL;
  PyObject *m = PyModule_Create(&hgcall_module);
  if (!m) return NULL;
  Py_INCREF(&CallType);
  if (PyModule_AddObject(m, "Call", (PyObject *)&CallType) < 0) {
    Py_DECREF(&CallType);
    Py_DECREF(m);
    return NULL;
  }
  return m;
}

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
 *
 * norm_rows, norm_rows_grad, beam_select and beam_reorder do it for the norm and
 * the beam search.
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
    *g_get_device, *g_element_size;

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

/* ---- the norm and the beam search ------------------------------------------- */

/* Their handles' `desc` has the same layout with other sizes in it: for the norm (handle,
 * element type's code, 0, hidden, device), for the beam search (handle, beams, picks,
 * vocab, device). */
typedef int (*norm_rows_fn)(void *h, const void *x, size_t ld_x, const void *residual,
                            size_t ld_residual, void *sum, size_t ld_sum, const void *gain,
                            float eps, int N, void *out, size_t ld_out, int out_type,
                            float *scales, int scale_block, float *rstd, void *stream);
typedef int (*norm_rows_grad_fn)(void *h, const void *s, size_t ld_s, const void *gain,
                                 const float *rstd, const void *grad_out, size_t ld_grad_out,
                                 const void *grad_sum, size_t ld_grad_sum, int N, void *grad_x,
                                 size_t ld_grad_x, void *grad_gain, int accumulate, void *stream);
typedef int (*beam_select_fn)(void *h, const void *logits, size_t ld, const float *lse,
                              size_t lse_stride, const float *scores, const void *finished,
                              int end, int items, void *tokens, void *parents, int id_bytes,
                              float *picked, void *picked_finished, void *stream);
typedef struct { /* hg_beam_state */
  void *data;
  size_t outer, outer_stride, row_stride, pieces, piece_stride, piece_bytes;
} BeamState;
typedef int (*beam_reorder_fn)(void *h, const void *parents, int id_bytes, int items,
                               const BeamState *states, int n_states, void *stream);

static void *g_step_entry[4]; /* the four entry points, in the order above */
static PyObject *g_e4m3, *g_bool, *g_uint8; /* torch's */

#define E4M3_CODE 3     /* HG_E4M3 */
#define MAX_STATES 256  /* HG_MAX_STATES */
#define MAX_DIMS 16

static int read_step_desc(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, VocabDesc *d) {
  if (n != want || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) != sizeof *d) {
    PyErr_SetString(PyExc_TypeError, "wrong arguments");
    return -1;
  }
  if (!g_step_entry[0]) {
    PyErr_SetString(PyExc_RuntimeError, "bind_steps has not been called");
    return -1;
  }
  memcpy(d, PyBytes_AS_STRING(args[0]), sizeof *d);
  return 1;
}

/* The length of a 2-D tensor. */
static int row_count(PyObject *t, int *n) {
  long long size[2];
  int ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 2);
  if (ok == 1) ok = size[0] <= 0x7fffffffLL;
  if (ok == 1) *n = (int)size[0];
  return ok;
}

/* A contiguous [rows, cols] tensor of one of two types (b may be NULL). */
static int table_tensor(PyObject *t, const VocabDesc *d, PyObject *a, PyObject *b, long long rows,
                        long long cols, void **ptr, PyObject **dtype) {
  PyObject *type = NULL;
  long long size[2];
  int ok = cuda_tensor(t, d, &type, ptr);
  if (ok == 1) ok = type == a || (b && type == b);
  if (ok == 1) ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 2);
  if (ok == 1) ok = size[0] == rows && size[1] == cols;
  if (ok == 1) ok = is_true_call(t, g_is_contiguous);
  if (ok == 1 && dtype) *dtype = type;
  return ok;
}

/* A contiguous [n] tensor. */
static int line_tensor(PyObject *t, const VocabDesc *d, PyObject *want, long long n, void **ptr) {
  PyObject *dtype = NULL;
  long long size[1];
  int ok = cuda_tensor(t, d, &dtype, ptr);
  if (ok == 1) ok = dtype == want;
  if (ok == 1) ok = read_sizes(PyObject_GetAttr(t, g_shape), size, 1);
  if (ok == 1) ok = size[0] == n;
  if (ok == 1) ok = is_true_call(t, g_is_contiguous);
  return ok;
}

/* norm_rows(desc, dtype, x, gain, out, residual or None, sum or None, rstd or None,
 * scales or None, eps, stream) */
static PyObject *norm_rows(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *x, *gain, *out, *res = NULL, *sum = NULL, *rstd = NULL, *scales = NULL, *stream;
  size_t ld_x = 0, ld_out = 0, ld_res = 0, ld_sum = 0;
  int N = 0, st = 0, block = 0, type = 0;
  int ok = read_step_desc(a, n, 11, &d);
  if (ok == 1) ok = row_count(a[2], &N);
  if (ok == 1) ok = row_tensor(a[2], &d, a[1], N, &x, &ld_x);
  if (ok == 1) ok = line_tensor(a[3], &d, a[1], d.hidden, &gain);
  if (ok == 1) {
    type = a[8] == Py_None ? (int)d.tp : E4M3_CODE;
    ok = row_tensor(a[4], &d, a[8] == Py_None ? a[1] : g_e4m3, N, &out, &ld_out);
  }
  if (ok == 1 && a[5] != Py_None) ok = row_tensor(a[5], &d, a[1], N, &res, &ld_res);
  if (ok == 1 && a[6] != Py_None) ok = row_tensor(a[6], &d, a[1], N, &sum, &ld_sum);
  if (ok == 1 && a[7] != Py_None) ok = line_tensor(a[7], &d, g_float32, N, &rstd);
  if (ok == 1 && a[8] != Py_None) {
    ok = table_tensor(a[8], &d, g_float32, NULL, N, 1, &scales, NULL);
    if (ok == 0) {
      block = 128;
      ok = table_tensor(a[8], &d, g_float32, NULL, N, (d.hidden + 127) / 128, &scales, NULL);
    }
  }
  if (ok == 1) ok = raw_stream(a[10], &d, &stream);
  if (ok == 1) {
    const double eps = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) return NULL;
    st = ((norm_rows_fn)g_step_entry[0])(d.h, x, ld_x, res, ld_res, sum, ld_sum, gain, (float)eps,
                                         N, out, ld_out, type, scales, block, rstd, stream);
  }
  return answer(ok, st);
}

/* norm_rows_grad(desc, dtype, s, gain, rstd, grad_out, grad_x or None, grad_gain or
 * None, grad_sum or None, accumulate, stream) */
static PyObject *norm_rows_grad(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *s, *gain, *rstd, *up, *grad_x = NULL, *grad_gain = NULL, *more = NULL, *stream;
  size_t ld_s = 0, ld_up = 0, ld_x = 0, ld_more = 0;
  int N = 0, st = 0;
  int ok = read_step_desc(a, n, 11, &d);
  if (ok == 1) ok = row_count(a[2], &N);
  if (ok == 1) ok = row_tensor(a[2], &d, a[1], N, &s, &ld_s);
  if (ok == 1) ok = line_tensor(a[3], &d, a[1], d.hidden, &gain);
  if (ok == 1) ok = line_tensor(a[4], &d, g_float32, N, &rstd);
  if (ok == 1) ok = row_tensor(a[5], &d, a[1], N, &up, &ld_up);
  if (ok == 1 && a[6] != Py_None) ok = row_tensor(a[6], &d, a[1], N, &grad_x, &ld_x);
  if (ok == 1 && a[7] != Py_None) ok = line_tensor(a[7], &d, a[1], d.hidden, &grad_gain);
  if (ok == 1 && a[8] != Py_None) ok = row_tensor(a[8], &d, a[1], N, &more, &ld_more);
  if (ok == 1) ok = raw_stream(a[10], &d, &stream);
  if (ok == 1) {
    const int add = PyObject_IsTrue(a[9]);
    if (PyErr_Occurred()) return NULL;
    st = ((norm_rows_grad_fn)g_step_entry[1])(d.h, s, ld_s, gain, rstd, up, ld_up, more, ld_more,
                                              N, grad_x, ld_x, grad_gain, add, stream);
  }
  return answer(ok, st);
}

/* beam_select(desc, dtype, logits, scores, tokens, parents, picked, lse or None,
 * finished or None, end, picked_finished or None, stream) */
static PyObject *beam_select(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *logits, *scores, *tokens, *parents, *picked, *lse = NULL, *fin = NULL, *fin_out = NULL;
  void *stream;
  size_t ld = 0;
  long long lse_stride = 1;
  PyObject *id_type = NULL;
  int items = 0, st = 0;
  int ok = read_step_desc(a, n, 12, &d);
  if (ok == 1) ok = row_count(a[3], &items);
  if (ok == 1) ok = items * d.tp <= 0x7fffffffLL;
  if (ok == 1) ok = table_tensor(a[3], &d, g_float32, NULL, items, d.tp, &scores, NULL);
  if (ok == 1) ok = row_tensor(a[2], &d, a[1], (int)(items * d.tp), &logits, &ld);
  if (ok == 1) ok = table_tensor(a[4], &d, g_int64, g_int32, items, d.cols, &tokens, &id_type);
  if (ok == 1) ok = table_tensor(a[5], &d, id_type, NULL, items, d.cols, &parents, NULL);
  if (ok == 1) ok = table_tensor(a[6], &d, g_float32, NULL, items, d.cols, &picked, NULL);
  if (ok == 1 && a[7] != Py_None) {
    PyObject *dtype = NULL;
    long long size[1];
    ok = cuda_tensor(a[7], &d, &dtype, &lse);
    if (ok == 1) ok = dtype == g_float32;
    if (ok == 1) ok = read_sizes(PyObject_GetAttr(a[7], g_shape), size, 1);
    if (ok == 1) ok = size[0] == items * d.tp;
    if (ok == 1) ok = read_sizes(PyObject_CallMethodNoArgs(a[7], g_stride), &lse_stride, 1);
    if (ok == 1 && size[0] <= 1) lse_stride = 1;
    if (ok == 1) ok = lse_stride >= 1;
  }
  if (ok == 1 && a[8] != Py_None)
    ok = table_tensor(a[8], &d, g_bool, g_uint8, items, d.tp, &fin, NULL);
  if (ok == 1 && a[10] != Py_None)
    ok = table_tensor(a[10], &d, g_bool, g_uint8, items, d.cols, &fin_out, NULL);
  if (ok == 1) ok = raw_stream(a[11], &d, &stream);
  if (ok == 1) {
    int over = 0;
    const long long end = PyLong_AsLongLongAndOverflow(a[9], &over);
    if (PyErr_Occurred()) return NULL;
    if (over || end < -1 || end >= d.hidden) return answer(0, 0);
    st = ((beam_select_fn)g_step_entry[2])(d.h, logits, ld, lse, (size_t)lse_stride, scores, fin,
                                           (int)end, items, tokens, parents,
                                           id_type == g_int64 ? 8 : 4, picked, fin_out, stream);
  }
  return answer(ok, st);
}

/* A state tensor whose dimension `dim` has `rows` rows, as a record. Its other dimensions,
 * from the longest stride to the shortest and with neighbours that continue one another
 * taken as one, are at most an outer one, pieces and a contiguous run. */
static int state_record(PyObject *t, PyObject *dim_obj, const VocabDesc *d, long long rows,
                        BeamState *out) {
  PyObject *dtype = NULL, *shape;
  long long size[MAX_DIMS], stride[MAX_DIMS], count[MAX_DIMS], step[MAX_DIMS];
  void *ptr;
  int ok = cuda_tensor(t, d, &dtype, &ptr);
  if (ok != 1) return ok;
  shape = PyObject_GetAttr(t, g_shape);
  if (!shape) return -1;
  const Py_ssize_t nd = PyTuple_Check(shape) ? PyTuple_GET_SIZE(shape) : 0;
  if (nd < 1 || nd > MAX_DIMS) {
    Py_DECREF(shape);
    return 0;
  }
  ok = read_sizes(shape, size, nd);
  if (ok == 1) ok = read_sizes(PyObject_CallMethodNoArgs(t, g_stride), stride, nd);
  if (ok != 1) return ok;
  long long dim = 0;
  if (dim_obj) {
    int over = 0;
    dim = PyLong_AsLongLongAndOverflow(dim_obj, &over);
    if (PyErr_Occurred()) return -1;
    if (over) return 0;
  }
  if (dim < 0) dim += nd;
  if (dim < 0 || dim >= nd || size[dim] != rows) return 0;
  PyObject *x = PyObject_CallMethodNoArgs(t, g_element_size);
  if (!x) return -1;
  const long long elem = PyLong_AsLongLong(x);
  Py_DECREF(x);
  if (PyErr_Occurred()) return -1;
  int n = 0;
  memset(out, 0, sizeof *out);
  for (Py_ssize_t i = 0; i < nd; ++i) {
    if (size[i] == 0) return 1; /* nothing in it */
    if (stride[i] < 0) return 0;
    if (i == dim || size[i] == 1) continue;
    int at = n++;
    for (; at > 0 && step[at - 1] < stride[i]; --at) {
      step[at] = step[at - 1];
      count[at] = count[at - 1];
    }
    step[at] = stride[i];
    count[at] = size[i];
  }
  int kept = 0;
  for (int i = 0; i < n; ++i) {
    if (kept > 0 && step[kept - 1] == step[i] * count[i]) {
      step[kept - 1] = step[i];
      count[kept - 1] *= count[i];
    } else {
      step[kept] = step[i];
      count[kept++] = count[i];
    }
  }
  out->data = ptr;
  out->row_stride = (size_t)(stride[dim] * elem);
  out->outer = out->pieces = 1;
  out->piece_bytes = (size_t)elem;
  if (kept > 0 && step[kept - 1] == 1) out->piece_bytes = (size_t)(count[--kept] * elem);
  if (kept > 2) return 0;
  if (kept > 0) {
    --kept;
    out->pieces = (size_t)count[kept];
    out->piece_stride = (size_t)(step[kept] * elem);
  }
  if (kept > 0) {
    out->outer = (size_t)count[0];
    out->outer_stride = (size_t)(step[0] * elem);
  }
  return 1;
}

/* beam_reorder(desc, parents, states, stream): each state a tensor (rows in dimension
 * 0) or a pair of a tensor and the dimension of its rows */
static PyObject *beam_reorder(PyObject *m, PyObject *const *a, Py_ssize_t n) {
  (void)m;
  VocabDesc d;
  void *parents, *stream;
  PyObject *id_type = NULL;
  BeamState states[MAX_STATES];
  int items = 0, st = 0;
  Py_ssize_t count = 0;
  int ok = read_step_desc(a, n, 4, &d);
  if (ok == 1) ok = row_count(a[1], &items);
  if (ok == 1) ok = table_tensor(a[1], &d, g_int64, g_int32, items, d.tp, &parents, &id_type);
  if (ok == 1) ok = PyList_Check(a[2]) || PyTuple_Check(a[2]);
  if (ok == 1) {
    count = PySequence_Fast_GET_SIZE(a[2]);
    ok = count <= MAX_STATES;
  }
  for (Py_ssize_t i = 0; ok == 1 && i < count; ++i) {
    PyObject *t = PySequence_Fast_GET_ITEM(a[2], i), *dim = NULL;
    if (PyTuple_Check(t)) {
      if (PyTuple_GET_SIZE(t) != 2 || !PyLong_Check(PyTuple_GET_ITEM(t, 1))) return answer(0, 0);
      dim = PyTuple_GET_ITEM(t, 1);
      t = PyTuple_GET_ITEM(t, 0);
    }
    if (!PyObject_HasAttr(t, g_is_cuda)) return answer(0, 0);
    ok = state_record(t, dim, &d, items * d.tp, &states[i]);
  }
  if (ok == 1) ok = raw_stream(a[3], &d, &stream);
  if (ok == 1)
    st = ((beam_reorder_fn)g_step_entry[3])(d.h, parents, id_type == g_int64 ? 8 : 4, items,
                                            states, (int)count, stream);
  return answer(ok, st);
}

/* bind_steps(norm_rows, norm_rows_grad, beam_select, beam_reorder addresses, int32, int64,
 * float32, float8_e4m3fn, bool, uint8, raw stream getter) */
static PyObject *bind_steps(PyObject *m, PyObject *args) {
  PyObject *p[4], *type[6], *getter;
  PyObject **const held[6] = {&g_int32, &g_int64, &g_float32, &g_e4m3, &g_bool, &g_uint8};
  void *entry[4];
  (void)m;
  if (!PyArg_ParseTuple(args, "OOOOOOOOOOO", &p[0], &p[1], &p[2], &p[3], &type[0], &type[1],
                        &type[2], &type[3], &type[4], &type[5], &getter))
    return NULL;
  for (int i = 0; i < 4; ++i) {
    entry[i] = PyLong_AsVoidPtr(p[i]);
    if (!entry[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address");
      return NULL;
    }
  }
  memcpy(g_step_entry, entry, sizeof entry);
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(type[i]);
    Py_XSETREF(*held[i], type[i]);
  }
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
    {"bind_steps", bind_steps, METH_VARARGS, NULL},
    FAST(norm_rows),
    FAST(norm_rows_grad),
    FAST(beam_select),
    FAST(beam_reorder),
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
  g_element_size = PyUnicode_InternFromString("element_size");
  if (!g_element_size || !g_ptr_name || !g_is_cuda || !g_dtype || !g_shape || !g_stride || !g_is_contiguous ||
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

/* Argument marshalling of the operators over a caller-owned cache: torch
 * tensors in, the C ABI's pointers, strides and host arrays out. A call's
 * kernels take 2 to 10 microseconds when the work is small; the same
 * marshalling in Python and ctypes took 5 to 7 of a call's 8 to 10 on the host,
 * this one takes about 2.5, 1 of it for the checks of lazy tensors and for
 * autograd's version counters. It knows tensors by their public attributes only
 * (no torch headers). What a tensor can tell is checked here (shape, type,
 * device, strides), the rest by the library; ops.py documents the calls. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "lps.h"

/* ---- what init() is given ------------------------------------------------- */

static PyObject *g_bf16, *g_fp16, *g_int32;             /* torch dtypes */
static PyObject *g_empty, *g_stream, *g_device, *g_set, *g_grad, *g_written; /* torch functions */
static PyObject *g_error;                                /* LpsError */
static PyObject *g_dual;  /* the __dict__ of torch.autograd.forward_ad */
static PyObject *s_level, *s_unpack; /* in it: the current level of forward derivatives (-1: none), unpack_dual */
static PyObject *s_dtype, *s_get_device, *s_data_ptr, *s_shape, *s_stride, *s_requires_grad, *s_device, *s_is_cuda, *s_is_neg;
static PyObject *g_empty_names; /* ("dtype", "device") */

#define MAX_DIM 5

typedef struct {
  PyObject *obj, *dtype; /* borrowed: dtypes live as long as torch */
  int64_t shape[MAX_DIM], stride[MAX_DIM];
  int dim, device, grad;
  void *ptr;
} tensor;

static int ints_of(PyObject *seq, int64_t *out, const char *what) {
  const Py_ssize_t n = PyTuple_Check(seq) ? PyTuple_GET_SIZE(seq) : -1;
  if (n < 0 || n > MAX_DIM) {
    PyErr_Format(PyExc_ValueError, "%s: not a tensor of at most %d axes", what, MAX_DIM);
    return -1;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

static int g_duals; /* the running call: tensors may carry forward derivatives (read once, under the interpreter lock) */

/* Whether `obj` carries a forward derivative, which the calls would lose; -1 on an error. Its requires_grad
 * is false and its memory the primal's, so nothing else tells. */
static int has_tangent(PyObject *obj) {
  if (!g_duals) return 0;
  PyObject *unpack = PyDict_GetItemWithError(g_dual, s_unpack); /* borrowed */
  if (!unpack && !PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "this torch has no forward_ad.unpack_dual");
  PyObject *dual = unpack ? PyObject_CallOneArg(unpack, obj) : NULL, *tangent = dual ? PySequence_GetItem(dual, 1) : NULL;
  const int has = tangent ? tangent != Py_None : -1;
  Py_XDECREF(tangent);
  Py_XDECREF(dual);
  return has;
}

/* The facts of `obj`; strides of axes with one entry are set to dense. */
static int tensor_of(PyObject *obj, tensor *t, const char *what) {
  PyObject *x = PyObject_GetAttr(obj, s_dtype);
  if (!x) goto not_tensor;
  t->obj = obj;
  t->dtype = x;
  Py_DECREF(x);
  if (!(x = PyObject_GetAttr(obj, s_shape))) goto not_tensor;
  t->dim = ints_of(x, t->shape, what);
  Py_DECREF(x);
  if (t->dim < 0) return -1;
  if (!(x = PyObject_CallMethodNoArgs(obj, s_stride))) goto not_tensor;
  const int n = ints_of(x, t->stride, what);
  Py_DECREF(x);
  if (n != t->dim) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: not a strided tensor", what);
    return -1;
  }
  if (!(x = PyObject_CallMethodNoArgs(obj, s_get_device))) goto not_tensor;
  t->device = (int)PyLong_AsLong(x);
  Py_DECREF(x);
  if (!(x = PyObject_GetAttr(obj, s_requires_grad))) goto not_tensor;
  t->grad = x == Py_True;
  Py_DECREF(x);
  if (t->dtype != g_int32) {
    if (!(x = PyObject_CallMethodNoArgs(obj, s_is_neg))) goto not_tensor;
    const int neg = x == Py_True;
    Py_DECREF(x);
    if (neg) { /* a lazy view: its memory holds the values before their sign changes */
      PyErr_Format(PyExc_ValueError, "%s is a negative view: pass its resolve_neg()", what);
      return -1;
    }
  }
  if (!(x = PyObject_CallMethodNoArgs(obj, s_data_ptr))) goto not_tensor;
  t->ptr = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  if (PyErr_Occurred()) return -1;
  const int dual = has_tangent(obj);
  if (dual > 0) PyErr_Format(PyExc_ValueError, "%s carries a forward derivative, and there is none of these operators", what);
  if (dual) return -1;
  int64_t dense = 1;
  for (int i = t->dim - 1; i >= 0; --i) {
    if (t->shape[i] == 1) t->stride[i] = dense;
    dense *= t->shape[i];
  }
  return 0;
not_tensor:
  if (PyErr_ExceptionMatches(PyExc_AttributeError)) PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
  return -1;
}

static int refuse(const char *why) {
  PyErr_SetString(PyExc_ValueError, why);
  return -1;
}

/* The library type that n tensors share, which are on one GPU and need no gradient. */
static int alike(const tensor *t, int n, int *kind) {
  if (t[0].dtype == g_bf16) *kind = LPS_TYPE_BF16;
  else if (t[0].dtype == g_fp16) *kind = LPS_TYPE_FP16;
  else return refuse("tensors must be bfloat16 or float16");
  if (t[0].device < 0) return refuse("tensors must be on a CUDA device");
  int grad = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].dtype != t[0].dtype || t[i].device != t[0].device) return refuse("tensors must share one type and one device");
    grad |= t[i].grad;
  }
  if (grad) {
    PyObject *on = PyObject_CallNoArgs(g_grad);
    if (!on) return -1;
    grad = on == Py_True;
    Py_DECREF(on);
    if (grad) return refuse("there is no backward pass: detach the tensors or call under torch.no_grad()");
  }
  return 0;
}

static int same_shape(const tensor *a, const tensor *b) {
  return a->dim == b->dim && !memcmp(a->shape, b->shape, sizeof(int64_t) * (size_t)a->dim);
}

static int dense(const tensor *t) {
  int64_t d = 1;
  for (int i = t->dim - 1; i >= 0; --i) {
    if (t->shape[i] == 0) return 1;
    if (t->stride[i] != d) return 0;
    d *= t->shape[i];
  }
  return 1;
}

static int int_rows(const tensor *t, int device, int dim, int64_t n0, int64_t n1, const char *what) {
  if (t->dtype != g_int32 || t->device != device || t->dim != dim || t->shape[0] != n0 || (dim > 1 && t->shape[1] != n1) ||
      !dense(t)) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous int32 tensor [batch%s] on the same device", what,
                 dim > 1 ? ", width" : "");
    return -1;
  }
  return 0;
}

/* Sizes go to the library as int. */
static int fits(int64_t x) { return x >= 0 && x <= INT32_MAX; }

/* ---- host integers ----------------------------------------------------------- */

typedef struct {
  int32_t *v;
  int32_t own[260]; /* what most calls need */
  void *heap;
  Py_ssize_t n;
} ints;

static void ints_free(ints *a) { PyMem_Free(a->heap); }

static int ints_room(ints *a, Py_ssize_t n) {
  a->n = n;
  a->v = a->own;
  if (n > (Py_ssize_t)(sizeof a->own / sizeof *a->own)) {
    if (!(a->heap = PyMem_Malloc(sizeof(int32_t) * (size_t)n))) {
      PyErr_NoMemory();
      return -1;
    }
    a->v = a->heap;
  }
  return 0;
}

/* A one-axis array or sequence of integers (n of them where n >= 0) as int32. */
static int ints_from(PyObject *obj, Py_ssize_t n, const char *what, ints *a) {
  Py_buffer b;
  a->heap = NULL;
  if (PyObject_CheckBuffer(obj) && !PyBytes_Check(obj)) {
    if (PyObject_GetBuffer(obj, &b, PyBUF_STRIDED_RO | PyBUF_FORMAT)) return -1;
    const char f = b.format ? b.format[0] : 'B';
    const int wide = f == 'l' || f == 'q', plain = f == 'i' && b.itemsize == 4;
    int rc = -1;
    if (b.ndim != 1 || (n >= 0 && b.shape[0] != n)) {
      if (b.ndim != 1 || n < 0) PyErr_Format(PyExc_ValueError, "%s must hold its values on one axis", what);
      else PyErr_Format(PyExc_ValueError, "%s must hold %zd values, not %zd", what, n, b.shape[0]);
    } else if (b.format && b.format[1] == 0 && (plain || (wide && b.itemsize == 8))) {
      if (!ints_room(a, b.shape[0])) {
        rc = 0;
        for (Py_ssize_t i = 0; i < a->n; ++i) {
          const char *at = (const char *)b.buf + i * b.strides[0];
          int64_t x = 0;
          int32_t y;
          if (plain) {
            memcpy(&y, at, 4);
          } else {
            memcpy(&x, at, 8);
            if (x < INT32_MIN || x > INT32_MAX) {
              PyErr_Format(PyExc_ValueError, "%s must fit 32 bits", what);
              rc = -1;
              break;
            }
            y = (int32_t)x;
          }
          a->v[i] = y;
        }
      }
    } else if (f == 'e' || f == 'f' || f == 'd' || f == 'g' || f == '?' || f == 'Z') {
      PyErr_Format(PyExc_ValueError, "%s must hold integers", what);
    } else {
      PyBuffer_Release(&b);
      goto sequence;
    }
    PyBuffer_Release(&b);
    return rc;
  }
sequence:;
  PyObject *cuda = PyObject_GetAttr(obj, s_is_cuda); /* a tensor: on the host, please */
  if (cuda) {
    const int on = cuda == Py_True;
    Py_DECREF(cuda);
    if (on) {
      PyErr_Format(PyExc_ValueError, "%s must be host integers, not a CUDA tensor", what);
      return -1;
    }
  } else {
    PyErr_Clear();
  }
  PyObject *seq = PySequence_Fast(obj, "host integers must be a sequence");
  if (!seq) return -1;
  const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
  int rc = -1;
  if (n >= 0 && len != n) {
    PyErr_Format(PyExc_ValueError, "%s must hold %zd values, not %zd", what, n, len);
  } else if (!ints_room(a, len)) {
    rc = 0;
    for (Py_ssize_t i = 0; i < len && !rc; ++i) {
      if (i >= PySequence_Fast_GET_SIZE(seq)) { /* an item's __index__ is any code */
        PyErr_Format(PyExc_ValueError, "%s changed while it was read", what);
        rc = -1;
        break;
      }
      PyObject *item = PySequence_Fast_GET_ITEM(seq, i);
      Py_INCREF(item);
      PyObject *x = PyNumber_Index(item);
      Py_DECREF(item);
      int over = 0;
      const long long y = x ? PyLong_AsLongLongAndOverflow(x, &over) : 0;
      Py_XDECREF(x);
      if (!x) {
        PyErr_Clear();
        PyErr_Format(PyExc_ValueError, "%s must hold integers", what);
        rc = -1;
      } else if (over || y < INT32_MIN || y > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s must fit 32 bits", what);
        rc = -1;
      } else {
        a->v[i] = (int32_t)y;
      }
    }
  }
  Py_DECREF(seq);
  return rc;
}

/* ---- the device and its stream -------------------------------------------------- */

typedef struct {
  int device, before; /* before: the device to go back to, or -1 */
  void *stream;
} place;

static int set_device(int device) {
  PyObject *d = PyLong_FromLong(device), *r = d ? PyObject_CallOneArg(g_set, d) : NULL;
  Py_XDECREF(d);
  Py_XDECREF(r);
  return r ? 0 : -1;
}

static int enter(place *p, int device) {
  PyObject *x = PyObject_CallNoArgs(g_device);
  if (!x) return -1;
  const int here = (int)PyLong_AsLong(x);
  Py_DECREF(x);
  p->device = device;
  p->before = -1;
  if (here != device) {
    if (set_device(device)) return -1;
    p->before = here;
  }
  PyObject *d = PyLong_FromLong(device);
  x = d ? PyObject_CallOneArg(g_stream, d) : NULL;
  Py_XDECREF(d);
  if (x) p->stream = PyLong_AsVoidPtr(x);
  Py_XDECREF(x);
  if (!x || PyErr_Occurred()) {
    if (p->before >= 0) {
      PyObject *t, *v, *tb;
      PyErr_Fetch(&t, &v, &tb);
      set_device(p->before);
      PyErr_Restore(t, v, tb);
    }
    return -1;
  }
  return 0;
}

/* Back to the device that was current; the library's refusal as LpsError. */
static int leave(const place *p, int rc) {
  if (rc < 0) {
    PyObject *args = Py_BuildValue("(is)", rc, last_error_string());
    PyObject *e = args ? PyObject_CallObject(g_error, args) : NULL;
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(args);
    Py_XDECREF(e);
  }
  if (p->before >= 0) {
    PyObject *t, *v, *tb;
    PyErr_Fetch(&t, &v, &tb);
    const int back = set_device(p->before);
    if (t) PyErr_Restore(t, v, tb);
    else if (back) return -1;
  }
  return rc < 0 ? -1 : 0;
}

/* The scale as the library takes it, where 0 stands for 1/sqrt(head_dim): a scale
 * that only comes to 0 in 32 bits is refused. */
static int scale_of(PyObject *obj, float *scale) {
  const double x = PyFloat_AsDouble(obj);
  if (PyErr_Occurred()) return -1;
  *scale = (float)x;
  return *scale == 0.f && x != 0. ? refuse("scale must be 0 or a number that 32 bits hold") : 0;
}

/* The output: `out` checked against q, or a new dense tensor like q (a new reference). */
static PyObject *output_like(PyObject *out, const tensor *q, tensor *o) {
  if (out != Py_None) {
    Py_INCREF(out);
    return out;
  }
  PyObject *shape = PyObject_GetAttr(q->obj, s_shape), *device = PyObject_GetAttr(q->obj, s_device);
  if (shape && device) {
    PyObject *const args[3] = {shape, q->dtype, device};
    out = PyObject_Vectorcall(g_empty, args, 1, g_empty_names);
  } else {
    out = NULL;
  }
  Py_XDECREF(shape);
  Py_XDECREF(device);
  if (out && tensor_of(out, o, "out")) Py_CLEAR(out);
  return out;
}

/* Tells autograd that a call that has been enqueued writes `a` (and `b`) in place: an earlier operation that
 * saved one of them for its backward then refuses to run on the new values. */
static int written(PyObject *a, PyObject *b) {
  PyObject *both = b ? PyTuple_Pack(2, a, b) : PyTuple_Pack(1, a), *r = both ? PyObject_CallOneArg(g_written, both) : NULL;
  Py_XDECREF(both);
  Py_XDECREF(r);
  return r ? 0 : -1;
}

static int contiguous_heads(const tensor *t) {
  return t->shape[t->dim - 1] <= 1 || t->stride[t->dim - 1] == 1 ? 0 : refuse("the head dimension must be contiguous");
}

static int argc_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return -1;
}

/* The start of a call on tensors. */
static int begin(Py_ssize_t n, Py_ssize_t want) {
  if (argc_is(n, want)) return -1;
  PyObject *level = PyDict_GetItemWithError(g_dual, s_level);
  g_duals = !(level && PyLong_Check(level) && PyLong_AsLong(level) < 0);
  return PyErr_Occurred() ? -1 : 0;
}

/* A library call without the interpreter lock: a launch waits while the stream's
 * queue is full, and what the queue waits for may need the lock. */
#define UNLOCKED(call)                     \
  __extension__({                          \
    int rc_;                               \
    Py_BEGIN_ALLOW_THREADS rc_ = (call);   \
    Py_END_ALLOW_THREADS rc_;              \
  })

/* ---- the calls --------------------------------------------------------------------- */

/* prompt(q, k, v, offsets, out, scale) -> out */
static PyObject *prompt(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  tensor t[4];
  ints off;
  place at;
  int kind = 0;
  (void)self;
  if (begin(n, 6) || tensor_of(args[0], &t[0], "q") || tensor_of(args[1], &t[1], "k") || tensor_of(args[2], &t[2], "v")) return NULL;
  const tensor *q = &t[0], *k = &t[1];
  if (q->dim != 3 || k->dim != 3) return refuse("q, k and v must be [tokens, heads, head_dim]"), NULL;
  if (k->shape[0] != q->shape[0] || k->shape[2] != q->shape[2] || !same_shape(k, &t[2]))
    return refuse("k and v must be [tokens, kv heads, head_dim] of q's tokens and head_dim"), NULL;
  const int given = args[4] != Py_None;
  if (given) {
    if (tensor_of(args[4], &t[3], "out")) return NULL;
    if (!same_shape(&t[3], q)) return refuse("out must have q's shape"), NULL;
  }
  float scale;
  if (scale_of(args[5], &scale) || alike(t, given ? 4 : 3, &kind)) return NULL;
  for (int i = 0; i < 3 + given; ++i)
    if (contiguous_heads(&t[i])) return NULL;
  if (!fits(q->shape[0]) || !fits(q->shape[1]) || !fits(k->shape[1])) return refuse("tensors are too large"), NULL;
  if (ints_from(args[3], -1, "offsets", &off)) return ints_free(&off), NULL;
  PyObject *out = NULL;
  if (off.n < 1) refuse("offsets must hold n + 1 values");
  else if (off.v[off.n - 1] > q->shape[0]) refuse("offsets reach past the tokens");
  else out = output_like(args[4], q, &t[3]);
  if (out && off.n > 1 && q->shape[0] > 0) {
    const int64_t st[8] = {q->stride[0], q->stride[1], k->stride[0], k->stride[1], t[2].stride[0], t[2].stride[1], t[3].stride[0], t[3].stride[1]};
    if (enter(&at, q->device) ||
        leave(&at, UNLOCKED(attention_prompt_packed(q->ptr, k->ptr, t[2].ptr, t[3].ptr, kind, (int)(off.n - 1), off.v, (int)q->shape[1],
                                           (int)k->shape[1], (int)q->shape[2], st, scale, at.stream))) ||
        (given && written(out, NULL)))
      Py_CLEAR(out);
  }
  ints_free(&off);
  return out;
}

/* tree(q, k_cache, v_cache, parents, pos, rows, out, scale) -> out */
static PyObject *tree(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  tensor t[4], par;
  ints pos, rows;
  place at;
  int kind = 0;
  (void)self;
  if (begin(n, 8) || tensor_of(args[0], &t[0], "q") || tensor_of(args[1], &t[1], "k_cache") ||
      tensor_of(args[2], &t[2], "v_cache") || tensor_of(args[3], &par, "parents"))
    return NULL;
  const tensor *q = &t[0], *kc = &t[1];
  if (q->dim != 4 || kc->dim != 4)
    return refuse("q must be [batch, width, q heads, head_dim], the caches [batch, kv heads, max_ctx, head_dim]"), NULL;
  if (kc->shape[0] != q->shape[0] || kc->shape[3] != q->shape[3] || !same_shape(kc, &t[2]))
    return refuse("the caches must be [batch, kv heads, max_ctx, head_dim] of q's batch and head_dim"), NULL;
  const int given = args[6] != Py_None;
  if (given) {
    if (tensor_of(args[6], &t[3], "out")) return NULL;
    if (!same_shape(&t[3], q)) return refuse("out must have q's shape"), NULL;
  }
  float scale;
  if (scale_of(args[7], &scale) || alike(t, given ? 4 : 3, &kind)) return NULL;
  if (!dense(kc) || !dense(&t[2])) return refuse("the caches must be contiguous [batch, kv heads, max_ctx, head_dim]"), NULL;
  if (contiguous_heads(q) || (given && contiguous_heads(&t[3]))) return NULL;
  const int64_t batch = q->shape[0], width = q->shape[1];
  if (int_rows(&par, q->device, 2, batch, width, "parents")) return NULL;
  if (!fits(batch) || !fits(width) || !fits(q->shape[2]) || !fits(kc->shape[1]) || !fits(kc->shape[2]))
    return refuse("tensors are too large"), NULL;
  rows.heap = NULL;
  PyObject *out = NULL;
  if (!ints_from(args[4], batch, "pos", &pos) && !ints_from(args[5], batch, "rows", &rows) &&
      (out = output_like(args[6], q, &t[3]))) {
    const int64_t st[6] = {q->stride[0], q->stride[1], q->stride[2], t[3].stride[0], t[3].stride[1], t[3].stride[2]};
    if (enter(&at, q->device) ||
        leave(&at, UNLOCKED(attention_tree_verify(q->ptr, kc->ptr, t[2].ptr, t[3].ptr, kind, (int)batch, (int)width, pos.v, rows.v, par.ptr,
                                         (int)q->shape[2], (int)kc->shape[1], (int)q->shape[3], (int)kc->shape[2], st, scale,
                                         at.stream))) ||
        (given && written(out, NULL)))
      Py_CLEAR(out);
  }
  ints_free(&pos);
  ints_free(&rows);
  return out;
}

/* append(k, v, offsets, k_cache, v_cache, start) */
static PyObject *append(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  tensor t[4];
  ints off, start;
  place at;
  int kind = 0;
  (void)self;
  if (begin(n, 6) || tensor_of(args[0], &t[0], "k") || tensor_of(args[1], &t[1], "v") || tensor_of(args[3], &t[2], "k_cache") ||
      tensor_of(args[4], &t[3], "v_cache"))
    return NULL;
  const tensor *k = &t[0], *kc = &t[2];
  if (k->dim != 3 || kc->dim != 4)
    return refuse("k and v must be [tokens, kv heads, head_dim], the caches [sequences, kv heads, max_ctx, head_dim]"), NULL;
  if (!same_shape(&t[1], k) || kc->shape[1] != k->shape[1] || kc->shape[3] != k->shape[2] || !same_shape(&t[3], kc))
    return refuse("k and v, and the two caches, must agree in shape, kv heads and head_dim"), NULL;
  if (alike(t, 4, &kind)) return NULL;
  if (!dense(kc) || !dense(&t[3])) return refuse("the caches must be contiguous [batch, kv heads, max_ctx, head_dim]"), NULL;
  if (contiguous_heads(k) || contiguous_heads(&t[1])) return NULL;
  if (!fits(k->shape[0]) || !fits(k->shape[1]) || !fits(kc->shape[0] + 1) || !fits(kc->shape[2]))
    return refuse("tensors are too large"), NULL;
  start.heap = NULL;
  int ok = 0;
  if (!ints_from(args[2], kc->shape[0] + 1, "offsets", &off) && !ints_from(args[5], kc->shape[0], "start", &start)) {
    if (off.v[kc->shape[0]] > k->shape[0]) {
      refuse("offsets reach past the tokens");
    } else if (k->shape[0] == 0) {
      ok = 1;
    } else {
      const int64_t st[4] = {k->stride[0], k->stride[1], t[1].stride[0], t[1].stride[1]};
      ok = !enter(&at, k->device) &&
           !leave(&at, UNLOCKED(kv_rows_append(k->ptr, t[1].ptr, (int)kc->shape[0], off.v, kc->ptr, t[3].ptr, start.v, (int)k->shape[1],
                                      (int)k->shape[2], (int)kc->shape[2], st, at.stream))) &&
           !written(kc->obj, t[3].obj);
    }
  }
  ints_free(&off);
  ints_free(&start);
  if (!ok) return NULL;
  Py_RETURN_NONE;
}

/* accept(k_cache, v_cache, pos, path, accepted) */
static PyObject *accept(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  tensor t[2], path, taken;
  ints pos;
  place at;
  int kind = 0;
  (void)self;
  if (begin(n, 5) || tensor_of(args[0], &t[0], "k_cache") || tensor_of(args[1], &t[1], "v_cache")) return NULL;
  const tensor *kc = &t[0];
  if ((kc->dim != 4 && kc->dim != 5) || !same_shape(&t[1], kc))
    return refuse("the caches must be [layers, batch, kv heads, max_ctx, head_dim], both alike"), NULL;
  if (alike(t, 2, &kind)) return NULL;
  if (!dense(kc) || !dense(&t[1])) return refuse("the caches must be contiguous [layers, batch, kv heads, max_ctx, head_dim]"), NULL;
  const int64_t *s = kc->shape + kc->dim - 4, layers = kc->dim == 5 ? kc->shape[0] : 1;
  if (tensor_of(args[3], &path, "path") || tensor_of(args[4], &taken, "accepted")) return NULL;
  if (path.dim != 2) return refuse("path must be [batch, width]"), NULL;
  if (int_rows(&path, kc->device, 2, s[0], path.shape[1], "path") || int_rows(&taken, kc->device, 1, s[0], s[0], "accepted")) return NULL;
  if (!fits(layers) || !fits(s[0]) || !fits(s[1]) || !fits(s[2]) || !fits(path.shape[1])) return refuse("tensors are too large"), NULL;
  int ok = 0;
  if (!ints_from(args[2], s[0], "pos", &pos))
    ok = !enter(&at, kc->device) &&
         !leave(&at, UNLOCKED(kv_rows_accept(kc->ptr, t[1].ptr, (int)layers, (int)s[0], (int)s[1], (int)s[3], (int)s[2], pos.v,
                                    (int)path.shape[1], path.ptr, taken.ptr, at.stream))) &&
         !written(kc->obj, t[1].obj);
  ints_free(&pos);
  if (!ok) return NULL;
  Py_RETURN_NONE;
}

/* host_ints(values, count or -1) -> list: how the calls read their host integers, for tests without a GPU. */
static PyObject *host_ints(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  ints a;
  (void)self;
  if (argc_is(n, 2)) return NULL;
  const Py_ssize_t want = PyLong_AsSsize_t(args[1]);
  if (want == -1 && PyErr_Occurred()) return NULL;
  if (ints_from(args[0], want, "values", &a)) return ints_free(&a), NULL;
  PyObject *list = PyList_New(a.n);
  for (Py_ssize_t i = 0; list && i < a.n; ++i) {
    PyObject *x = PyLong_FromLong(a.v[i]);
    if (!x) Py_CLEAR(list);
    else PyList_SET_ITEM(list, i, x);
  }
  ints_free(&a);
  return list;
}

/* init(LpsError, torch): what the calls need of torch, looked up once. */
static PyObject *init(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (argc_is(n, 2)) return NULL;
  PyObject *torch = args[1], *cuda = PyObject_GetAttrString(torch, "cuda"), *c = PyObject_GetAttrString(torch, "_C");
  Py_INCREF(args[0]);
  g_error = args[0];
  g_bf16 = PyObject_GetAttrString(torch, "bfloat16");
  g_fp16 = PyObject_GetAttrString(torch, "float16");
  g_int32 = PyObject_GetAttrString(torch, "int32");
  g_empty = PyObject_GetAttrString(torch, "empty");
  PyObject *dual = PyImport_ImportModule("torch.autograd.forward_ad");
  g_dual = dual ? PyModule_GetDict(dual) : NULL;
  Py_XINCREF(g_dual);
  Py_XDECREF(dual);
  g_grad = PyObject_GetAttrString(torch, "is_grad_enabled");
  /* what torch.autograd.graph.increment_version calls, without its trip through Python */
  g_written = c && PyObject_HasAttrString(c, "_increment_version") ? PyObject_GetAttrString(c, "_increment_version") : NULL;
  if (!g_written) {
    PyObject *graph = PyImport_ImportModule("torch.autograd.graph");
    g_written = graph ? PyObject_GetAttrString(graph, "increment_version") : NULL;
    Py_XDECREF(graph);
  }
  /* the calls' tensors are on a GPU, so torch's lazy initialisation has been */
  g_device = c && PyObject_HasAttrString(c, "_cuda_getDevice") ? PyObject_GetAttrString(c, "_cuda_getDevice")
             : cuda ? PyObject_GetAttrString(cuda, "current_device") : NULL;
  g_set = cuda ? PyObject_GetAttrString(cuda, "set_device") : NULL;
  g_stream = c && PyObject_HasAttrString(c, "_cuda_getCurrentRawStream") ? PyObject_GetAttrString(c, "_cuda_getCurrentRawStream") : NULL;
  Py_XDECREF(cuda);
  Py_XDECREF(c);
  if (!g_stream && !PyErr_Occurred()) { /* a torch without CUDA: every call is refused before it asks for a stream */
    Py_INCREF(Py_None);
    g_stream = Py_None;
  }
  if (!g_bf16 || !g_fp16 || !g_int32 || !g_empty || !g_dual || !g_grad || !g_written || !g_device || !g_set || PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void (*)(void))f
static PyMethodDef methods[] = {{"init", FAST(init), METH_FASTCALL, NULL},     {"prompt", FAST(prompt), METH_FASTCALL, NULL},
                                {"tree", FAST(tree), METH_FASTCALL, NULL},     {"append", FAST(append), METH_FASTCALL, NULL},
                                {"accept", FAST(accept), METH_FASTCALL, NULL}, {"host_ints", FAST(host_ints), METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  s_level = PyUnicode_InternFromString("_current_level");
  s_unpack = PyUnicode_InternFromString("unpack_dual");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_requires_grad = PyUnicode_InternFromString("requires_grad");
  s_device = PyUnicode_InternFromString("device");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_neg = PyUnicode_InternFromString("is_neg");
  g_empty_names = Py_BuildValue("(ss)", "dtype", "device");
  return g_empty_names ? PyModule_Create(&module) : NULL;
}

/*
 * The short way from Python into the serving entry points of libtlq.
 *
 * A serving step makes several of these calls, each of which launches kernels
 * of a few microseconds, so reading the tensors' attributes in the interpreter
 * and passing twenty arguments through ctypes took longer than the kernels.
 * Here the same is done through CPython's C API.  Each function takes what the
 * Python function of its name takes, reads what the tensors say of themselves
 * and calls the library; it returns the library's status, or -1 without having
 * called it when an argument is not as it should be (the Python function then
 * goes through its own checks, which name what is wrong).  Tensors are read
 * through tensors.cpp where that was built for the torch in use, else through
 * their attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "../../include/tlq.h"
#include "tensors.h"

#define FALLBACK (-1)

static PyObject *s_dtype, *s_is_cuda, *s_is_contiguous, *s_data_ptr, *s_numel, *s_shape, *s_stride;
static PyObject *t_f16, *t_f32, *t_i32, *t_i64, *t_u8; /* torch's types */
static PyObject *get_device, *get_stream;              /* torch's current device and its current stream */

static tlq_status (*f_plan)(const int32_t*, const int32_t*, int, int32_t*, int, const int32_t*, int, const int32_t*, int,
                            int64_t, int32_t*, int32_t*, int32_t*, int32_t*, int64_t*, int, int32_t*, void*);
static tlq_status (*f_append)(const tl_kv4_cache*, const uint16_t*, int64_t, const uint16_t*, int64_t, const int64_t*,
                              int, void*);
static tlq_status (*f_read)(const tl_kv4_cache*, const int64_t*, int, uint16_t*, uint16_t*, void*);
static tlq_status (*f_attention)(const tl_kv4_cache*, const uint16_t*, int64_t, int, uint16_t*, int64_t, const int32_t*,
                                 const int32_t*, const int32_t*, int, int, int, int, float, int, void*, size_t, void*);
static tlq_status (*f_lora)(const uint16_t*, int64_t, const uint16_t*, const uint16_t*, const float*, const int32_t*,
                            const int32_t*, int, int, int, int, int, int, int, const uint16_t*, int64_t, uint16_t*,
                            int64_t, void*);

static tlq_status (*f_norm_rope)(const tl_rope*, const int32_t*, const uint16_t*, int64_t, int, const uint16_t*, uint16_t*,
                                 int64_t, const uint16_t*, int64_t, int, const uint16_t*, uint16_t*, int64_t, int, float,
                                 int, void*);
static tlq_status (*f_append_rope)(const tl_kv4_cache*, const tl_rope*, const int32_t*, const uint16_t*, int64_t,
                                   const uint16_t*, const uint16_t*, int64_t, const int64_t*, const uint16_t*, int64_t,
                                   int, const uint16_t*, uint16_t*, int64_t, float, int, void*);
static tlq_status (*f_sample)(const void*, int, int64_t, int, int, const float*, const float*, const int32_t*, const float*,
                              const float*, int32_t*, float*, void*);

static tlq_status (*f_attention_prefix)(const tl_kv4_cache*, const uint16_t*, int64_t, int, uint16_t*, int64_t,
                                        const int32_t*, const int32_t*, const int32_t*, int, const int32_t*,
                                        const int32_t*, int, int, int, int, float, void*, size_t, void*);

/* 1 if attribute `name` of o is `want` (an object compared by identity). */
static int attr_is(PyObject* o, PyObject* name, PyObject* want) {
  PyObject* v = PyObject_GetAttr(o, name);
  Py_XDECREF(v); /* the types and the truth values outlive this */
  return v == want;
}

static int call_long(PyObject* o, PyObject* name, long long* out) {
  PyObject* v = PyObject_CallMethodNoArgs(o, name);
  if (!v) return 0;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return !(*out == -1 && PyErr_Occurred());
}

/* The way past the interpreter, once read_tensors has been called: for torch's
 * own two classes only (a subclass may answer for itself). */
static int (*f_tensor)(PyObject*, tlq_tensor*);
static PyTypeObject *tensor_class, *parameter_class;

static int known(PyObject* t, tlq_tensor* x) {
  return f_tensor && (Py_TYPE(t) == tensor_class || Py_TYPE(t) == parameter_class) && f_tensor(t, x);
}

static int type_of(PyObject* type) {
  return type == t_f16 ? TLQ_TENSOR_F16
         : type == t_f32 ? TLQ_TENSOR_F32
         : type == t_i32 ? TLQ_TENSOR_I32
         : type == t_i64 ? TLQ_TENSOR_I64
                         : TLQ_TENSOR_U8;
}

/* Sizes (s_shape) or strides (s_stride) of a tensor of `dims` dimensions. */
static int extents(PyObject* t, int strides, int dims, long long* out) {
  tlq_tensor x;
  if (known(t, &x)) {
    if (x.dims != dims) return 0;
    memcpy(out, strides ? x.step : x.size, dims * sizeof *out);
    return 1;
  }
  PyObject* v = strides ? PyObject_CallMethodNoArgs(t, s_stride) : PyObject_GetAttr(t, s_shape);
  if (!v || !PyTuple_Check(v) || PyTuple_GET_SIZE(v) != dims) {
    Py_XDECREF(v);
    return 0;
  }
  for (int i = 0; i < dims; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
  Py_DECREF(v);
  return !PyErr_Occurred();
}

static int pointer(PyObject* t, void** p) {
  PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!v) return 0;
  *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

/* A contiguous CUDA tensor of one type; n >= 0: of that many elements, else
 * *n_out takes the number (if asked for). */
static int flat(PyObject* t, PyObject* type, long long n, void** p, long long* n_out) {
  tlq_tensor x;
  if (known(t, &x)) {
    if (x.type != type_of(type) || !x.contiguous || (n >= 0 && x.numel != n)) return 0;
    if (n_out) *n_out = x.numel;
    *p = x.data;
    return 1;
  }
  if (!attr_is(t, s_dtype, type) || !attr_is(t, s_is_cuda, Py_True)) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  Py_XDECREF(c);
  if (c != Py_True) return 0;
  if (n >= 0 || n_out) {
    long long got;
    if (!call_long(t, s_numel, &got) || (n >= 0 && got != n)) return 0;
    if (n_out) *n_out = got;
  }
  return pointer(t, p);
}

/* Rows [tokens, a] (dims = 2) or [tokens, a, b] (dims = 3), contiguous but for
 * the token stride; at least one (whose stride says nothing). */
static int rows(PyObject* t, int dims, long long a, long long b, void** p, int64_t* ld, long long* tokens) {
  tlq_tensor x;
  long long size[3], step[3];
  const int direct = known(t, &x);
  if (direct) {
    if (x.type != TLQ_TENSOR_F16 || x.dims != dims) return 0;
    memcpy(size, x.size, dims * sizeof *size);
    memcpy(step, x.step, dims * sizeof *step);
  } else if (!attr_is(t, s_dtype, t_f16) || !attr_is(t, s_is_cuda, Py_True) || !extents(t, 0, dims, size) ||
             !extents(t, 1, dims, step)) {
    return 0;
  }
  if (size[0] < 1 || size[1] != a || (dims == 3 && (size[2] != b || step[1] != b)) || step[dims - 1] != 1) return 0;
  *ld = size[0] > 1 ? step[0] : (dims == 3 ? a * b : a);
  *tokens = size[0];
  if (direct) {
    *p = x.data;
    return 1;
  }
  return pointer(t, p);
}

static int as_int(PyObject* o, long long* out) {
  if (!PyLong_CheckExact(o)) return 0;
  *out = PyLong_AsLongLong(o);
  return !PyErr_Occurred() && *out <= 0x7fffffffll && *out >= -0x7fffffffll;
}

/* The stream asked for: None (torch's current one) or a handle. */
static int stream_of(PyObject* o, void** s) {
  PyObject* v = NULL;
  if (o == Py_None) {
    PyObject* d = PyObject_CallNoArgs(get_device);
    if (!d) return 0;
    v = PyObject_CallOneArg(get_stream, d);
    Py_DECREF(d);
    if (!v) return 0;
  } else if (PyLong_CheckExact(o)) {
    v = Py_NewRef(o);
  } else {
    return 0;
  }
  *s = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

static PyObject* answer(int status) {
  if (status < 0 && PyErr_Occurred()) PyErr_Clear();
  return PyLong_FromLong(status);
}

/* The library's answer, with the interpreter's lock released over the call: a
 * first launch loads modules, a full queue waits for the GPU, and a callback on
 * the stream may need the interpreter.  The arguments are C values by then. */
#define CALL(f, ...)          \
  do {                        \
    tlq_status st;            \
    Py_BEGIN_ALLOW_THREADS    \
    st = f(__VA_ARGS__);      \
    Py_END_ALLOW_THREADS      \
    return (int)st;           \
  } while (0)

/* The cache's descriptor, by its address. */
static int cache_of(PyObject* o, const tl_kv4_cache** c) {
  *c = (const tl_kv4_cache*)PyLong_AsVoidPtr(o);
  return *c && !PyErr_Occurred();
}

static int plan(PyObject* const* a, Py_ssize_t n) {
  /* cached, added, table, free_pages, q_start, seq_lens, token_req, token_pos, slots, counts, page_size, num_pages,
   * free_head, stream */
  void *cached, *added, *table, *free_pages, *q_start, *lens, *req, *pos, *slots, *counts, *head = NULL, *s;
  long long requests, room, num_free, size[2], page, pages;
  if (n != 14 || !flat(a[0], t_i32, -1, &cached, &requests) || !flat(a[1], t_i32, requests, &added, NULL) ||
      !flat(a[2], t_i32, -1, &table, NULL) || !extents(a[2], 0, 2, size) || size[0] != requests ||
      !flat(a[3], t_i32, -1, &free_pages, &num_free) || !flat(a[4], t_i32, requests + 1, &q_start, NULL) ||
      !flat(a[5], t_i32, requests, &lens, NULL) || !flat(a[8], t_i64, -1, &slots, &room) ||
      !flat(a[6], t_i32, room, &req, NULL) || !flat(a[7], t_i32, room, &pos, NULL) ||
      !flat(a[9], t_i32, 4, &counts, NULL) || !as_int(a[10], &page) || !as_int(a[11], &pages) ||
      (a[12] != Py_None && !flat(a[12], t_i32, 1, &head, NULL)) || !stream_of(a[13], &s) || requests > 0x7fffffffll ||
      room > 0x7fffffffll || num_free > 0x7fffffffll || size[1] > 0x7fffffffll)
    return FALLBACK;
  CALL(f_plan, cached, added, (int)requests, table, (int)size[1], free_pages, (int)num_free, head, (int)page, pages,
       q_start, lens, req, pos, slots, (int)room, counts, s);
}

static int append(PyObject* const* a, Py_ssize_t n) {
  /* cache address, heads, head_dim, k, v, slots, stream */
  const tl_kv4_cache* c;
  void *k, *v, *slots, *s;
  int64_t ldk, ldv;
  long long heads, dim, tokens, nv;
  if (n != 7 || !cache_of(a[0], &c) || !as_int(a[1], &heads) || !as_int(a[2], &dim) ||
      !rows(a[3], 3, heads, dim, &k, &ldk, &tokens) || !rows(a[4], 3, heads, dim, &v, &ldv, &nv) || nv != tokens ||
      !flat(a[5], t_i64, tokens, &slots, NULL) || !stream_of(a[6], &s) || tokens > 0x7fffffffll)
    return FALLBACK;
  CALL(f_append, c, k, ldk, v, ldv, slots, (int)tokens, s);
}

static int read_back(PyObject* const* a, Py_ssize_t n) {
  /* cache address, heads, head_dim, slots, k, v, stream */
  const tl_kv4_cache* c;
  void *k, *v, *slots, *s;
  int64_t ldk, ldv;
  long long heads, dim, tokens, nv;
  if (n != 7 || !cache_of(a[0], &c) || !as_int(a[1], &heads) || !as_int(a[2], &dim) ||
      !rows(a[4], 3, heads, dim, &k, &ldk, &tokens) || !rows(a[5], 3, heads, dim, &v, &ldv, &nv) || nv != tokens ||
      ldk != heads * dim || ldv != heads * dim || !flat(a[3], t_i64, tokens, &slots, NULL) || !stream_of(a[6], &s) ||
      tokens > 0x7fffffffll)
    return FALLBACK;
  CALL(f_read, c, slots, (int)tokens, k, v, s);
}

static int attention(PyObject* const* a, Py_ssize_t n) {
  /* cache address, head_dim, q, out, q_start, seq_lens, table, max_q, scale, window, workspace, stream */
  const tl_kv4_cache* c;
  void *q, *out, *q_start, *lens, *table, *ws, *s;
  int64_t ldq, ldo;
  long long dim, tokens, no, requests, max_q, window, bytes, qs[3], size[2];
  if (n != 12 || !cache_of(a[0], &c) || !as_int(a[1], &dim) || !extents(a[2], 0, 3, qs) ||
      !rows(a[2], 3, qs[1], dim, &q, &ldq, &tokens) || !rows(a[3], 3, qs[1], dim, &out, &ldo, &no) || no != tokens ||
      !flat(a[5], t_i32, -1, &lens, &requests) || !flat(a[4], t_i32, requests + 1, &q_start, NULL) ||
      !flat(a[6], t_i32, -1, &table, NULL) || !extents(a[6], 0, 2, size) || size[0] != requests ||
      !as_int(a[7], &max_q) || !PyFloat_CheckExact(a[8]) || !as_int(a[9], &window) ||
      !flat(a[10], t_u8, -1, &ws, &bytes) || !stream_of(a[11], &s) || tokens > 0x7fffffffll ||
      requests > 0x7fffffffll || size[1] > 0x7fffffffll || qs[1] > 0x7fffffffll)
    return FALLBACK;
  const float scale = (float)PyFloat_AS_DOUBLE(a[8]);
  CALL(f_attention, c, q, ldq, (int)qs[1], out, ldo, q_start, lens, table, (int)size[1], (int)requests, (int)tokens,
       (int)max_q, scale, (int)window, ws, (size_t)bytes, s);
}

static int lora(PyObject* const* a, Py_ssize_t n) {
  /* x, A, B, scales, q_start, adapters, max_q, y, out, stream */
  void *x, *A, *B, *scales, *q_start, *adapters, *y, *out, *s;
  int64_t ldx, ldy, ldo;
  long long sa[3], sb[3], tokens, ny, no, requests, max_q;
  if (n != 10 || !flat(a[1], t_f16, -1, &A, NULL) || !extents(a[1], 0, 3, sa) || !flat(a[2], t_f16, -1, &B, NULL) ||
      !extents(a[2], 0, 3, sb) || sa[0] != sb[0] || sa[1] != sb[2] || !rows(a[0], 2, sa[2], 0, &x, &ldx, &tokens) ||
      !rows(a[7], 2, sb[1], 0, &y, &ldy, &ny) || !rows(a[8], 2, sb[1], 0, &out, &ldo, &no) || ny != tokens ||
      no != tokens || !flat(a[3], t_f32, sa[0], &scales, NULL) || !flat(a[5], t_i32, -1, &adapters, &requests) ||
      !flat(a[4], t_i32, requests + 1, &q_start, NULL) || !as_int(a[6], &max_q) || !stream_of(a[9], &s) ||
      tokens > 0x7fffffffll || requests > 0x7fffffffll || sa[0] > 0x7fffffffll || sa[2] > 0x7fffffffll ||
      sb[1] > 0x7fffffffll)
    return FALLBACK;
  CALL(f_lora, x, ldx, A, B, scales, q_start, adapters, (int)requests, (int)tokens, (int)max_q, (int)sa[2], (int)sb[1],
       (int)sa[1], (int)sa[0], y, ldy, out, ldo, s);
}

/* As flat(), with None for NULL. */
static int flat_or_none(PyObject* t, PyObject* type, long long n, void** p) {
  *p = NULL;
  return t == Py_None || flat(t, type, n, p, NULL);
}

/* Heads [tokens, heads, dim] (None: none) with their output (out NULL: they have
 * none) and weight; *tokens is checked, or filled in where it is negative. */
typedef struct {
  void *x, *out, *weight;
  int64_t ld, ldo;
  long long heads;
} head_rows;
static int heads_of(PyObject* x, PyObject* out, PyObject* weight, long long dim, long long* tokens, head_rows* r) {
  long long size[3], n;
  memset(r, 0, sizeof *r);
  if (x == Py_None) return 1;
  if (!extents(x, 0, 3, size) || !rows(x, 3, size[1], dim, &r->x, &r->ld, &n) || (*tokens >= 0 && n != *tokens) ||
      size[1] > 0x7fffffffll || !flat_or_none(weight, t_f16, dim, &r->weight))
    return 0;
  *tokens = n;
  r->heads = size[1];
  if (!out) return 1;
  return rows(out, 3, size[1], dim, &r->out, &r->ldo, &n) && n == *tokens;
}

/* The rope's descriptor by its address, and its positions [axes, tokens] (of one
 * axis: that many of any shape); None: neither. */
static int rope_of(PyObject* address, PyObject* axes, PyObject* positions, long long tokens, const tl_rope** r, void** p) {
  long long n, size[2];
  *r = NULL;
  *p = NULL;
  if (address == Py_None) return 1;
  *r = (const tl_rope*)PyLong_AsVoidPtr(address);
  return *r && !PyErr_Occurred() && as_int(axes, &n) && flat(positions, t_i32, n * tokens, p, NULL) &&
         (n == 1 || (extents(positions, 0, 2, size) && size[0] == n));
}

static int norm_rope(PyObject* const* a, Py_ssize_t n) {
  /* rope address, axes, q, k, positions, q_out, k_out, q_weight, k_weight, eps, stream */
  const tl_rope* rope;
  void *positions, *s;
  long long size[3], tokens = -1;
  head_rows q, k;
  if (n != 11 || (a[2] == Py_None && a[3] == Py_None) || !extents(a[2] != Py_None ? a[2] : a[3], 0, 3, size) ||
      !heads_of(a[2], a[5], a[7], size[2], &tokens, &q) || !heads_of(a[3], a[6], a[8], size[2], &tokens, &k) ||
      !rope_of(a[0], a[1], a[4], tokens, &rope, &positions) || !PyFloat_CheckExact(a[9]) || !stream_of(a[10], &s) ||
      tokens > 0x7fffffffll || size[2] > 0x7fffffffll)
    return FALLBACK;
  const float eps = (float)PyFloat_AS_DOUBLE(a[9]);
  CALL(f_norm_rope, rope, positions, q.x, q.ld, (int)q.heads, q.weight, q.out, q.ldo, k.x, k.ld, (int)k.heads, k.weight,
       k.out, k.ldo, (int)size[2], eps, (int)tokens, s);
}

static int append_rope(PyObject* const* a, Py_ssize_t n) {
  /* cache address, heads, head_dim, rope address, axes, k, v, positions, slots, k_weight, q, q_out, q_weight, eps,
   * stream */
  const tl_kv4_cache* c;
  const tl_rope* rope;
  void *positions, *slots, *s;
  long long heads, dim, tokens = -1;
  head_rows q, k, v;
  if (n != 15 || !cache_of(a[0], &c) || !as_int(a[1], &heads) || !as_int(a[2], &dim) ||
      !heads_of(a[5], NULL, a[9], dim, &tokens, &k) || k.heads != heads ||
      !heads_of(a[6], NULL, Py_None, dim, &tokens, &v) || v.heads != heads ||
      !heads_of(a[10], a[11], a[12], dim, &tokens, &q) || !flat(a[8], t_i64, tokens, &slots, NULL) ||
      !rope_of(a[3], a[4], a[7], tokens, &rope, &positions) || !PyFloat_CheckExact(a[13]) || !stream_of(a[14], &s) ||
      tokens > 0x7fffffffll)
    return FALLBACK;
  const float eps = (float)PyFloat_AS_DOUBLE(a[13]);
  CALL(f_append_rope, c, rope, positions, k.x, k.ld, k.weight, v.x, v.ld, slots, q.x, q.ld, (int)q.heads, q.weight, q.out,
       q.ldo, eps, (int)tokens, s);
}

static int attention_prefix(PyObject* const* a, Py_ssize_t n) {
  /* cache address, head_dim, q, out, q_start, seq_lens, table, prefix_len, prefix_table, max_q, scale, workspace,
   * stream */
  const tl_kv4_cache* c;
  void *q, *out, *q_start, *lens, *table, *prefix_len, *prefix_table, *ws, *s;
  int64_t ldq, ldo;
  long long dim, tokens, no, requests, max_q, pages, bytes, qs[3], size[2];
  if (n != 13 || !cache_of(a[0], &c) || !as_int(a[1], &dim) || !extents(a[2], 0, 3, qs) ||
      !rows(a[2], 3, qs[1], dim, &q, &ldq, &tokens) || !rows(a[3], 3, qs[1], dim, &out, &ldo, &no) || no != tokens ||
      !flat(a[5], t_i32, -1, &lens, &requests) || !flat(a[4], t_i32, requests + 1, &q_start, NULL) ||
      !flat(a[6], t_i32, -1, &table, NULL) || !extents(a[6], 0, 2, size) || size[0] != requests ||
      !flat(a[7], t_i32, 1, &prefix_len, NULL) || !flat(a[8], t_i32, -1, &prefix_table, &pages) ||
      !as_int(a[9], &max_q) || !PyFloat_CheckExact(a[10]) || !flat(a[11], t_u8, -1, &ws, &bytes) ||
      !stream_of(a[12], &s) || tokens > 0x7fffffffll || requests > 0x7fffffffll || size[1] > 0x7fffffffll ||
      pages > 0x7fffffffll || qs[1] > 0x7fffffffll)
    return FALLBACK;
  const float scale = (float)PyFloat_AS_DOUBLE(a[10]);
  CALL(f_attention_prefix, c, q, ldq, (int)qs[1], out, ldo, q_start, lens, table, (int)size[1], prefix_len, prefix_table,
       (int)pages, (int)requests, (int)tokens, (int)max_q, scale, ws, (size_t)bytes, s);
}

static int sample(PyObject* const* a, Py_ssize_t n) {
  /* logits, uniform, tokens, temperature, top_k, top_p, min_p, logprobs, stream */
  void *x, *uniform, *tokens, *temperature, *top_k, *top_p, *min_p, *logprobs, *s;
  long long size[2], step[2];
  tlq_tensor logits;
  if (n != 9 || !extents(a[0], 0, 2, size) || !extents(a[0], 1, 2, step) || size[0] < 1 || step[1] != 1)
    return FALLBACK;
  if (known(a[0], &logits)) {
    x = logits.data;
  } else {
    if (!attr_is(a[0], s_is_cuda, Py_True) || !pointer(a[0], &x)) return FALLBACK;
    logits.type = attr_is(a[0], s_dtype, t_f16) ? TLQ_TENSOR_F16 : attr_is(a[0], s_dtype, t_f32) ? TLQ_TENSOR_F32 : 0;
  }
  const int half = logits.type == TLQ_TENSOR_F16;
  if ((!half && logits.type != TLQ_TENSOR_F32) || !flat(a[1], t_f32, size[0], &uniform, NULL) ||
      !flat(a[2], t_i32, size[0], &tokens, NULL) || !flat_or_none(a[3], t_f32, size[0], &temperature) ||
      !flat_or_none(a[4], t_i32, size[0], &top_k) || !flat_or_none(a[5], t_f32, size[0], &top_p) ||
      !flat_or_none(a[6], t_f32, size[0], &min_p) || !flat_or_none(a[7], t_f32, size[0], &logprobs) ||
      !stream_of(a[8], &s) || size[0] > 0x7fffffffll || size[1] > 0x7fffffffll)
    return FALLBACK;
  CALL(f_sample, x, half, size[0] > 1 ? step[0] : size[1], (int)size[0], (int)size[1], uniform, temperature, top_k, top_p,
       min_p, tokens, logprobs, s);
}

#define METHOD(name)                                                              \
  static PyObject* py_##name(PyObject* self, PyObject* const* a, Py_ssize_t n) { \
    (void)self;                                                                   \
    return answer(name(a, n));                                                    \
  }
METHOD(plan)
METHOD(append)
METHOD(read_back)
METHOD(attention)
METHOD(lora)
METHOD(norm_rope)
METHOD(append_rope)
METHOD(sample)
METHOD(attention_prefix)

/* bind(float16, float32, int32, int64, uint8, get_device, get_stream, and the
 * addresses of the five entry points in the order above) */
static PyObject* bind(PyObject* self, PyObject* args) {
  PyObject *o[7], *f[5];
  (void)self;
  if (!PyArg_ParseTuple(args, "OOOOOOOOOOOO", &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &o[6], &f[0], &f[1], &f[2],
                        &f[3], &f[4]))
    return NULL;
  t_f16 = Py_NewRef(o[0]);
  t_f32 = Py_NewRef(o[1]);
  t_i32 = Py_NewRef(o[2]);
  t_i64 = Py_NewRef(o[3]);
  t_u8 = Py_NewRef(o[4]);
  get_device = Py_NewRef(o[5]);
  get_stream = Py_NewRef(o[6]);
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(f[i]);
    if (!p[i] || PyErr_Occurred()) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
      return NULL;
    }
  }
  *(void**)&f_plan = p[0];
  *(void**)&f_append = p[1];
  *(void**)&f_read = p[2];
  *(void**)&f_attention = p[3];
  *(void**)&f_lora = p[4];
  Py_RETURN_NONE;
}

/* bind_step(addresses of tl_qk_norm_rope, tl_kv4_append_rope, tl_sample, tl_kv4_attention_prefix) */
static PyObject* bind_step(PyObject* self, PyObject* args) {
  PyObject* f[4];
  void* p[4];
  (void)self;
  if (!PyArg_ParseTuple(args, "OOOO", &f[0], &f[1], &f[2], &f[3])) return NULL;
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(f[i]);
    if (!p[i] || PyErr_Occurred()) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
      return NULL;
    }
  }
  *(void**)&f_norm_rope = p[0];
  *(void**)&f_append_rope = p[1];
  *(void**)&f_sample = p[2];
  *(void**)&f_attention_prefix = p[3];
  Py_RETURN_NONE;
}

/* read_tensors(the address of tlq_tensor_read, torch.Tensor, torch.nn.Parameter) */
static PyObject* read_tensors(PyObject* self, PyObject* args) {
  PyObject *f, *tensor, *parameter;
  (void)self;
  if (!PyArg_ParseTuple(args, "OO!O!", &f, &PyType_Type, &tensor, &PyType_Type, &parameter)) return NULL;
  void* p = PyLong_AsVoidPtr(f);
  if (PyErr_Occurred()) return NULL;
  tensor_class = (PyTypeObject*)Py_NewRef(tensor);
  parameter_class = (PyTypeObject*)Py_NewRef(parameter);
  *(void**)&f_tensor = p;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "Torch's types and the library's entry points; once."},
    {"plan", (PyCFunction)(void (*)(void))py_plan, METH_FASTCALL, "tl_kv_plan"},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, "tl_kv4_append"},
    {"read", (PyCFunction)(void (*)(void))py_read_back, METH_FASTCALL, "tl_kv4_read"},
    {"attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, "tl_kv4_attention"},
    {"lora", (PyCFunction)(void (*)(void))py_lora, METH_FASTCALL, "tl_lora_add"},
    {"bind_step", bind_step, METH_VARARGS, "The entry points of a step's other calls; once, after bind."},
    {"read_tensors", read_tensors, METH_VARARGS, "The way to read tensors past the interpreter; once."},
    {"norm_rope", (PyCFunction)(void (*)(void))py_norm_rope, METH_FASTCALL, "tl_qk_norm_rope"},
    {"append_rope", (PyCFunction)(void (*)(void))py_append_rope, METH_FASTCALL, "tl_kv4_append_rope"},
    {"sample", (PyCFunction)(void (*)(void))py_sample, METH_FASTCALL, "tl_sample"},
    {"attention_prefix", (PyCFunction)(void (*)(void))py_attention_prefix, METH_FASTCALL, "tl_kv4_attention_prefix"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tlq_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tlq_binding(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_numel = PyUnicode_InternFromString("numel");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  if (!s_dtype || !s_is_cuda || !s_is_contiguous || !s_data_ptr || !s_numel || !s_shape || !s_stride) return NULL;
  return PyModule_Create(&module);
}

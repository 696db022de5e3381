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
 * goes through its own checks, which name what is wrong).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/tlq.h"

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

/* Sizes (s_shape) or strides (s_stride) of a tensor of `dims` dimensions. */
static int extents(PyObject* t, int strides, int dims, long long* out) {
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
  long long size[3], step[3];
  if (!attr_is(t, s_dtype, t_f16) || !attr_is(t, s_is_cuda, Py_True) || !extents(t, 0, dims, size) ||
      !extents(t, 1, dims, step))
    return 0;
  if (size[0] < 1 || size[1] != a || (dims == 3 && (size[2] != b || step[1] != b)) || step[dims - 1] != 1) return 0;
  *ld = size[0] > 1 ? step[0] : (dims == 3 ? a * b : a);
  *tokens = size[0];
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

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "Torch's types and the library's entry points; once."},
    {"plan", (PyCFunction)(void (*)(void))py_plan, METH_FASTCALL, "tl_kv_plan"},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, "tl_kv4_append"},
    {"read", (PyCFunction)(void (*)(void))py_read_back, METH_FASTCALL, "tl_kv4_read"},
    {"attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, "tl_kv4_attention"},
    {"lora", (PyCFunction)(void (*)(void))py_lora, METH_FASTCALL, "tl_lora_add"},
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

/* _fastcall.c -- CPython entry points for the per-step calls of libqsa.so.
 *
 * Marshalling only, like the ctypes path it stands in for: each function
 * takes the C function's arguments in order (device pointers as Python ints
 * or None, sizes as ints, the RoPE base as a float), calls the library and
 * returns its status.  It exists because a ctypes call converts its
 * arguments one by one through their declared types (about 0.13 us each on
 * the host, 26 of them per decode step), which is a large share of a decode
 * step's host time.  The Python module falls back to ctypes when this
 * extension was not built.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "qsa.h"

/* Argument i as a pointer (None -> NULL), a 64-bit or 32-bit integer, a
 * size or a double; any failure leaves a Python error set. */
static void* arg_ptr(PyObject* const* a, Py_ssize_t i) {
  if (a[i] == Py_None) return NULL;
  return PyLong_AsVoidPtr(a[i]);
}
static int64_t arg_i64(PyObject* const* a, Py_ssize_t i) { return (int64_t)PyLong_AsLongLong(a[i]); }
static int32_t arg_i32(PyObject* const* a, Py_ssize_t i) {
  const long long v = PyLong_AsLongLong(a[i]);
  if (!PyErr_Occurred() && (v < INT32_MIN || v > INT32_MAX)) PyErr_SetString(PyExc_OverflowError, "int32 argument");
  return (int32_t)v;
}
static size_t arg_size(PyObject* const* a, Py_ssize_t i) { return (size_t)PyLong_AsSize_t(a[i]); }

static int want_args(Py_ssize_t got, Py_ssize_t n, const char* fn) {
  if (got == n) return 1;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", fn, n, got);
  return 0;
}

/* qsa_decode_step and qsa_decode_step_gated share every argument but the
 * gates (after q). */
static PyObject* decode_step_impl(PyObject* const* a, Py_ssize_t n, int gated) {
  const Py_ssize_t g = gated ? 1 : 0;
  if (!want_args(n, 26 + g, gated ? "decode_step_gated" : "decode_step")) return NULL;
  const void* new_keys = arg_ptr(a, 0);
  const int32_t* req_tok_start = arg_ptr(a, 1);
  const int32_t* req_first_pos = arg_ptr(a, 2);
  void* ring = arg_ptr(a, 3);
  const double rope_base = PyFloat_AsDouble(a[4]);
  const void* q = arg_ptr(a, 5);
  const float* gates = gated ? (const float*)arg_ptr(a, 6) : NULL;
  void* pool = arg_ptr(a, 6 + g);
  const int64_t pool_rows = arg_i64(a, 7 + g);
  const int32_t n_req = arg_i32(a, 8 + g);
  const int32_t* req_row_start = arg_ptr(a, 9 + g);
  const int32_t n_rows = arg_i32(a, 10 + g);
  const int32_t* row_len = arg_ptr(a, 11 + g);
  const int32_t max_len = arg_i32(a, 12 + g), max_rows_per_req = arg_i32(a, 13 + g);
  const int32_t* page_table = arg_ptr(a, 14 + g);
  const int64_t ld_pt = arg_i64(a, 15 + g);
  const int32_t page_size = arg_i32(a, 16 + g), k_blk = arg_i32(a, 17 + g);
  int32_t* out_blocks = arg_ptr(a, 18 + g);
  int32_t* out_pos = arg_ptr(a, 19 + g);
  int32_t* out_slots = arg_ptr(a, 20 + g);
  float* scores_out = arg_ptr(a, 21 + g);
  const int64_t ld_scores = arg_i64(a, 22 + g);
  void* workspace = arg_ptr(a, 23 + g);
  const size_t ws_bytes = arg_size(a, 24 + g);
  void* stream = arg_ptr(a, 25 + g);
  if (PyErr_Occurred()) return NULL;
  const qsa_status st =
      gated ? qsa_decode_step_gated(new_keys, req_tok_start, req_first_pos, ring, rope_base, q, gates, pool,
                                    pool_rows, n_req, req_row_start, n_rows, row_len, max_len, max_rows_per_req,
                                    page_table, ld_pt, page_size, k_blk, out_blocks, out_pos, out_slots,
                                    scores_out, ld_scores, workspace, ws_bytes, stream)
            : qsa_decode_step(new_keys, req_tok_start, req_first_pos, ring, rope_base, q, pool, pool_rows, n_req,
                              req_row_start, n_rows, row_len, max_len, max_rows_per_req, page_table, ld_pt,
                              page_size, k_blk, out_blocks, out_pos, out_slots, scores_out, ld_scores, workspace,
                              ws_bytes, stream);
  return PyLong_FromLong((long)st);
}

static PyObject* fc_decode_step(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return decode_step_impl(a, n, 0);
}
static PyObject* fc_decode_step_gated(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return decode_step_impl(a, n, 1);
}

/* qsa_indexer_select (pool) and qsa_indexer_select_gated (gates, pool). */
static PyObject* indexer_select_impl(PyObject* const* a, Py_ssize_t n, int gated) {
  const Py_ssize_t g = gated ? 1 : 0;
  if (!want_args(n, 21 + g, gated ? "indexer_select_gated" : "indexer_select")) return NULL;
  const void* q = arg_ptr(a, 0);
  const float* gates = gated ? (const float*)arg_ptr(a, 1) : NULL;
  const void* pool = arg_ptr(a, 1 + g);
  const int64_t pool_rows = arg_i64(a, 2 + g);
  const int32_t n_req = arg_i32(a, 3 + g);
  const int32_t* req_row_start = arg_ptr(a, 4 + g);
  const int32_t n_rows = arg_i32(a, 5 + g);
  const int32_t* row_len = arg_ptr(a, 6 + g);
  const int32_t max_len = arg_i32(a, 7 + g), max_rows_per_req = arg_i32(a, 8 + g);
  const int32_t* page_table = arg_ptr(a, 9 + g);
  const int64_t ld_pt = arg_i64(a, 10 + g);
  const int32_t page_size = arg_i32(a, 11 + g), k_blk = arg_i32(a, 12 + g);
  int32_t* out_blocks = arg_ptr(a, 13 + g);
  int32_t* out_pos = arg_ptr(a, 14 + g);
  int32_t* out_slots = arg_ptr(a, 15 + g);
  float* scores_out = arg_ptr(a, 16 + g);
  const int64_t ld_scores = arg_i64(a, 17 + g);
  void* workspace = arg_ptr(a, 18 + g);
  const size_t ws_bytes = arg_size(a, 19 + g);
  void* stream = arg_ptr(a, 20 + g);
  if (PyErr_Occurred()) return NULL;
  const qsa_status st =
      gated ? qsa_indexer_select_gated(q, gates, pool, pool_rows, n_req, req_row_start, n_rows, row_len, max_len,
                                       max_rows_per_req, page_table, ld_pt, page_size, k_blk, out_blocks, out_pos,
                                       out_slots, scores_out, ld_scores, workspace, ws_bytes, stream)
            : qsa_indexer_select(q, pool, pool_rows, n_req, req_row_start, n_rows, row_len, max_len,
                                 max_rows_per_req, page_table, ld_pt, page_size, k_blk, out_blocks, out_pos,
                                 out_slots, scores_out, ld_scores, workspace, ws_bytes, stream);
  return PyLong_FromLong((long)st);
}

static PyObject* fc_indexer_select(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return indexer_select_impl(a, n, 0);
}
static PyObject* fc_indexer_select_gated(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return indexer_select_impl(a, n, 1);
}

/* The calls of the 4-bit cache and the window attention: one argument after
 * the other in the C function's order. */
static float arg_f32(PyObject* const* a, Py_ssize_t i) { return (float)PyFloat_AsDouble(a[i]); }

static PyObject* fc_append_kv_fp4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!want_args(n, 21, "append_kv_fp4")) return NULL;
  const void *k_new = arg_ptr(a, 0), *v_new = arg_ptr(a, 1);
  const int64_t ld_k = arg_i64(a, 2), ld_v = arg_i64(a, 3);
  const int32_t n_tok = arg_i32(a, 4), h_kv = arg_i32(a, 5), d = arg_i32(a, 6);
  const int32_t *start = arg_ptr(a, 7), *first = arg_ptr(a, 8);
  const int32_t n_req = arg_i32(a, 9);
  const int32_t* pt = arg_ptr(a, 10);
  const int64_t ld_pt = arg_i64(a, 11);
  const int32_t page = arg_i32(a, 12);
  const float ks = arg_f32(a, 13), vs = arg_f32(a, 14);
  void *c0 = arg_ptr(a, 15), *c1 = arg_ptr(a, 16), *c2 = arg_ptr(a, 17), *c3 = arg_ptr(a, 18);
  const int64_t n_slots = arg_i64(a, 19);
  void* stream = arg_ptr(a, 20);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong((long)qsa_append_kv_fp4(k_new, v_new, ld_k, ld_v, n_tok, h_kv, d, start, first, n_req, pt,
                                                 ld_pt, page, ks, vs, c0, c1, c2, c3, n_slots, stream));
}

static PyObject* fc_gather_kv_fp4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!want_args(n, 14, "gather_kv_fp4")) return NULL;
  const void *c0 = arg_ptr(a, 0), *c1 = arg_ptr(a, 1), *c2 = arg_ptr(a, 2), *c3 = arg_ptr(a, 3);
  const int64_t n_slots = arg_i64(a, 4);
  const int32_t h_kv = arg_i32(a, 5), d = arg_i32(a, 6);
  const int32_t* slots = arg_ptr(a, 7);
  const int64_t cnt = arg_i64(a, 8);
  const float ks = arg_f32(a, 9), vs = arg_f32(a, 10);
  void *k_out = arg_ptr(a, 11), *v_out = arg_ptr(a, 12), *stream = arg_ptr(a, 13);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong((long)qsa_gather_kv_fp4(c0, c1, c2, c3, n_slots, h_kv, d, slots, cnt, ks, vs, k_out, v_out,
                                                 stream));
}

static PyObject* fc_sparse_attn_fp4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!want_args(n, 22, "sparse_attn_fp4")) return NULL;
  const void* q = arg_ptr(a, 0);
  const int64_t ld_q = arg_i64(a, 1);
  const void *c0 = arg_ptr(a, 2), *c1 = arg_ptr(a, 3), *c2 = arg_ptr(a, 4), *c3 = arg_ptr(a, 5);
  const int64_t n_slots = arg_i64(a, 6);
  const int32_t n_rows = arg_i32(a, 7), h_q = arg_i32(a, 8), h_kv = arg_i32(a, 9), d = arg_i32(a, 10);
  const int32_t* slots = arg_ptr(a, 11);
  const int64_t ld_slots = arg_i64(a, 12);
  const int32_t n_idx = arg_i32(a, 13);
  const float scale = arg_f32(a, 14), ks = arg_f32(a, 15), vs = arg_f32(a, 16);
  float *out = arg_ptr(a, 17), *lse = arg_ptr(a, 18);
  void* ws = arg_ptr(a, 19);
  const size_t ws_bytes = arg_size(a, 20);
  void* stream = arg_ptr(a, 21);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromLong((long)qsa_sparse_attn_fp4(q, ld_q, c0, c1, c2, c3, n_slots, n_rows, h_q, h_kv, d, slots,
                                                   ld_slots, n_idx, scale, ks, vs, out, lse, ws, ws_bytes, stream));
}

/* qsa_window_attn (two cache arrays, no tensor scales) and
 * qsa_window_attn_fp4 (four arrays, two scales). */
static PyObject* window_attn_impl(PyObject* const* a, Py_ssize_t n, int fp4) {
  const Py_ssize_t c = fp4 ? 2 : 0;
  if (!want_args(n, 25 + 2 * c, fp4 ? "window_attn_fp4" : "window_attn")) return NULL;
  const void* q = arg_ptr(a, 0);
  const int64_t ld_q = arg_i64(a, 1);
  const void *c0 = arg_ptr(a, 2), *c1 = arg_ptr(a, 3);
  const void *c2 = fp4 ? arg_ptr(a, 4) : NULL, *c3 = fp4 ? arg_ptr(a, 5) : NULL;
  const int64_t n_slots = arg_i64(a, 4 + c);
  const int32_t n_req = arg_i32(a, 5 + c);
  const int32_t* start = arg_ptr(a, 6 + c);
  const int32_t n_rows = arg_i32(a, 7 + c);
  const int32_t* row_len = arg_ptr(a, 8 + c);
  const int32_t max_len = arg_i32(a, 9 + c), max_rows = arg_i32(a, 10 + c);
  const int32_t h_q = arg_i32(a, 11 + c), h_kv = arg_i32(a, 12 + c), d = arg_i32(a, 13 + c);
  const int32_t* pt = arg_ptr(a, 14 + c);
  const int64_t ld_pt = arg_i64(a, 15 + c);
  const int32_t page = arg_i32(a, 16 + c), window = arg_i32(a, 17 + c), sinks = arg_i32(a, 18 + c);
  const float scale = arg_f32(a, 19 + c);
  const float ks = fp4 ? arg_f32(a, 22) : 1.0f, vs = fp4 ? arg_f32(a, 23) : 1.0f;
  void* out = arg_ptr(a, 20 + 2 * c);
  float* lse = arg_ptr(a, 21 + 2 * c);
  void* ws = arg_ptr(a, 22 + 2 * c);
  const size_t ws_bytes = arg_size(a, 23 + 2 * c);
  void* stream = arg_ptr(a, 24 + 2 * c);
  if (PyErr_Occurred()) return NULL;
  const qsa_status st =
      fp4 ? qsa_window_attn_fp4(q, ld_q, c0, c1, c2, c3, n_slots, n_req, start, n_rows, row_len, max_len, max_rows,
                                h_q, h_kv, d, pt, ld_pt, page, window, sinks, scale, ks, vs, out, lse, ws, ws_bytes,
                                stream)
          : qsa_window_attn(q, ld_q, c0, c1, n_slots, n_req, start, n_rows, row_len, max_len, max_rows, h_q, h_kv, d,
                            pt, ld_pt, page, window, sinks, scale, out, lse, ws, ws_bytes, stream);
  return PyLong_FromLong((long)st);
}
static PyObject* fc_window_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return window_attn_impl(a, n, 0);
}
static PyObject* fc_window_attn_fp4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return window_attn_impl(a, n, 1);
}

/* The workspace queries of those calls: int32 arguments, a size. */
static PyObject* fc_sparse_attn_fp4_workspace_size(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!want_args(n, 5, "sparse_attn_fp4_workspace_size")) return NULL;
  const int32_t v0 = arg_i32(a, 0), v1 = arg_i32(a, 1), v2 = arg_i32(a, 2), v3 = arg_i32(a, 3), v4 = arg_i32(a, 4);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromSize_t(qsa_sparse_attn_fp4_workspace_size(v0, v1, v2, v3, v4));
}
static PyObject* fc_window_attn_workspace_size(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!want_args(n, 7, "window_attn_workspace_size")) return NULL;
  const int32_t v0 = arg_i32(a, 0), v1 = arg_i32(a, 1), v2 = arg_i32(a, 2), v3 = arg_i32(a, 3), v4 = arg_i32(a, 4);
  const int32_t v5 = arg_i32(a, 5), v6 = arg_i32(a, 6);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromSize_t(qsa_window_attn_workspace_size(v0, v1, v2, v3, v4, v5, v6));
}

static PyMethodDef fc_methods[] = {
    {"qsa_decode_step", (PyCFunction)(void (*)(void))fc_decode_step, METH_FASTCALL, "qsa_decode_step"},
    {"qsa_decode_step_gated", (PyCFunction)(void (*)(void))fc_decode_step_gated, METH_FASTCALL,
     "qsa_decode_step_gated"},
    {"qsa_indexer_select", (PyCFunction)(void (*)(void))fc_indexer_select, METH_FASTCALL, "qsa_indexer_select"},
    {"qsa_indexer_select_gated", (PyCFunction)(void (*)(void))fc_indexer_select_gated, METH_FASTCALL,
     "qsa_indexer_select_gated"},
    {"qsa_append_kv_fp4", (PyCFunction)(void (*)(void))fc_append_kv_fp4, METH_FASTCALL, "qsa_append_kv_fp4"},
    {"qsa_gather_kv_fp4", (PyCFunction)(void (*)(void))fc_gather_kv_fp4, METH_FASTCALL, "qsa_gather_kv_fp4"},
    {"qsa_sparse_attn_fp4", (PyCFunction)(void (*)(void))fc_sparse_attn_fp4, METH_FASTCALL, "qsa_sparse_attn_fp4"},
    {"qsa_window_attn", (PyCFunction)(void (*)(void))fc_window_attn, METH_FASTCALL, "qsa_window_attn"},
    {"qsa_window_attn_fp4", (PyCFunction)(void (*)(void))fc_window_attn_fp4, METH_FASTCALL, "qsa_window_attn_fp4"},
    {"qsa_sparse_attn_fp4_workspace_size", (PyCFunction)(void (*)(void))fc_sparse_attn_fp4_workspace_size, METH_FASTCALL, "qsa_sparse_attn_fp4_workspace_size"},
    {"qsa_window_attn_workspace_size", (PyCFunction)(void (*)(void))fc_window_attn_workspace_size, METH_FASTCALL, "qsa_window_attn_workspace_size"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef fc_module = {PyModuleDef_HEAD_INIT,
                                       "_fastcall",
                                       "Per-step calls of libqsa.so without ctypes argument conversion.",
                                       -1,
                                       fc_methods,
                                       NULL,
                                       NULL,
                                       NULL,
                                       NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&fc_module); }

/*
 * CPython entry points for the router's hot calls: argument conversion only.
 *
 * Each function takes the arguments of the C entry point of the same name
 * (include/moe_router.h) as Python integers and floats -- device pointers as
 * integers, 0 for NULL, the stream as its raw handle -- converts them, calls
 * the library and returns its status code.  The Python binding uses these
 * instead of ctypes where the module was built: for decode-sized calls the
 * host cost of converting fourteen arguments through ctypes is a large part
 * of the latency.  Nothing here computes anything on the router's data.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "moe_router.h"

/* Convert args[0 .. n-1] by the format string: 'p' pointer (unsigned
 * integer), 'i' int, 'f' float.  Returns 0 on success, -1 with a Python
 * exception set. */
static int convert(PyObject* const* args, Py_ssize_t nargs, const char* fmt, void** out) {
  const Py_ssize_t n = (Py_ssize_t)strlen(fmt);
  if (nargs != n) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, nargs);
    return -1;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (fmt[i] == 'p') {
      const unsigned long long v = PyLong_AsUnsignedLongLong(args[i]);
      if (v == (unsigned long long)-1 && PyErr_Occurred()) return -1;
      *(uintptr_t*)out[i] = (uintptr_t)v;
    } else if (fmt[i] == 'i') {
      const long v = PyLong_AsLong(args[i]);
      if (v == -1 && PyErr_Occurred()) return -1;
      if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "integer argument out of int range");
        return -1;
      }
      *(int*)out[i] = (int)v;
    } else {
      const double v = PyFloat_AsDouble(args[i]);
      if (v == -1.0 && PyErr_Occurred()) return -1;
      *(float*)out[i] = (float)v;
    }
  }
  return 0;
}

static PyObject* call_topk_fwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t logits, bias, probs, map, scores, stream;
  int dt, T, E, K, sf, ng, gk;
  float c;
  void* out[] = {&logits, &dt, &T, &E, &K, &sf, &ng, &gk, &c, &bias, &probs, &map, &scores,
                 &stream};
  if (convert(args, nargs, "piiiiiiifppppp", out) != 0) return NULL;
  const int rc = router_topk_fwd((const void*)logits, (mr_dtype)dt, T, E, K, (mr_score_func)sf,
                                 ng, gk, c, (const float*)bias, (void*)probs, (uint8_t*)map,
                                 (float*)scores, (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_topk_bwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t grad, map, scores, grad_logits, stream;
  int dt, T, E, K, sf;
  float c;
  void* out[] = {&grad, &map, &scores, &dt, &T, &E, &K, &sf, &c, &grad_logits, &stream};
  if (convert(args, nargs, "pppiiiiifpp", out) != 0) return NULL;
  const int rc = router_topk_bwd((const void*)grad, (const uint8_t*)map, (const float*)scores,
                                 (mr_dtype)dt, T, E, K, (mr_score_func)sf, c, (void*)grad_logits,
                                 (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_aux_scores_fwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t logits, scores, map, inter, stream;
  int dt, T, E, K, sf;
  void* out[] = {&logits, &dt, &T, &E, &K, &sf, &scores, &map, &inter, &stream};
  if (convert(args, nargs, "piiiiipppp", out) != 0) return NULL;
  const int rc = router_aux_scores_fwd((const void*)logits, (mr_dtype)dt, T, E, K,
                                       (mr_score_func)sf, (float*)scores, (uint8_t*)map,
                                       (float*)inter, (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_aux_scores_bwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t grad, saved, grad_logits, stream;
  int dt, T, E, K, sf;
  void* out[] = {&grad, &saved, &dt, &T, &E, &K, &sf, &grad_logits, &stream};
  if (convert(args, nargs, "ppiiiiipp", out) != 0) return NULL;
  const int rc = router_aux_scores_bwd((const float*)grad, (const float*)saved, (mr_dtype)dt, T,
                                       E, K, (mr_score_func)sf, (void*)grad_logits,
                                       (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_expert_matmul(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t x, w, off, p2u, o, stream;
  int dt, T, P, E, N, D, odt;
  void* out[] = {&x, &dt, &w, &off, &p2u, &T, &P, &E, &N, &D, &o, &odt, &stream};
  if (convert(args, nargs, "pipppiiiiipip", out) != 0) return NULL;
  const int rc = router_expert_matmul((const void*)x, (mr_dtype)dt, (const void*)w,
                                      (const int32_t*)off, (const int32_t*)p2u, T, P, E, N, D,
                                      (void*)o, (mr_dtype)odt, (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_expert_matmul_w4(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t x, q, sc, z, off, p2u, o, stream;
  int group, T, P, E, N, D, odt;
  void* out[] = {&x, &q, &sc, &z, &group, &off, &p2u, &T, &P, &E, &N, &D, &o, &odt, &stream};
  if (convert(args, nargs, "ppppippiiiiipip", out) != 0) return NULL;
  const int rc = router_expert_matmul_w4(
      (const void*)x, (const uint8_t*)q, (const void*)sc, (const uint8_t*)z, group,
      (const int32_t*)off, (const int32_t*)p2u, T, P, E, N, D, (void*)o, (mr_dtype)odt,
      (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_combine_fwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t z, u2p, w, o, stream;
  int dt, ld, T, K, D;
  void* out[] = {&z, &dt, &u2p, &w, &ld, &T, &K, &D, &o, &stream};
  if (convert(args, nargs, "pippiiiipp", out) != 0) return NULL;
  const int rc =
      router_combine_fwd((const void*)z, (mr_dtype)dt, (const int32_t*)u2p, (const float*)w, ld,
                         T, K, D, (void*)o, (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_combine_bwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  uintptr_t g, u2p, z, w, gz, gw, stream;
  int dt, ld, T, K, D;
  void* out[] = {&g, &dt, &u2p, &z, &w, &ld, &T, &K, &D, &gz, &gw, &stream};
  if (convert(args, nargs, "pipppiiiippp", out) != 0) return NULL;
  const int rc = router_combine_bwd((const void*)g, (mr_dtype)dt, (const int32_t*)u2p,
                                    (const void*)z, (const float*)w, ld, T, K, D, (void*)gz,
                                    (float*)gw, (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_expert_matmul_bwd_input(PyObject* self, PyObject* const* args,
                                              Py_ssize_t nargs) {
  uintptr_t g, w, off, gx, stream;
  int dt, P, E, N, D, odt;
  void* out[] = {&g, &dt, &w, &off, &P, &E, &N, &D, &gx, &odt, &stream};
  if (convert(args, nargs, "pippiiiipip", out) != 0) return NULL;
  const int rc = router_expert_matmul_bwd_input((const void*)g, (mr_dtype)dt, (const void*)w,
                                                (const int32_t*)off, P, E, N, D, (void*)gx,
                                                (mr_dtype)odt, (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyObject* call_expert_matmul_bwd_weight(PyObject* self, PyObject* const* args,
                                               Py_ssize_t nargs) {
  uintptr_t g, x, off, p2u, gw, stream;
  int dt, T, P, E, N, D, odt;
  void* out[] = {&g, &dt, &x, &off, &p2u, &T, &P, &E, &N, &D, &gw, &odt, &stream};
  if (convert(args, nargs, "pipppiiiiipip", out) != 0) return NULL;
  const int rc = router_expert_matmul_bwd_weight((const void*)g, (mr_dtype)dt, (const void*)x,
                                                 (const int32_t*)off, (const int32_t*)p2u, T, P,
                                                 E, N, D, (void*)gw, (mr_dtype)odt,
                                                 (mr_stream_t)stream);
  return PyLong_FromLong(rc);
}

static PyMethodDef kMethods[] = {
    {"router_topk_fwd", (PyCFunction)(void (*)(void))call_topk_fwd, METH_FASTCALL,
     "router_topk_fwd(logits, dtype, T, E, K, score_func, num_groups, group_topk, "
     "scaling_factor, expert_bias, probs, routing_map, scores, stream) -> status"},
    {"router_topk_bwd", (PyCFunction)(void (*)(void))call_topk_bwd, METH_FASTCALL,
     "router_topk_bwd(grad_probs, routing_map, scores, dtype, T, E, K, score_func, "
     "scaling_factor, grad_logits, stream) -> status"},
    {"router_aux_scores_fwd", (PyCFunction)(void (*)(void))call_aux_scores_fwd, METH_FASTCALL,
     "router_aux_scores_fwd(logits, dtype, T, E, K, score_func, scores, routing_map, "
     "intermediate, stream) -> status"},
    {"router_aux_scores_bwd", (PyCFunction)(void (*)(void))call_aux_scores_bwd, METH_FASTCALL,
     "router_aux_scores_bwd(grad_scores, saved, dtype, T, E, K, score_func, grad_logits, "
     "stream) -> status"},
    {"router_expert_matmul", (PyCFunction)(void (*)(void))call_expert_matmul, METH_FASTCALL,
     "router_expert_matmul(x, dtype, weight, offsets, p2u, T, P, E, N, D, out, out_dtype, "
     "stream) -> status"},
    {"router_expert_matmul_w4", (PyCFunction)(void (*)(void))call_expert_matmul_w4,
     METH_FASTCALL,
     "router_expert_matmul_w4(x, qweight, scales, zeros, group_size, offsets, p2u, T, P, E, N, "
     "D, out, out_dtype, stream) -> status"},
    {"router_combine_fwd", (PyCFunction)(void (*)(void))call_combine_fwd, METH_FASTCALL,
     "router_combine_fwd(expert_out, dtype, u2p, topk_weights, ld_weights, T, K, D, out, "
     "stream) -> status"},
    {"router_combine_bwd", (PyCFunction)(void (*)(void))call_combine_bwd, METH_FASTCALL,
     "router_combine_bwd(grad_out, dtype, u2p, expert_out, topk_weights, ld_weights, T, K, D, "
     "grad_expert_out, grad_weights, stream) -> status"},
    {"router_expert_matmul_bwd_input",
     (PyCFunction)(void (*)(void))call_expert_matmul_bwd_input, METH_FASTCALL,
     "router_expert_matmul_bwd_input(grad_out, dtype, weight, offsets, P, E, N, D, grad_x, "
     "out_dtype, stream) -> status"},
    {"router_expert_matmul_bwd_weight",
     (PyCFunction)(void (*)(void))call_expert_matmul_bwd_weight, METH_FASTCALL,
     "router_expert_matmul_bwd_weight(grad_out, dtype, x, offsets, p2u, T, P, E, N, D, "
     "grad_weight, out_dtype, stream) -> status"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pycalls",
                                     "CPython entry points of the router's hot calls.", -1,
                                     kMethods};

PyMODINIT_FUNC PyInit__pycalls(void) { return PyModule_Create(&kModule); }

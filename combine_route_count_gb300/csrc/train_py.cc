// CPython module _train: the argument checks of train.py on torch tensors and the
// calls into libmoe.so (include/moe_train.h), as ffn_py.cc's for ffn.py.

#include "moe_train.h"
#include "py_args.h"

namespace {

using namespace moe_py;

int type_of(PyObject* o) {
  return THPVariable_Unpack(o).scalar_type() == at::ScalarType::Float ? MOE_TYPE_F32 : MOE_TYPE_BF16;
}

bool int_of(PyObject* o, int* v) {
  const long got = PyLong_AsLong(o);
  if (got == -1 && PyErr_Occurred()) return false;
  *v = static_cast<int>(got);
  return true;
}

// The first tensor of a call: two dimensions, on the current device; -1 if not.
int rows_of(const char* name, PyObject* o, int64_t* n0, int64_t* n1) {
  const at::Tensor* t = tensor(name, o);
  if (!t) return -1;
  if (t->dim() != 2) {
    fail(MOE_EINVAL, "%s must have 2 dimensions", name);
    return -1;
  }
  *n0 = t->size(0);
  *n1 = t->size(1);
  return device_of(name, *t);
}

// The second dimension of a tensor that has two.
bool columns_of(const char* name, PyObject* o, int64_t* n1) {
  const at::Tensor* t = tensor(name, o);
  if (!t) return false;
  if (t->dim() != 2) {
    fail(MOE_EINVAL, "%s must have 2 dimensions", name);
    return false;
  }
  *n1 = t->size(1);
  return true;
}

// Weights [E, n, k], or [n, k] for one expert.
bool weights_of(const char* name, PyObject* o, int* one, int64_t* E, int64_t* n, int64_t* k) {
  const at::Tensor* t = tensor(name, o);
  if (!t) return false;
  if (t->dim() != 2 && t->dim() != 3) {
    fail(MOE_EINVAL, "%s must have 3 dimensions, or 2 for one expert", name);
    return false;
  }
  *one = t->dim() == 2;
  *E = *one ? 1 : t->size(0);
  *n = t->size(1 - *one);
  *k = t->size(2 - *one);
  return true;
}

bool arg_or_none(const char* name, PyObject* o, unsigned types, int64_t n0, int64_t n1, int device, void** address) {
  *address = nullptr;
  return o == Py_None || arg2(name, o, types, n0, n1, device, address);
}

// expert_offsets and status, either may be None.
bool groups_of(PyObject* offsets, PyObject* status, int64_t E, int device, void** offsets_at, void** status_at) {
  *offsets_at = *status_at = nullptr;
  return (offsets == Py_None || arg1("expert_offsets", offsets, kI32, E + 1, device, offsets_at)) &&
         (status == Py_None || arg1("status", status, kI32, 1, device, status_at));
}

float* f32(void* p) { return static_cast<float*>(p); }
int32_t* i32(void* p) { return static_cast<int32_t*>(p); }

// (logits, topk_idx, topk_w, bias, score, normalize, scale, stream)
PyObject* router_topk(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 8)) return nullptr;
  int64_t T, E, K;
  const int dev = rows_of("logits", v[0], &T, &E);
  if (dev < 0 || !columns_of("topk_idx", v[1], &K)) return nullptr;
  void *pl, *pi, *pw, *pb = nullptr, *stream;
  if (!arg2("logits", v[0], kFloat, T, E, dev, &pl) || !arg2("topk_idx", v[1], kI32, T, K, dev, &pi) ||
      !arg2("topk_w", v[2], kF32, T, K, dev, &pw) || (v[3] != Py_None && !arg1("bias", v[3], kF32, E, dev, &pb)))
    return nullptr;
  int score;
  const double scale = PyFloat_AsDouble(v[6]);
  if ((scale == -1.0 && PyErr_Occurred()) || !int_of(v[4], &score) || !stream_of(v[7], &stream) || !fits("E", E) ||
      !fits("K", K))
    return nullptr;
  const int normalize = PyObject_IsTrue(v[5]), type = type_of(v[0]);
  if (normalize < 0) return nullptr;
  return call("moe_router_topk", [&] {
    return moe_router_topk(pl, type, f32(pb), T, static_cast<int32_t>(E), static_cast<int32_t>(K), score, normalize,
                           static_cast<float>(scale), i32(pi), f32(pw), stream);
  });
}

// (logits, topk_idx, d_topk_w, d_logits, score, normalize, scale, stream)
PyObject* router_topk_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 8)) return nullptr;
  int64_t T, E, K;
  const int dev = rows_of("logits", v[0], &T, &E);
  if (dev < 0 || !columns_of("topk_idx", v[1], &K)) return nullptr;
  void *pl, *pi, *pw, *pd, *stream;
  if (!arg2("logits", v[0], kFloat, T, E, dev, &pl) || !arg2("topk_idx", v[1], kI32, T, K, dev, &pi) ||
      !arg2("d_topk_w", v[2], kF32, T, K, dev, &pw) || !arg2("d_logits", v[3], kFloat, T, E, dev, &pd))
    return nullptr;
  if (type_of(v[0]) != type_of(v[3])) return fail(MOE_EINVAL, "d_logits must be of the logits' type");
  int score;
  const double scale = PyFloat_AsDouble(v[6]);
  if ((scale == -1.0 && PyErr_Occurred()) || !int_of(v[4], &score) || !stream_of(v[7], &stream) || !fits("E", E) ||
      !fits("K", K))
    return nullptr;
  const int normalize = PyObject_IsTrue(v[5]), type = type_of(v[0]);
  if (normalize < 0) return nullptr;
  return call("moe_router_topk_backward", [&] {
    return moe_router_topk_backward(pl, type, i32(pi), f32(pw), T, static_cast<int32_t>(E), static_cast<int32_t>(K),
                                    score, normalize, static_cast<float>(scale), pd, stream);
  });
}

// (d_out, slot_row, topk_w, d_expert_y, expert_y, d_topk_w, stream)
PyObject* combine_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 7)) return nullptr;
  int64_t T, H, K;
  const int dev = rows_of("d_out", v[0], &T, &H);
  const at::Tensor* dy = dev < 0 ? nullptr : tensor("d_expert_y", v[3]);
  if (!dy || !columns_of("slot_row", v[1], &K)) return nullptr;
  if (dy->dim() != 2) return fail(MOE_EINVAL, "d_expert_y must have 2 dimensions");
  const int64_t rows = dy->size(0);
  void *pg, *ps, *pw, *pd, *py, *pt, *stream;
  if (!arg2("d_out", v[0], kBf16, T, H, dev, &pg) || !arg2("slot_row", v[1], kI32, T, K, dev, &ps) ||
      !arg2("topk_w", v[2], kF32, T, K, dev, &pw) || !arg2("d_expert_y", v[3], kBf16, rows, H, dev, &pd) ||
      !arg_or_none("expert_y", v[4], kBf16, rows, H, dev, &py) ||
      !arg_or_none("d_topk_w", v[5], kF32, T, K, dev, &pt))
    return nullptr;
  if ((v[4] == Py_None) != (v[5] == Py_None)) return fail(MOE_EINVAL, "expert_y and d_topk_w go together");
  if (!stream_of(v[6], &stream) || !fits("H", H) || !fits("K", K)) return nullptr;
  return call("moe_combine_backward", [&] {
    return moe_combine_backward(pg, py, f32(pw), i32(ps), T, static_cast<int32_t>(H), static_cast<int32_t>(K), rows, pd,
                                f32(pt), stream);
  });
}

// (d_expert_x, slot_row, d_x, add, stream)
PyObject* dispatch_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  int64_t rows, H, K;
  const int dev = rows_of("d_expert_x", v[0], &rows, &H);
  const at::Tensor* dx = dev < 0 ? nullptr : tensor("d_x", v[2]);
  if (!dx || !columns_of("slot_row", v[1], &K)) return nullptr;
  if (dx->dim() != 2) return fail(MOE_EINVAL, "d_x must have 2 dimensions");
  const int64_t T = dx->size(0);
  void *pe, *ps, *px, *pa, *stream;
  if (!arg2("d_expert_x", v[0], kBf16, rows, H, dev, &pe) || !arg2("slot_row", v[1], kI32, T, K, dev, &ps) ||
      !arg2("d_x", v[2], kBf16, T, H, dev, &px) || !arg_or_none("add", v[3], kBf16, T, H, dev, &pa))
    return nullptr;
  if (!stream_of(v[4], &stream) || !fits("H", H) || !fits("K", K)) return nullptr;
  return call("moe_dispatch_backward", [&] {
    return moe_dispatch_backward(pe, i32(ps), pa, T, static_cast<int32_t>(H), static_cast<int32_t>(K), rows, px,
                                 stream);
  });
}

// (a, w, out, bias, activation, residual, pre, expert_offsets, status, stream)
PyObject* expert_linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 10)) return nullptr;
  int64_t rows, K, E, N, k;
  int one, act;
  const int dev = rows_of("a", v[0], &rows, &K);
  if (dev < 0 || !weights_of("w", v[1], &one, &E, &N, &k) || !int_of(v[4], &act)) return nullptr;
  const int64_t w_shape[3] = {E, N, K}, b_shape[2] = {E, N};
  const int64_t n_out = act == MOE_ACT_SWIGLU ? N / 2 : N;
  void *pa, *pw, *po, *pb = nullptr, *pr, *pp, *pe, *pt, *stream;
  if (!arg2("a", v[0], kBf16, rows, K, dev, &pa) || !arg("w", v[1], kBf16, 3 - one, w_shape + one, dev, &pw) ||
      !arg2("out", v[2], kFloat, rows, n_out, dev, &po) ||
      (v[3] != Py_None && !arg("bias", v[3], kFloat, 2 - one, b_shape + one, dev, &pb)) ||
      !arg_or_none("residual", v[5], kBf16, rows, n_out, dev, &pr) ||
      !arg_or_none("pre", v[6], kBf16, rows, N, dev, &pp) || !groups_of(v[7], v[8], E, dev, &pe, &pt))
    return nullptr;
  if (!stream_of(v[9], &stream) || !fits("K", K) || !fits("N", N) || !fits("E", E)) return nullptr;
  const int bias_type = v[3] == Py_None ? MOE_TYPE_F32 : type_of(v[3]), type = type_of(v[2]);
  return call("moe_expert_linear", [&] {
    return moe_expert_linear(pa, rows, static_cast<int32_t>(K), pw, static_cast<int32_t>(N), static_cast<int32_t>(E),
                             i32(pe), pb, bias_type, act, pr, pp, po, type, i32(pt), stream);
  });
}

// (dy, w, dx, activation, pre, expert_offsets, status, stream)
PyObject* expert_linear_backward_input(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 8)) return nullptr;
  int64_t rows, N, E, n_w, K;
  int one, act;
  const int dev = rows_of("dy", v[0], &rows, &N);
  if (dev < 0 || !weights_of("w", v[1], &one, &E, &n_w, &K) || !int_of(v[3], &act)) return nullptr;
  const int64_t w_shape[3] = {E, N, K}, wide = act == MOE_ACT_SWIGLU ? 2 * K : K;
  void *pd, *pw, *px, *pp, *pe, *pt, *stream;
  if (!arg2("dy", v[0], kBf16, rows, N, dev, &pd) || !arg("w", v[1], kBf16, 3 - one, w_shape + one, dev, &pw) ||
      !arg2("dx", v[2], kBf16, rows, wide, dev, &px) || !arg_or_none("pre", v[4], kBf16, rows, wide, dev, &pp) ||
      !groups_of(v[5], v[6], E, dev, &pe, &pt))
    return nullptr;
  if ((v[4] == Py_None) != (act == MOE_ACT_NONE)) return fail(MOE_EINVAL, "an activation and pre go together");
  if (!stream_of(v[7], &stream) || !fits("K", K) || !fits("N", N) || !fits("E", E)) return nullptr;
  return call("moe_expert_linear_backward_input", [&] {
    return moe_expert_linear_backward_input(pd, rows, static_cast<int32_t>(N), pw, static_cast<int32_t>(K),
                                            static_cast<int32_t>(E), i32(pe), act, pp, px, i32(pt), stream);
  });
}

// (dy, a, dw, db, accumulate, expert_offsets, status, stream)
PyObject* expert_linear_backward_weight(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 8)) return nullptr;
  int64_t rows, N, K, E, n_w, k_w;
  int one;
  const int dev = rows_of("dy", v[0], &rows, &N);
  if (dev < 0 || !columns_of("a", v[1], &K) || !weights_of("dw", v[2], &one, &E, &n_w, &k_w)) return nullptr;
  const int64_t w_shape[3] = {E, N, K}, b_shape[2] = {E, N};
  void *pd, *pa, *pw, *pb = nullptr, *pe, *pt, *stream;
  if (!arg2("dy", v[0], kBf16, rows, N, dev, &pd) || !arg2("a", v[1], kBf16, rows, K, dev, &pa) ||
      !arg("dw", v[2], kFloat, 3 - one, w_shape + one, dev, &pw) ||
      (v[3] != Py_None && !arg("db", v[3], kF32, 2 - one, b_shape + one, dev, &pb)) ||
      !groups_of(v[5], v[6], E, dev, &pe, &pt))
    return nullptr;
  if (!stream_of(v[7], &stream) || !fits("K", K) || !fits("N", N) || !fits("E", E)) return nullptr;
  const int accumulate = PyObject_IsTrue(v[4]), type = type_of(v[2]);
  if (accumulate < 0) return nullptr;
  return call("moe_expert_linear_backward_weight", [&] {
    return moe_expert_linear_backward_weight(pd, rows, static_cast<int32_t>(N), pa, static_cast<int32_t>(K),
                                             static_cast<int32_t>(E), i32(pe), pw, type, f32(pb), accumulate, i32(pt),
                                             stream);
  });
}

PyMethodDef kMethods[] = {
    {"init", init, METH_O, "Sets the error class."},
    {"router_topk", fast<router_topk>(), METH_FASTCALL, nullptr},
    {"router_topk_backward", fast<router_topk_backward>(), METH_FASTCALL, nullptr},
    {"combine_backward", fast<combine_backward>(), METH_FASTCALL, nullptr},
    {"dispatch_backward", fast<dispatch_backward>(), METH_FASTCALL, nullptr},
    {"expert_linear", fast<expert_linear>(), METH_FASTCALL, nullptr},
    {"expert_linear_backward_input", fast<expert_linear_backward_input>(), METH_FASTCALL, nullptr},
    {"expert_linear_backward_weight", fast<expert_linear_backward_weight>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_train", "Argument checks and calls of train.py.", -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__train() { return PyModule_Create(&kModule); }

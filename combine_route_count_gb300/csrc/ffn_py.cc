// CPython module _ffn: the argument checks of ffn.py on torch tensors and the
// calls into libmoe.so (include/moe_ffn.h).
//
// A feed-forward call on a few tokens takes a few microseconds on the GPU; the
// same checks in Python (type, shape, contiguity, device and address of five to
// seven tensors) took as long as the launch (one token's norm: 8.2 us a call
// in Python, 3.2 us here).  Nothing is kept between calls.  A wrong argument
// raises the error class given to init with MOE_EINVAL, before anything is
// enqueued.

#include <cstring>

#include "moe_ffn.h"
#include "py_args.h"

namespace {

using namespace moe_py;

int64_t blocks(int64_t n) { return (n + MOE_FP8_BLOCK - 1) / MOE_FP8_BLOCK; }

// (x, weight, xq, x_scales, eps, residual, residual_out, y, stream)
PyObject* add_rms_norm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 9)) return nullptr;
  const at::Tensor* x = tensor("x", a[0]);
  if (!x) return nullptr;
  if (x->dim() != 2) return fail(MOE_EINVAL, "x must have 2 dimensions");
  const int dev = device_of("x", *x);
  if (dev < 0) return nullptr;
  const int64_t T = x->size(0), H = x->size(1);
  void *px, *pw, *pq, *ps, *pr = nullptr, *po = nullptr, *py = nullptr, *stream;
  if (!arg2("x", a[0], kBf16, T, H, dev, &px) || !arg1("weight", a[1], kFloat, H, dev, &pw) ||
      !arg2("xq", a[2], kFp8, T, H, dev, &pq) || !arg2("x_scales", a[3], kF32, T, H / MOE_FP8_BLOCK, dev, &ps))
    return nullptr;
  if ((a[5] == Py_None) != (a[6] == Py_None)) return fail(MOE_EINVAL, "residual and residual_out go together");
  if (a[5] != Py_None && (!arg2("residual", a[5], kBf16, T, H, dev, &pr) ||
                          !arg2("residual_out", a[6], kBf16, T, H, dev, &po)))
    return nullptr;
  if (a[7] != Py_None && !arg2("y", a[7], kBf16, T, H, dev, &py)) return nullptr;
  const double eps = PyFloat_AsDouble(a[4]);
  if ((eps == -1.0 && PyErr_Occurred()) || !stream_of(a[8], &stream) || !fits("H", H)) return nullptr;
  const int type = THPVariable_Unpack(a[1]).scalar_type() == at::ScalarType::Float ? MOE_TYPE_F32 : MOE_TYPE_BF16;
  return call("moe_add_rms_norm_fp8", [&] {
    return moe_add_rms_norm_fp8(px, pr, pw, type, T, static_cast<int32_t>(H), static_cast<float>(eps), po, py, pq,
                                static_cast<float*>(ps), stream);
  });
}

// (glu, a, a_scales, w, w_scales, out or hq, None or h_scales, expert_offsets, status, stream)
PyObject* expert_product(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 10)) return nullptr;
  const bool glu = v[0] == Py_True;
  const at::Tensor *a = tensor("a", v[1]), *w = a ? tensor("w", v[3]) : nullptr;
  if (!w) return nullptr;
  if (a->dim() != 2) return fail(MOE_EINVAL, "a must have 2 dimensions");
  if (w->dim() != 2 && w->dim() != 3) return fail(MOE_EINVAL, "w must have 3 dimensions, or 2 for one expert");
  const int dev = device_of("a", *a);
  if (dev < 0) return nullptr;
  const int one = w->dim() == 2;  // shapes without the experts' dimension
  const int64_t rows = a->size(0), K = a->size(1), E = one ? 1 : w->size(0), N = w->size(1 - one);
  const int64_t w_shape[3] = {E, N, K}, s_shape[3] = {E, blocks(N), blocks(K)};
  void *pa, *ps, *pw, *pv, *po, *ph = nullptr, *pe = nullptr, *pt = nullptr, *stream;
  if (!arg2("a", v[1], kFp8, rows, K, dev, &pa) || !arg2("a_scales", v[2], kF32, rows, blocks(K), dev, &ps) ||
      !arg("w", v[3], kFp8, 3 - one, w_shape + one, dev, &pw) ||
      !arg("w_scales", v[4], kF32, 3 - one, s_shape + one, dev, &pv))
    return nullptr;
  if (v[7] != Py_None && !arg1("expert_offsets", v[7], kI32, E + 1, dev, &pe)) return nullptr;
  if (v[8] != Py_None && !arg1("status", v[8], kI32, 1, dev, &pt)) return nullptr;
  if (!stream_of(v[9], &stream) || !fits("K", K) || !fits("N", N) || !fits("E", E)) return nullptr;
  const int32_t k = static_cast<int32_t>(K), experts = static_cast<int32_t>(E);
  if (glu) {
    if (N % (2 * MOE_FP8_BLOCK) != 0)
      return fail(MOE_EINVAL, "w13 has %lld rows, must be twice a multiple of %d", static_cast<long long>(N),
                  MOE_FP8_BLOCK);
    if (!arg2("hq", v[5], kFp8, rows, N / 2, dev, &po) ||
        !arg2("h_scales", v[6], kF32, rows, N / 2 / MOE_FP8_BLOCK, dev, &ph))
      return nullptr;
    return call("moe_expert_glu_fp8", [&] {
      return moe_expert_glu_fp8(pa, static_cast<float*>(ps), rows, k, pw, static_cast<float*>(pv),
                                static_cast<int32_t>(N / 2), experts, static_cast<int32_t*>(pe), po,
                                static_cast<float*>(ph), static_cast<int32_t*>(pt), stream);
    });
  }
  if (!arg2("out", v[5], kFloat, rows, N, dev, &po)) return nullptr;
  const int type = THPVariable_Unpack(v[5]).scalar_type() == at::ScalarType::Float ? MOE_TYPE_F32 : MOE_TYPE_BF16;
  return call("moe_expert_gemm_fp8", [&] {
    return moe_expert_gemm_fp8(pa, static_cast<float*>(ps), rows, k, pw, static_cast<float*>(pv),
                               static_cast<int32_t>(N), experts, static_cast<int32_t*>(pe), po, type,
                               static_cast<int32_t*>(pt), stream);
  });
}

// What DecodeLayer keeps, packed by Python's struct ("6i3Q").
struct Plan {
  int32_t max_tokens, H, K, E, I, device;
  uint64_t status, workspace, workspace_bytes;
};

// Whether the tuple (w13, w13_scales, w2, w2_scales) is what DecodeLayer takes; the addresses.
bool weights(PyObject* tuple, int64_t E, int64_t H, int64_t I, int device, void** at) {
  if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != 4) {
    PyErr_SetString(PyExc_TypeError, "weights must be a tuple of four tensors");
    return false;
  }
  const int64_t w13[3] = {E, 2 * I, H}, s13[3] = {E, blocks(2 * I), blocks(H)};
  const int64_t w2[3] = {E, H, I}, s2[3] = {E, blocks(H), blocks(I)};
  return arg("w13", PyTuple_GET_ITEM(tuple, 0), kFp8, 3, w13, device, at) &&
         arg("w13_scales", PyTuple_GET_ITEM(tuple, 1), kF32, 3, s13, device, at + 1) &&
         arg("w2", PyTuple_GET_ITEM(tuple, 2), kFp8, 3, w2, device, at + 2) &&
         arg("w2_scales", PyTuple_GET_ITEM(tuple, 3), kF32, 3, s2, device, at + 3);
}

// (plan, weights, xq, x_scales, topk_idx, topk_w, out, stream)
PyObject* decode_layer_fp8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 8)) return nullptr;
  if (!PyBytes_Check(v[0]) || PyBytes_GET_SIZE(v[0]) != static_cast<Py_ssize_t>(sizeof(Plan))) {
    PyErr_SetString(PyExc_TypeError, "plan must be packed as the module expects");
    return nullptr;
  }
  Plan p;
  std::memcpy(&p, PyBytes_AS_STRING(v[0]), sizeof p);
  const at::Tensor* x = tensor("xq", v[2]);
  if (!x) return nullptr;
  if (x->dim() != 2) return fail(MOE_EINVAL, "xq must have 2 dimensions");
  const int dev = device_of("xq", *x);
  if (dev < 0) return nullptr;
  const int64_t T = x->size(0);
  if (T > p.max_tokens || dev != p.device)
    return fail(MOE_EINVAL, "xq has %lld tokens on cuda:%d, must have at most %d on cuda:%d", static_cast<long long>(T),
                dev, p.max_tokens, p.device);
  void *px, *ps, *pi, *pw, *po, *w[4], *stream;
  if (!arg2("xq", v[2], kFp8, T, p.H, dev, &px) ||
      !arg2("x_scales", v[3], kF32, T, p.H / MOE_FP8_BLOCK, dev, &ps) ||
      !arg2("topk_idx", v[4], kI32, T, p.K, dev, &pi) || !arg2("topk_w", v[5], kF32, T, p.K, dev, &pw) ||
      !arg2("out", v[6], kBf16, T, p.H, dev, &po) || !weights(v[1], p.E, p.H, p.I, dev, w) ||
      !stream_of(v[7], &stream))
    return nullptr;
  const moe_config cfg = {static_cast<int32_t>(T), p.H, p.K, p.E, 1};
  auto at = [](uint64_t address) { return reinterpret_cast<void*>(address); };
  return call("moe_decode_layer_fp8", [&] {
    return moe_decode_layer_fp8(&cfg, p.I, px, static_cast<float*>(ps), static_cast<int32_t*>(pi),
                                static_cast<float*>(pw), w[0], static_cast<float*>(w[1]), w[2],
                                static_cast<float*>(w[3]), po, static_cast<int32_t*>(at(p.status)), at(p.workspace),
                                p.workspace_bytes, stream);
  });
}

// (weights, E, H, I, device): refuses weights that DecodeLayer does not take.
PyObject* check_weights(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  int64_t size[4];
  for (int i = 0; i < 4; ++i) {
    size[i] = PyLong_AsLongLong(v[1 + i]);
    if (size[i] == -1 && PyErr_Occurred()) return nullptr;
  }
  void* at[4];
  if (!weights(v[0], size[0], size[1], size[2], static_cast<int>(size[3]), at)) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"init", init, METH_O, "Sets the error class."},
    {"add_rms_norm_fp8", fast<add_rms_norm_fp8>(), METH_FASTCALL, nullptr},
    {"expert_product", fast<expert_product>(), METH_FASTCALL, nullptr},
    {"decode_layer_fp8", fast<decode_layer_fp8>(), METH_FASTCALL, nullptr},
    {"check_weights", fast<check_weights>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ffn", "Argument checks and calls of ffn.py.", -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__ffn() { return PyModule_Create(&kModule); }

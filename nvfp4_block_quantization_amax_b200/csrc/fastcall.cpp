// fastcall.cpp -- the host path of the small calls, in C++.
//
// Routing, dispatch, combine and the few-row products take 3 to 8 us on the
// GPU at a few tokens.  Around the call of the C ABI Python took longer: 9 to
// 11 us a call (checks, two or three new tensors, a dozen arguments converted).
// Here the whole call takes 3.9 to 5.4 us, 2.7 of them the launch (routing 64
// tokens 10.5 -> 5.1 us per pass, dispatch 11.1 -> 5.0, combine 9.7 -> 4.8).
// These functions take the same arguments as api.py's, in order, check them,
// allocate the results and call the library.  They answer
//   a tuple      the call was made: its results
//   a number     the library's status, where it is not NVFP4_OK
//   None         something is not as expected (a type, a shape, a device that
//                is not the current one, no tokens): nothing was done, and
//                api.py's own checks say what is wrong or make the call.
// So every condition here is at least as strict as api.py's, which makes all the
// calls where this file is not built for the torch and the Python at hand.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "nvfp4.h"

namespace {

decltype(&nvfp4_route) g_route;
decltype(&nvfp4_route_backward) g_route_backward;
decltype(&nvfp4_dispatch) g_dispatch;
decltype(&nvfp4_combine) g_combine;
decltype(&nvfp4_combine_backward) g_combine_backward;
decltype(&nvfp4_gemv) g_gemv;

constexpr auto kInt = at::kInt;
constexpr auto kFloat = at::kFloat;
constexpr auto kBF16 = at::kBFloat16;

PyObject* decline() { Py_RETURN_NONE; }

// The arguments of one call.  ok turns false where one is not as expected.
struct Call {
  PyObject* const* args;
  bool ok = true;
  int device = -1;

  const at::Tensor* tensor(int i, at::ScalarType type) {
    if (!THPVariable_Check(args[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.scalar_type() != type || t.layout() != at::kStrided) return fail();
    if (device < 0) device = t.get_device();
    return t.get_device() == device ? &t : fail();
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  bool given(int i) const { return args[i] != Py_None; }
  // contiguous, of at least n values
  const at::Tensor* flat(int i, at::ScalarType type, int64_t n) {
    const at::Tensor* t = tensor(i, type);
    return t && t->is_contiguous() && t->numel() >= n ? t : fail();
  }
  // contiguous [rows, cols]
  const at::Tensor* pairs(int i, at::ScalarType type, int64_t rows, int64_t cols) {
    const at::Tensor* t = flat(i, type, 0);
    return t && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols ? t : fail();
  }
  // bf16 [rows, cols] with unit column stride
  const at::Tensor* rows(int i, int64_t n, int64_t cols) {
    const at::Tensor* t = tensor(i, kBF16);
    return t && t->dim() == 2 && t->size(0) == n && t->size(1) == cols && t->stride(1) == 1 ? t : fail();
  }
  int64_t number(int i) {
    if (!PyLong_CheckExact(args[i])) {
      ok = false;
      return 0;
    }
    const long long v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int32_t* status(int i) {
    if (!given(i)) return nullptr;
    const at::Tensor* t = flat(i, kInt, 1);
    return t ? t->data_ptr<int32_t>() : nullptr;
  }
  // On the device that is current (it is, where ok stays true).
  void here() { ok = ok && device >= 0 && c10::cuda::current_device() == device; }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
  at::Tensor make(int64_t rows, int64_t cols, at::ScalarType type) const {
    return at::detail::empty_strided_cuda({rows, cols}, {cols, 1}, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
  }
};

int64_t stride_of(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// args[i] where a tensor was given, else the new one.
PyObject* result(const Call& c, int i, const at::Tensor& made) {
  if (!c.given(i)) return THPVariable_Wrap(made);
  Py_INCREF(c.args[i]);
  return c.args[i];
}

template <typename F>
PyObject* answer(nvfp4_status_t st, F results) {
  return st == NVFP4_OK ? results() : PyLong_FromLong(st);
}

// [rows, cols] logits, fp32 or bf16, unit column stride.
const at::Tensor* logits_of(Call& c, int i, int* dtype) {
  if (!THPVariable_Check(c.args[i])) return c.fail();
  const at::ScalarType type = THPVariable_Unpack(c.args[i]).scalar_type();
  if (type != kFloat && type != kBF16) return c.fail();
  *dtype = type == kFloat ? NVFP4_OUT_DTYPE_FP32 : NVFP4_OUT_DTYPE_BF16;
  const at::Tensor* t = c.tensor(i, type);
  return t && t->dim() == 2 && t->size(0) > 0 && t->size(1) > 0 && t->stride(1) == 1 ? t : c.fail();
}

// C++ exceptions (an allocation that fails, say) become torch's in Python.
template <PyObject* (*f)(Call&)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t) {
  HANDLE_TH_ERRORS
  Call c{args};
  return f(c);
  END_HANDLE_TH_ERRORS
}

// Allocations and launches may wait (for memory, for a full queue): other
// Python threads run meanwhile.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// (logits, k, score, flags, bias, groups, groups_kept, scale, ids, weights, status)
PyObject* route(Call& c) {
  int dtype = 0;
  const at::Tensor* z = logits_of(c, 0, &dtype);
  if (!z) return decline();
  const int64_t T = z->size(0), E = z->size(1), k = c.number(1), score = c.number(2), flags = c.number(3);
  const int64_t groups = c.number(5), kept = c.number(6);
  if (!c.ok || k < 1 || k > 32 || flags < 0 || flags > 255 || score < 0 || score > 255 || !PyFloat_CheckExact(c.args[7])) return decline();
  const at::Tensor* bias = c.given(4) ? c.flat(4, kFloat, E) : nullptr;
  const at::Tensor* ids = c.given(8) ? c.pairs(8, kInt, T, k) : nullptr;
  const at::Tensor* weights = c.given(9) ? c.pairs(9, kFloat, T, k) : nullptr;
  int32_t* const status = c.status(10);
  c.here();
  if (!c.ok) return decline();
  at::Tensor new_ids, new_weights;
  nvfp4_status_t st;
  {
    const Unlocked unlocked;
    if (!ids) new_ids = c.make(T, k, kInt);
    if (!weights) new_weights = c.make(T, k, kFloat);
    st = g_route(z->data_ptr(), stride_of(*z), dtype, bias ? bias->data_ptr<float>() : nullptr, T, E, k, groups, kept,
                 static_cast<int>(score), static_cast<uint32_t>(flags), static_cast<float>(PyFloat_AS_DOUBLE(c.args[7])),
                 (ids ? *ids : new_ids).data_ptr<int32_t>(), (weights ? *weights : new_weights).data_ptr<float>(), status, c.stream());
  }
  return answer(st, [&] { return Py_BuildValue("(NN)", result(c, 8, new_ids), result(c, 9, new_weights)); });
}

// (dweights, ids, logits, score, flags, scale, out, status)
PyObject* route_backward(Call& c) {
  int dtype = 0;
  const at::Tensor* z = logits_of(c, 2, &dtype);
  const at::Tensor* ids = z ? c.flat(1, kInt, 0) : nullptr;
  if (!ids || ids->dim() != 2 || ids->size(0) != z->size(0)) return decline();
  const int64_t T = z->size(0), E = z->size(1), k = ids->size(1), score = c.number(3), flags = c.number(4);
  const at::Tensor* dw = c.pairs(0, kFloat, T, k);
  const at::Tensor* out = nullptr;
  if (c.given(6)) {
    out = c.tensor(6, z->scalar_type());
    if (!out || out->dim() != 2 || out->size(0) != T || out->size(1) != E || out->stride(1) != 1) return decline();
  }
  int32_t* const status = c.status(7);
  c.here();
  if (!c.ok || flags < 0 || flags > 255 || score < 0 || score > 255 || !PyFloat_CheckExact(c.args[5])) return decline();
  at::Tensor made;
  nvfp4_status_t st;
  {
    const Unlocked unlocked;
    if (!out) made = c.make(T, E, z->scalar_type());
    st = g_route_backward(dw->data_ptr<float>(), ids->data_ptr<int32_t>(), z->data_ptr(), stride_of(*z), dtype, T, E, k,
                          static_cast<int>(score), static_cast<uint32_t>(flags), static_cast<float>(PyFloat_AS_DOUBLE(c.args[5])),
                          (out ? *out : made).data_ptr(), stride_of(out ? *out : made), status, c.stream());
  }
  return answer(st, [&] { return Py_BuildValue("(N)", result(c, 6, made)); });
}

// (x, ids, E, out, rows, offsets, status)
PyObject* dispatch(Call& c) {
  const at::Tensor* ids = c.flat(1, kInt, 1);
  const int64_t E = c.number(2);
  if (!c.ok || ids->dim() != 2 || E < 1 || E > 1024) return decline();
  const int64_t T = ids->size(0), k = ids->size(1);
  int64_t C = 8;
  const at::Tensor *x = nullptr, *out = nullptr;
  if (c.given(0)) {
    x = c.tensor(0, kBF16);
    if (!x || x->dim() != 2) return decline();
    C = x->size(1);
    x = c.rows(0, T, C);
    if (c.given(3)) out = c.rows(3, T * k, C);
  } else if (c.given(3)) {
    return decline();
  }
  const at::Tensor* rows = c.given(4) ? c.pairs(4, kInt, T, k) : nullptr;
  const at::Tensor* offsets = c.given(5) ? c.flat(5, kInt, E + 1) : nullptr;
  int32_t* const status = c.status(6);
  c.here();
  if (!c.ok) return decline();
  at::Tensor new_out, new_rows, new_offsets;
  nvfp4_status_t st;
  {
    const Unlocked unlocked;
    if (!rows) new_rows = c.make(T, k, kInt);
    if (!offsets)
      new_offsets = at::detail::empty_strided_cuda({E + 1}, {1}, kInt, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
    if (x && !out) new_out = c.make(T * k, C, kBF16);
    const at::Tensor& xs = out ? *out : new_out;
    st = g_dispatch(x ? x->data_ptr() : nullptr, x ? stride_of(*x) : C, ids->data_ptr<int32_t>(), T, k, E, C,
                    x ? xs.data_ptr() : nullptr, x ? stride_of(xs) : C,
                    (offsets ? *offsets : new_offsets).data_ptr<int32_t>(),
                    (rows ? *rows : new_rows).data_ptr<int32_t>(), status, c.stream());
  }
  return answer(st, [&] {
    PyObject* first = nullptr;
    if (x) first = result(c, 3, new_out);
    else Py_INCREF(first = Py_None);
    return Py_BuildValue("(NNN)", first, result(c, 4, new_rows), result(c, 5, new_offsets));
  });
}

// Shape of the pairs: that of rows (i) and weights (j), one of which is given.
bool pairs_of(Call& c, int i, int j, const at::Tensor** rows, const at::Tensor** weights, int64_t* T, int64_t* k) {
  *rows = c.given(i) ? c.flat(i, kInt, 1) : nullptr;
  *weights = c.given(j) ? c.flat(j, kFloat, 1) : nullptr;
  const at::Tensor* t = *rows ? *rows : *weights;
  if (!c.ok || !t || t->dim() != 2 || (*rows && *weights && (*rows)->sizes() != (*weights)->sizes())) return false;
  *T = t->size(0);
  *k = t->size(1);
  return true;
}

// (y, rows, weights, residual, out, status)
PyObject* combine(Call& c) {
  const at::Tensor* y = c.tensor(0, kBF16);
  const at::Tensor *rows = nullptr, *weights = nullptr;
  int64_t T = 0, k = 0;
  if (!y || y->dim() != 2 || y->size(0) < 1 || y->stride(1) != 1 || !pairs_of(c, 1, 2, &rows, &weights, &T, &k)) return decline();
  const int64_t R = y->size(0), C = y->size(1);
  const at::Tensor* residual = c.given(3) ? c.rows(3, T, C) : nullptr;
  const at::Tensor* out = c.given(4) ? c.rows(4, T, C) : nullptr;
  int32_t* const status = c.status(5);
  c.here();
  if (!c.ok) return decline();
  at::Tensor made;
  nvfp4_status_t st;
  {
    const Unlocked unlocked;
    if (!out) made = c.make(T, C, kBF16);
    st = g_combine(y->data_ptr(), stride_of(*y), R, rows ? rows->data_ptr<int32_t>() : nullptr,
                   weights ? weights->data_ptr<float>() : nullptr, T, k, C, residual ? residual->data_ptr() : nullptr,
                   residual ? stride_of(*residual) : 0, (out ? *out : made).data_ptr(), stride_of(out ? *out : made), status, c.stream());
  }
  return answer(st, [&] { return Py_BuildValue("(N)", result(c, 4, made)); });
}

// (dout, rows, weights, y, need_dy, need_dweights, out, status)
PyObject* combine_backward(Call& c) {
  const at::Tensor* dout = c.tensor(0, kBF16);
  const at::Tensor *rows = nullptr, *weights = nullptr;
  int64_t T = 0, k = 0;
  if (!dout || dout->dim() != 2 || !pairs_of(c, 1, 2, &rows, &weights, &T, &k)) return decline();
  const int64_t C = dout->size(1);
  dout = c.rows(0, T, C);
  const at::Tensor* y = c.tensor(3, kBF16);
  if (!c.ok || y->dim() != 2 || y->size(0) < 1) return decline();
  const int64_t R = y->size(0);
  y = c.rows(3, R, C);
  const bool need_dy = c.args[4] == Py_True, need_dw = c.args[5] == Py_True;
  if (!PyBool_Check(c.args[4]) || !PyBool_Check(c.args[5]) || (c.given(6) && !need_dy)) return decline();
  const at::Tensor* out = c.given(6) ? c.rows(6, R, C) : nullptr;
  int32_t* const status = c.status(7);
  c.here();
  if (!c.ok) return decline();
  at::Tensor made, dw;
  nvfp4_status_t st;
  {
    const Unlocked unlocked;
    if (need_dy && !out) made = c.make(R, C, kBF16);
    if (need_dw) dw = c.make(T, k, kFloat);
    const at::Tensor& dy = out ? *out : made;
    st = g_combine_backward(dout->data_ptr(), stride_of(*dout), y->data_ptr(), stride_of(*y), R,
                            rows ? rows->data_ptr<int32_t>() : nullptr, weights ? weights->data_ptr<float>() : nullptr, T, k, C,
                            need_dy ? dy.data_ptr() : nullptr, need_dy ? stride_of(dy) : C, need_dw ? dw.data_ptr<float>() : nullptr,
                            status, c.stream());
  }
  return answer(st, [&] {
    PyObject *a = nullptr, *b = nullptr;
    if (need_dy) a = result(c, 6, made);
    else Py_INCREF(a = Py_None);
    if (need_dw) b = THPVariable_Wrap(dw);
    else Py_INCREF(b = Py_None);
    return Py_BuildValue("(NN)", a, b);
  });
}

// (x, W, sW, alphaW, ids, out_dtype, out, status)
PyObject* gemv(Call& c) {
  const at::Tensor* x = c.tensor(0, kBF16);
  const at::Tensor* W = c.flat(1, at::kByte, 1);
  const int64_t kind = c.number(5);
  if (!c.ok || x->dim() != 2 || (kind != NVFP4_OUT_DTYPE_BF16 && kind != NVFP4_OUT_DTYPE_FP32)) return decline();
  const int64_t X = x->size(0), K = x->size(1);
  x = c.rows(0, X, K);
  const bool by_id = c.given(4);
  if (X < 1 || W->dim() != (by_id ? 3 : 2) || 2 * W->size(-1) != K) return decline();
  const int64_t N = W->size(-2), E = by_id ? W->size(0) : 1;
  int64_t P = X, rep = 1;
  const at::Tensor* ids = nullptr;
  if (by_id) {
    ids = c.flat(4, kInt, 1);
    if (!ids || ids->dim() != 2) return decline();
    P = ids->size(0) * ids->size(1);
    if (X == ids->size(0)) rep = ids->size(1);
    else if (X != P) return decline();
  }
  if (P > 1024) return decline();   // before its results are allocated
  const at::Tensor* sW = c.flat(2, at::kByte, E * N * (K / 16));
  const at::Tensor* alpha = c.flat(3, kFloat, E);
  const at::ScalarType type = kind == NVFP4_OUT_DTYPE_FP32 ? kFloat : kBF16;
  const at::Tensor* out = nullptr;
  if (c.given(6)) {
    out = c.tensor(6, type);
    if (!out || out->dim() != 2 || out->size(0) < P || out->size(1) < N || out->stride(1) != 1) return decline();
  }
  int32_t* const status = c.status(7);
  c.here();
  if (!c.ok) return decline();
  at::Tensor made;
  nvfp4_status_t st;
  {
    const Unlocked unlocked;
    if (!out) made = c.make(P, N, type);
    st = g_gemv(x->data_ptr(), stride_of(*x), ids ? ids->data_ptr<int32_t>() : nullptr, P, rep, W->data_ptr<uint8_t>(),
                sW->data_ptr<uint8_t>(), alpha->data_ptr<float>(), E, N, K, (out ? *out : made).data_ptr(), static_cast<int>(kind),
                out && P > 1 ? out->stride(0) : N, status, c.stream());
  }
  return answer(st, [&] { return Py_BuildValue("(N)", result(c, 6, made)); });
}

// The library's entry points, by address: route, route_backward, dispatch,
// combine, combine_backward, gemv.
PyObject* use(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[6];
  for (Py_ssize_t i = 0; i < 6; ++i)
    if (n != 6 || !(p[i] = PyLong_AsVoidPtr(args[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "six addresses are needed");
      return nullptr;
    }
  g_route = reinterpret_cast<decltype(g_route)>(p[0]);
  g_route_backward = reinterpret_cast<decltype(g_route_backward)>(p[1]);
  g_dispatch = reinterpret_cast<decltype(g_dispatch)>(p[2]);
  g_combine = reinterpret_cast<decltype(g_combine)>(p[3]);
  g_combine_backward = reinterpret_cast<decltype(g_combine_backward)>(p[4]);
  g_gemv = reinterpret_cast<decltype(g_gemv)>(p[5]);
  Py_RETURN_NONE;
}

template <PyObject* (*f)(Call&), int count>
PyObject* entry(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  if (n != count || !g_gemv) return decline();
  return guarded<f>(self, args, n);
}
template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {{"use", fast(use), METH_FASTCALL, nullptr},
                         {"route", fast(entry<route, 11>), METH_FASTCALL, nullptr},
                         {"route_backward", fast(entry<route_backward, 8>), METH_FASTCALL, nullptr},
                         {"dispatch", fast(entry<dispatch, 7>), METH_FASTCALL, nullptr},
                         {"combine", fast(entry<combine, 6>), METH_FASTCALL, nullptr},
                         {"combine_backward", fast(entry<combine_backward, 8>), METH_FASTCALL, nullptr},
                         {"gemv", fast(entry<gemv, 8>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }

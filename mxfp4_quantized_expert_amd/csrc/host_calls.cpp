// Host side of the new entry points for a call that needs nothing special:
// the checks, the outputs and the C call in one step of native code.  A call of
// a few tokens is bound by its host time, and in Python the same steps take
// longer than the launch (9.4 against 5.0 us for a permute of four tokens).
//
// Every function takes the tensors of binding.py's function of that name and
// returns its outputs, or None for a call that is not as expected (a type, a
// shape, a stride, another device than the current one, a status): binding.py
// then makes it step by step and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxfp4moe.h"

namespace {

PyObject* g_raw_stream = nullptr;  // torch's function: device index -> current stream's handle

// The tensors of one call, all on one device.
struct Call {
  int device = -1;
  bool ok = true;

  // argument o as a contiguous device tensor of this type and shape
  const at::Tensor& tensor(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& t = any(o);
    ok = ok && t.scalar_type() == type && t.sizes() == shape;
    return t;
  }
  const at::Tensor& any(PyObject* o) {
    if (!ok || !THPVariable_Check(o)) {
      ok = false;
      return dummy();
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) {
      ok = false;
      return dummy();
    }
    if (device < 0) device = t.get_device();
    ok = device == t.get_device();
    return ok ? t : dummy();
  }
  // the current stream of the current device, which has to be the tensors'
  void* stream() {
    static const c10::impl::VirtualGuardImpl guard(c10::DeviceType::CUDA);
    // (under a mode that looks at torch's calls, or one that fills new tensors, outputs are torch's to make)
    if (!ok || guard.getDevice().index() != device || c10::impl::TorchDispatchModeTLS::any_modes_set() ||
        (at::globalContext().deterministicAlgorithms() && at::globalContext().deterministicFillUninitializedMemory())) {
      ok = false;
      return nullptr;
    }
    PyObject* index = PyLong_FromLong(device);
    PyObject* s = PyObject_CallOneArg(g_raw_stream, index);
    Py_DECREF(index);
    if (s == nullptr) {
      PyErr_Clear();
      ok = false;
      return nullptr;
    }
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return p;
  }

 private:
  // what stands in for an argument that does not fit: outlives the runtime's end, and so the mode of this call
  static const at::Tensor& dummy() {
    static const at::Tensor& t = *new at::Tensor(at::detail::empty_cpu({0, 0}, at::kFloat));
    return t;
  }
};

// A new tensor of like's type, on its device, without the way through the dispatcher (0.3 us each).
at::Tensor fresh(at::IntArrayRef shape, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, like.scalar_type(), like.device(), std::nullopt));
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

int element_type(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MXFP4MOE_BF16;
    case at::kHalf: return MXFP4MOE_F16;
    case at::kFloat: return MXFP4MOE_F32;
    default: return -1;
  }
}

// A 2-d tensor of a row type.
const at::Tensor& rows_of(Call& c, PyObject* o, int& type) {
  const at::Tensor& t = c.any(o);
  type = element_type(t);
  c.ok = c.ok && type >= 0 && t.dim() == 2;
  return t;
}

bool small_int(PyObject* o, int64_t& v) {
  if (!PyLong_Check(o)) return false;
  v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) PyErr_Clear();
  return v > 0 && v < ((int64_t)1 << 31);
}

bool number(PyObject* o, float& v) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  v = (float)PyFloat_AsDouble(o);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// A flag, or an argument for the longer way.
bool truth(PyObject* o, bool& v) {
  v = o == Py_True;
  return v || o == Py_False;
}

// The device pointer of an argument that may be None.
const void* optional(Call& c, PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
  return o == Py_None ? nullptr : c.tensor(o, type, shape).data_ptr();
}

template <typename F>
int unlocked(F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return st;
}

PyObject* result(int st, const at::Tensor& t) {
  if (st != MXFP4MOE_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* result(int st, const at::Tensor& a, const at::Tensor& b) {
  if (st != MXFP4MOE_OK) Py_RETURN_NONE;
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  PyObject* both = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
}

PyObject* result(int st, std::initializer_list<at::Tensor> all) {
  if (st != MXFP4MOE_OK) Py_RETURN_NONE;
  PyObject* both = PyTuple_New((Py_ssize_t)all.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& t : all) {
    PyObject* x = both != nullptr ? THPVariable_Wrap(t) : nullptr;
    if (x == nullptr) {
      Py_XDECREF(both);
      return nullptr;
    }
    PyTuple_SET_ITEM(both, i++, x);
  }
  return both;
}

// permute(x, sorted_pairs, top_k)
PyObject* permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  int64_t k;
  if (n != 3 || !small_int(a[2], k)) Py_RETURN_NONE;
  const at::Tensor& x = rows_of(c, a[0], type);
  const at::Tensor& pairs = c.any(a[1]);
  if (!c.ok || pairs.scalar_type() != at::kInt || pairs.dim() != 1) Py_RETURN_NONE;
  void* s = c.stream();
  const int64_t T = x.size(0), H = x.size(1), R = pairs.size(0);
  if (!c.ok || T > INT32_MAX / k) Py_RETURN_NONE;
  const at::Tensor rows = fresh({R, H}, x), at_row = fresh({T * k}, pairs);
  return result(unlocked([&] {
                  return moe_permute(x.data_ptr(), type, (const int32_t*)pairs.data_ptr(), T, H, k, R, rows.data_ptr(),
                                     (int32_t*)at_row.data_ptr(), s);
                }),
                rows, at_row);
  END_HANDLE_TH_ERRORS
}

// permute_backward(d_rows, pair_rows, top_k)
PyObject* permute_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  int64_t k;
  if (n != 3 || !small_int(a[2], k)) Py_RETURN_NONE;
  const at::Tensor& d = rows_of(c, a[0], type);
  const at::Tensor& at_row = c.any(a[1]);
  if (!c.ok || at_row.scalar_type() != at::kInt || at_row.dim() != 1 || at_row.size(0) % k != 0) Py_RETURN_NONE;
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const int64_t T = at_row.size(0) / k, H = d.size(1), R = d.size(0);
  const at::Tensor dx = fresh({T, H}, d);
  return result(unlocked([&] {
                  return moe_permute_backward(d.data_ptr(), type, (const int32_t*)at_row.data_ptr(), T, H, k, R,
                                              dx.data_ptr(), s);
                }),
                dx);
  END_HANDLE_TH_ERRORS
}

// unpermute(rows, pair_rows, topk_weights)
PyObject* unpermute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  if (n != 3) Py_RETURN_NONE;
  const at::Tensor& rows = rows_of(c, a[0], type);
  const at::Tensor& w = c.any(a[2]);
  if (!c.ok || w.scalar_type() != at::kFloat || w.dim() != 2) Py_RETURN_NONE;
  const int64_t T = w.size(0), k = w.size(1), H = rows.size(1), R = rows.size(0);
  const at::Tensor& at_row = c.tensor(a[1], at::kInt, {T * k});
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor y = fresh({T, H}, rows);
  return result(unlocked([&] {
                  return moe_unpermute(rows.data_ptr(), type, (const int32_t*)at_row.data_ptr(),
                                       (const float*)w.data_ptr(), T, H, k, R, y.data_ptr(), s);
                }),
                y);
  END_HANDLE_TH_ERRORS
}

// unpermute_backward(dy, rows, sorted_pairs, pair_rows, topk_weights)
PyObject* unpermute_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  if (n != 5) Py_RETURN_NONE;
  const at::Tensor& rows = rows_of(c, a[1], type);
  const at::Tensor& w = c.any(a[4]);
  if (!c.ok || w.scalar_type() != at::kFloat || w.dim() != 2) Py_RETURN_NONE;
  const int64_t T = w.size(0), k = w.size(1), H = rows.size(1), R = rows.size(0);
  const at::Tensor& dy = c.tensor(a[0], rows.scalar_type(), {T, H});
  const at::Tensor& pairs = c.tensor(a[2], at::kInt, {R});
  const at::Tensor& at_row = c.tensor(a[3], at::kInt, {T * k});
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor d_rows = fresh({R, H}, rows), dw = fresh({T, k}, w);
  return result(unlocked([&] {
                  return moe_unpermute_backward(dy.data_ptr(), rows.data_ptr(), type, (const int32_t*)pairs.data_ptr(),
                                                (const int32_t*)at_row.data_ptr(), (const float*)w.data_ptr(), T, H, k,
                                                R, d_rows.data_ptr(), (float*)dw.data_ptr(), s);
                }),
                d_rows, dw);
  END_HANDLE_TH_ERRORS
}

// route_backward(topk_ids, topk_weights, d_weights, num_experts)
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int64_t E;
  if (n != 4 || !small_int(a[3], E)) Py_RETURN_NONE;
  const at::Tensor& w = c.any(a[1]);
  if (!c.ok || w.scalar_type() != at::kFloat || w.dim() != 2) Py_RETURN_NONE;
  const int64_t T = w.size(0), k = w.size(1);
  const at::Tensor& ids = c.tensor(a[0], at::kInt, {T, k});
  const at::Tensor& dw = c.tensor(a[2], at::kFloat, {T, k});
  void* s = c.stream();
  if (!c.ok || E > MXFP4MOE_MAX_EXPERTS) Py_RETURN_NONE;
  const at::Tensor d = fresh({T, E}, w);
  return result(unlocked([&] {
                  return moe_route_backward((const int32_t*)ids.data_ptr(), (const float*)w.data_ptr(),
                                            (const float*)dw.data_ptr(), T, E, k, (float*)d.data_ptr(), s);
                }),
                d);
  END_HANDLE_TH_ERRORS
}

// linear(backward, group, rows, blocks, scales, scale2, bias, expert_offsets)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (n != 8) Py_RETURN_NONE;
  const bool backward = a[0] == Py_True;
  const int64_t group = PyLong_AsLong(a[1]);
  const bool grouped = a[7] != Py_None, nv = group == 16, biased = a[6] != Py_None;
  int type;
  const at::Tensor& rows = rows_of(c, a[2], type);
  const at::Tensor& blocks = c.any(a[3]);
  if (!c.ok || type != MXFP4MOE_BF16 || blocks.scalar_type() != at::kByte || blocks.dim() != (grouped ? 3 : 2))
    Py_RETURN_NONE;
  const int64_t E = grouped ? blocks.size(0) : 1, N = blocks.size(-2), K = 2 * blocks.size(-1), R = rows.size(0);
  const int64_t give = backward ? K : N;
  if (rows.size(1) != (backward ? N : K)) Py_RETURN_NONE;
  const at::Tensor& scales =
      grouped ? c.tensor(a[4], at::kByte, {E, N, K / group}) : c.tensor(a[4], at::kByte, {N, K / group});
  const float* scale2 = nv ? (const float*)c.tensor(a[5], at::kFloat, {E}).data_ptr() : nullptr;
  const uint16_t* bias = nullptr;
  if (biased)
    bias = (const uint16_t*)(grouped ? c.tensor(a[6], at::kBFloat16, {E, N}) : c.tensor(a[6], at::kBFloat16, {N}))
               .data_ptr();
  const int32_t* offsets = grouped ? (const int32_t*)c.tensor(a[7], at::kInt, {E + 1}).data_ptr() : nullptr;
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor out = fresh({R, give}, rows);
  const auto *x = (const uint16_t*)rows.data_ptr();
  const auto *b = (const uint8_t*)blocks.data_ptr(), *sc = (const uint8_t*)scales.data_ptr();
  auto* y = (uint16_t*)out.data_ptr();
  return result(unlocked([&] {
                  if (backward)
                    return nv ? moe_nvfp4_linear_backward(x, b, sc, scale2, offsets, R, K, N, E, y, s)
                              : moe_mxfp4_linear_backward(x, b, sc, offsets, R, K, N, E, y, s);
                  return nv ? moe_nvfp4_linear(x, b, sc, scale2, bias, offsets, R, K, N, E, y, s)
                            : moe_mxfp4_linear(x, b, sc, bias, offsets, R, K, N, E, y, s);
                }),
                out);
  END_HANDLE_TH_ERRORS
}

// A norm's weight: of the rows' type or float32.
const at::Tensor& weight_of(Call& c, PyObject* o, const at::Tensor& rows, int& type) {
  const at::Tensor& w = c.any(o);
  type = element_type(w);
  c.ok = c.ok && w.dim() == 1 && w.size(0) == rows.size(1) &&
         (w.scalar_type() == rows.scalar_type() || w.scalar_type() == at::kFloat);
  return w;
}

// rms_norm(x, weight, residual, eps, fp8)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type, wtype;
  float eps;
  bool fp8;
  if (n != 5 || !number(a[3], eps) || !truth(a[4], fp8)) Py_RETURN_NONE;
  const at::Tensor& x = rows_of(c, a[0], type);
  if (!c.ok) Py_RETURN_NONE;
  const int64_t T = x.size(0), H = x.size(1);
  const at::Tensor& w = weight_of(c, a[1], x, wtype);
  const void* residual = optional(c, a[2], x.scalar_type(), {T, H});
  void* s = c.stream();
  if (!c.ok || H < 1) Py_RETURN_NONE;
  const at::Tensor summed = a[2] != Py_None ? fresh({T, H}, x) : x, rstd = fresh({T}, at::kFloat, x);
  void* sum = a[2] != Py_None ? summed.data_ptr() : nullptr;
  auto* r = (float*)rstd.data_ptr();
  if (fp8) {
    const at::Tensor codes = fresh({T, H}, at::kFloat8_e4m3fn, x), scales = fresh({T, blocks_of(H)}, at::kFloat, x);
    return result(unlocked([&] {
                    return moe_rms_norm_fp8(x.data_ptr(), residual, w.data_ptr(), type, wtype, eps, T, H, sum,
                                            (uint8_t*)codes.data_ptr(), (float*)scales.data_ptr(), r, s);
                  }),
                  {codes, scales, summed, rstd});
  }
  const at::Tensor y = fresh({T, H}, x);
  return result(unlocked([&] {
                  return moe_rms_norm(x.data_ptr(), residual, w.data_ptr(), type, wtype, eps, T, H, sum, y.data_ptr(),
                                      r, s);
                }),
                {y, summed, rstd});
  END_HANDLE_TH_ERRORS
}

// rms_norm_backward(dy, summed, weight, rstd, d_summed)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type, wtype;
  if (n != 5) Py_RETURN_NONE;
  const at::Tensor& dy = rows_of(c, a[0], type);
  if (!c.ok) Py_RETURN_NONE;
  const int64_t T = dy.size(0), H = dy.size(1);
  const at::Tensor& summed = c.tensor(a[1], dy.scalar_type(), {T, H});
  const at::Tensor& w = weight_of(c, a[2], dy, wtype);
  const at::Tensor& rstd = c.tensor(a[3], at::kFloat, {T});
  const void* d_summed = optional(c, a[4], dy.scalar_type(), {T, H});
  void* s = c.stream();
  size_t bytes = 0;
  if (!c.ok || moe_rms_norm_backward(nullptr, nullptr, nullptr, nullptr, type, wtype, nullptr, T, H, nullptr, nullptr,
                                     nullptr, &bytes, nullptr) != MXFP4MOE_OK)
    Py_RETURN_NONE;
  const at::Tensor dx = fresh({T, H}, dy), dw = fresh({H}, at::kFloat, dy);
  const at::Tensor ws = fresh({(int64_t)bytes + 1}, at::kByte, dy);
  return result(unlocked([&] {
                  return moe_rms_norm_backward(dy.data_ptr(), d_summed, summed.data_ptr(), w.data_ptr(), type, wtype,
                                               (const float*)rstd.data_ptr(), T, H, dx.data_ptr(),
                                               (float*)dw.data_ptr(), ws.data_ptr(), &bytes, s);
                }),
                {dx, dw});
  END_HANDLE_TH_ERRORS
}

// fp8_quantize(x)
PyObject* fp8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  if (n != 1) Py_RETURN_NONE;
  const at::Tensor& x = rows_of(c, a[0], type);
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const int64_t R = x.size(0), K = x.size(1);
  const at::Tensor codes = fresh({R, K}, at::kFloat8_e4m3fn, x), scales = fresh({R, blocks_of(K)}, at::kFloat, x);
  return result(unlocked([&] {
                  return moe_fp8_quantize(x.data_ptr(), type, R, K, (uint8_t*)codes.data_ptr(),
                                          (float*)scales.data_ptr(), s);
                }),
                {codes, scales});
  END_HANDLE_TH_ERRORS
}

// The weights, scales, offsets and bias (nullptr: none wanted) of an 8-bit linear operator.
struct Fp8Weights {
  int64_t E = 1, N = 0, K = 0;
  const uint8_t* w = nullptr;
  const float* scales = nullptr;
  const int32_t* offsets = nullptr;
  const uint16_t* bias = nullptr;
  Fp8Weights(Call& c, PyObject* weight, PyObject* weight_scales, PyObject* o, PyObject* b) {
    const bool grouped = o != Py_None;
    const at::Tensor& t = c.any(weight);
    c.ok = c.ok && t.scalar_type() == at::kFloat8_e4m3fn && t.dim() == (grouped ? 3 : 2);
    if (!c.ok) return;
    if (grouped) E = t.size(0);
    N = t.size(-2);
    K = t.size(-1);
    w = (const uint8_t*)t.data_ptr();
    const int64_t nb = blocks_of(N), kb = blocks_of(K);
    scales = (const float*)(grouped ? c.tensor(weight_scales, at::kFloat, {E, nb, kb})
                                    : c.tensor(weight_scales, at::kFloat, {nb, kb}))
                 .data_ptr();
    if (grouped) offsets = (const int32_t*)c.tensor(o, at::kInt, {E + 1}).data_ptr();
    if (b != nullptr && b != Py_None)
      bias = (const uint16_t*)(grouped ? c.tensor(b, at::kBFloat16, {E, N}) : c.tensor(b, at::kBFloat16, {N})).data_ptr();
  }
};

// fp8_linear(x, x_scales, weight, weight_scales, bias, expert_offsets)
PyObject* fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  if (n != 6) Py_RETURN_NONE;
  const at::Tensor& x = c.any(a[0]);
  if (!c.ok || x.scalar_type() != at::kFloat8_e4m3fn || x.dim() != 2) Py_RETURN_NONE;
  const Fp8Weights w(c, a[2], a[3], a[5], a[4]);
  const int64_t R = x.size(0);
  const at::Tensor& xs = c.tensor(a[1], at::kFloat, {R, blocks_of(w.K)});
  void* s = c.stream();
  if (!c.ok || x.size(1) != w.K) Py_RETURN_NONE;
  const at::Tensor y = fresh({R, w.N}, at::kBFloat16, x);
  return result(unlocked([&] {
                  return moe_fp8_linear((const uint8_t*)x.data_ptr(), (const float*)xs.data_ptr(), w.w, w.scales,
                                        w.bias, w.offsets, R, w.K, w.N, w.E, (uint16_t*)y.data_ptr(), s);
                }),
                y);
  END_HANDLE_TH_ERRORS
}

// fp8_linear_backward(dy, weight, weight_scales, expert_offsets)
PyObject* fp8_linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  if (n != 4) Py_RETURN_NONE;
  const at::Tensor& dy = rows_of(c, a[0], type);
  if (!c.ok || type != MXFP4MOE_BF16) Py_RETURN_NONE;
  const Fp8Weights w(c, a[1], a[2], a[3], nullptr);
  void* s = c.stream();
  if (!c.ok || dy.size(1) != w.N) Py_RETURN_NONE;
  const int64_t R = dy.size(0);
  const at::Tensor dx = fresh({R, w.K}, dy);
  return result(unlocked([&] {
                  return moe_fp8_linear_backward((const uint16_t*)dy.data_ptr(), w.w, w.scales, w.offsets, R, w.K, w.N,
                                                 w.E, (uint16_t*)dx.data_ptr(), s);
                }),
                dx);
  END_HANDLE_TH_ERRORS
}

// swiglu(h, split, alpha, limit, offset, fp8)
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  float alpha, limit, offset;
  bool split, fp8;
  if (n != 6 || !truth(a[1], split) || !number(a[2], alpha) || !number(a[3], limit) || !number(a[4], offset) ||
      !truth(a[5], fp8))
    Py_RETURN_NONE;
  const at::Tensor& h = rows_of(c, a[0], type);
  void* s = c.stream();
  if (!c.ok || h.size(1) % 2 != 0) Py_RETURN_NONE;
  const int64_t R = h.size(0), I = h.size(1) / 2;
  if (fp8) {
    const at::Tensor codes = fresh({R, I}, at::kFloat8_e4m3fn, h), scales = fresh({R, blocks_of(I)}, at::kFloat, h);
    return result(unlocked([&] {
                    return moe_swiglu_fp8(h.data_ptr(), type, R, I, alpha, limit, offset, split,
                                          (uint8_t*)codes.data_ptr(), (float*)scales.data_ptr(), s);
                  }),
                  {codes, scales});
  }
  const at::Tensor out = fresh({R, I}, h);
  return result(unlocked([&] {
                  return moe_swiglu(h.data_ptr(), type, R, I, alpha, limit, offset, split, out.data_ptr(), s);
                }),
                out);
  END_HANDLE_TH_ERRORS
}

// swiglu_backward(da, h, split, alpha, limit, offset)
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  float alpha, limit, offset;
  bool split;
  if (n != 6 || !truth(a[2], split) || !number(a[3], alpha) || !number(a[4], limit) || !number(a[5], offset))
    Py_RETURN_NONE;
  const at::Tensor& h = rows_of(c, a[1], type);
  if (!c.ok || h.size(1) % 2 != 0) Py_RETURN_NONE;
  const int64_t R = h.size(0), I = h.size(1) / 2;
  const at::Tensor& da = c.tensor(a[0], h.scalar_type(), {R, I});
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor dh = fresh({R, 2 * I}, h);
  return result(unlocked([&] {
                  return moe_swiglu_backward(da.data_ptr(), h.data_ptr(), type, R, I, alpha, limit, offset, split,
                                             dh.data_ptr(), s);
                }),
                dh);
  END_HANDLE_TH_ERRORS
}

// balance_loss(router_logits, topk_ids, token_mask)
PyObject* balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  if (n != 3) Py_RETURN_NONE;
  const at::Tensor& logits = rows_of(c, a[0], type);
  const at::Tensor& ids = c.any(a[1]);
  if (!c.ok || type != MXFP4MOE_F32 || ids.scalar_type() != at::kInt || ids.dim() != 2 ||
      ids.size(0) != logits.size(0))
    Py_RETURN_NONE;
  const int64_t T = logits.size(0), E = logits.size(1), k = ids.size(1);
  const auto* mask = (const uint8_t*)optional(c, a[2], at::kBool, {T});
  void* s = c.stream();
  size_t bytes = 0;
  if (!c.ok || moe_balance_loss(nullptr, nullptr, nullptr, T, E, k, nullptr, nullptr, nullptr, nullptr, &bytes,
                                nullptr) != MXFP4MOE_OK)
    Py_RETURN_NONE;
  const at::Tensor loss = fresh({}, logits), counts = fresh({E}, ids), density = fresh({E}, logits);
  const at::Tensor ws = bytes > 0 ? fresh({(int64_t)bytes}, at::kByte, logits) : loss;  // any pointer, for none
  return result(unlocked([&] {
                  return moe_balance_loss((const float*)logits.data_ptr(), (const int32_t*)ids.data_ptr(), mask, T, E,
                                          k, (float*)loss.data_ptr(), (int32_t*)counts.data_ptr(),
                                          (float*)density.data_ptr(), ws.data_ptr(), &bytes, s);
                }),
                {loss, counts, density});
  END_HANDLE_TH_ERRORS
}

// balance_loss_backward(router_logits, density, d_loss, token_mask, add_to)
PyObject* balance_loss_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  int type;
  if (n != 5) Py_RETURN_NONE;
  const at::Tensor& logits = rows_of(c, a[0], type);
  const at::Tensor& d_loss = c.any(a[2]);
  if (!c.ok || type != MXFP4MOE_F32 || d_loss.scalar_type() != at::kFloat || d_loss.numel() != 1) Py_RETURN_NONE;
  const int64_t T = logits.size(0), E = logits.size(1);
  const at::Tensor& density = c.tensor(a[1], at::kFloat, {E});
  const auto* mask = (const uint8_t*)optional(c, a[3], at::kBool, {T});
  const auto* add = (const float*)optional(c, a[4], at::kFloat, {T, E});
  void* s = c.stream();
  if (!c.ok) Py_RETURN_NONE;
  const at::Tensor d = fresh({T, E}, logits);
  return result(unlocked([&] {
                  return moe_balance_loss_backward((const float*)logits.data_ptr(), (const float*)density.data_ptr(),
                                                   (const float*)d_loss.data_ptr(), mask, add, T, E,
                                                   (float*)d.data_ptr(), s);
                }),
                d);
  END_HANDLE_TH_ERRORS
}

#define MX_CALL(NAME) {#NAME, (PyCFunction)(void (*)(void))NAME, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MX_CALL(permute), MX_CALL(permute_backward), MX_CALL(unpermute), MX_CALL(unpermute_backward),
                           MX_CALL(route_backward), MX_CALL(linear), MX_CALL(rms_norm), MX_CALL(rms_norm_backward),
                           MX_CALL(fp8_quantize), MX_CALL(fp8_linear), MX_CALL(fp8_linear_backward), MX_CALL(swiglu),
                           MX_CALL(swiglu_backward), MX_CALL(balance_loss), MX_CALL(balance_loss_backward),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_host_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__host_calls(void) {
  PyObject* torch_c = PyImport_ImportModule("torch._C");
  if (torch_c == nullptr) return nullptr;
  g_raw_stream = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
  Py_DECREF(torch_c);
  return g_raw_stream != nullptr ? PyModule_Create(&g_module) : nullptr;
}

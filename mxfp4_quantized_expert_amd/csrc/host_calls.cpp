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

#define MX_CALL(NAME) {#NAME, (PyCFunction)(void (*)(void))NAME, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MX_CALL(permute), MX_CALL(permute_backward), MX_CALL(unpermute), MX_CALL(unpermute_backward),
                           MX_CALL(route_backward), MX_CALL(linear), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_host_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__host_calls(void) {
  PyObject* torch_c = PyImport_ImportModule("torch._C");
  if (torch_c == nullptr) return nullptr;
  g_raw_stream = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
  Py_DECREF(torch_c);
  return g_raw_stream != nullptr ? PyModule_Create(&g_module) : nullptr;
}

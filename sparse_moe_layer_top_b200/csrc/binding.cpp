// binding.cpp -- the regular case of the latency-bound calls, without Python.
//
// A call on a microsecond-sized problem spends most of its time in the checks and
// the argument marshalling of the Python binding (the few-token block: 13 of 20 us).
// These functions take the binding's arguments as they are, verify in C++ that
// everything is regular -- every tensor on the current CUDA device, contiguous, of
// the right element type and large enough, rows of the right length -- allocate the
// outputs that were not given, and make the one library call on the current stream.
// They return None when anything is not regular, with nothing done: the Python
// binding then checks again, in its own words, and raises or handles the call.  A
// status other than MOE_OK comes back as an int.
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstring>
#include <vector>

#include "../../include/moe.h"

namespace {

// The library's entry points, resolved by the Python side from the library it loaded.
decltype(&moe_mx4_quantize) f_quantize;
decltype(&moe_mx4_dequantize) f_dequantize;
decltype(&moe_expert_ffn) f_expert_ffn;
decltype(&moe_decode_forward) f_decode;
decltype(&moe_decode_workspace_size) f_decode_ws;
decltype(&moe_stage_workspace_size) f_stage_ws;

// Arguments of one call; `ok` turns false at the first that is not regular.
struct Call {
  bool ok = true;
  c10::DeviceIndex dev = c10::cuda::current_device();

  // The tensor behind o, or nullptr for None (not allowed: ok = false).
  const at::Tensor* tensor(PyObject* o, bool may_be_none = false) {
    if (o == Py_None) {
      ok = ok && may_be_none;
      return nullptr;
    }
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || t.get_device() != dev || !t.is_contiguous()) ok = false;
    return &t;
  }
  // At least n elements of type a (or b), rows of `row` elements (row < 0: any).
  void* need(PyObject* o, int64_t n, at::ScalarType a, at::ScalarType b, int64_t row, bool may_be_none = false) {
    const at::Tensor* t = tensor(o, may_be_none);
    if (!ok || !t) return nullptr;
    if ((t->scalar_type() != a && t->scalar_type() != b) || t->numel() < n ||
        (row >= 0 && t->dim() >= 2 && t->size(-1) != row)) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* need(PyObject* o, int64_t n, at::ScalarType a, int64_t row, bool may_be_none = false) {
    return need(o, n, a, a, row, may_be_none);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::empty(shape, at::TensorOptions().dtype(t).device(at::Device(at::kCUDA, dev)));
  }
};

// A copy of the moe_problem a ctypes structure holds.
bool problem(PyObject* o, moe_problem* p) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return false;
  }
  const bool ok = b.len == (Py_ssize_t)sizeof(moe_problem);
  if (ok) memcpy(p, b.buf, sizeof(moe_problem));
  PyBuffer_Release(&b);
  return ok;
}

struct Weights {
  const void *wg = nullptr, *wu = nullptr, *wd = nullptr, *sg = nullptr, *su = nullptr, *sd = nullptr, *scales = nullptr;
};
// The expert weights of a bf16 problem: o[0..5] and the scales o[6].
bool weights(Call& c, const moe_problem& p, PyObject* const* o, Weights* w) {
  const int64_t d = p.d, E = p.E, I = p.I, S = p.I_s;
  if (p.act_dtype != MOE_BF16 || d <= 0 || E <= 0 || I <= 0 || S < 0) return false;
  at::ScalarType a = at::kBFloat16, b = at::kBFloat16;
  int64_t per = 1;
  if (p.w_dtype == MOE_FP8_E4M3_B128) {
    a = at::kFloat8_e4m3fn;
    b = at::kByte;
  } else if (p.w_dtype == MOE_MXFP4_B32) {
    a = b = at::kByte;
    per = 2;
  } else if (p.w_dtype != MOE_BF16) {
    return false;
  }
  w->wg = c.need(o[0], E * I * d / per, a, b, d / per);
  w->wu = c.need(o[1], E * I * d / per, a, b, d / per);
  w->wd = c.need(o[2], E * d * I / per, a, b, I / per);
  if (S > 0) {
    w->sg = c.need(o[3], S * d / per, a, b, d / per);
    w->su = c.need(o[4], S * d / per, a, b, d / per);
    w->sd = c.need(o[5], d * S / per, a, b, S / per);
  } else if (o[3] != Py_None || o[4] != Py_None || o[5] != Py_None) {
    return false;  // (ignored matrices: the Python side knows)
  }
  const int64_t blocks = 3 * E * (I / 128) * (d / 128) + 3 * (S / 128) * (d / 128);
  if (p.w_dtype == MOE_FP8_E4M3_B128) w->scales = c.need(o[6], blocks, at::kFloat, -1);
  else if (p.w_dtype == MOE_MXFP4_B32) w->scales = c.need(o[6], blocks * 512, at::kByte, -1);
  else if (o[6] != Py_None) return false;
  return c.ok;
}

PyObject* none() { Py_RETURN_NONE; }

// The interpreter's lock is given up around the allocations and the launches, as a
// ctypes call gives it up: a launch may wait for a full queue.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A status as an int, else `result` (a new reference).
template <typename F>
PyObject* finish(int status, F result) {
  return status == MOE_OK ? result() : PyLong_FromLong(status);
}
// The given object, or the tensor made for it.
PyObject* given(PyObject* o, const at::Tensor& made) { return o == Py_None ? THPVariable_Wrap(made) : Py_NewRef(o); }

// (x, codes or None, scales or None) -> (codes, scales)
PyObject* quantize(PyObject* const* a) {
  Call c;
  const at::Tensor* x = c.tensor(a[0]);
  if (!c.ok || x->dim() < 2) return none();
  const bool f32 = x->scalar_type() == at::kFloat;
  const int64_t rows = x->size(-2), cols = x->size(-1);
  if ((!f32 && x->scalar_type() != at::kBFloat16) || cols <= 0 || cols % 32) return none();
  std::vector<int64_t> cs(x->sizes().begin(), x->sizes().end()), ss(cs);
  int64_t batch = 1;
  for (size_t i = 0; i + 2 < cs.size(); ++i) batch *= cs[i];
  cs.back() = cols / 2;
  ss[ss.size() - 2] = (rows + 127) / 128;
  ss.back() = (cols + 127) / 128;
  ss.push_back(512);
  void* codes = c.need(a[1], batch * rows * cols / 2, at::kByte, cols / 2, true);
  void* scales = c.need(a[2], batch * ss[ss.size() - 3] * ss[ss.size() - 2] * 512, at::kByte, 512, true);
  if (!c.ok) return none();
  at::Tensor tc, ts;
  int s;
  {
    Unlocked u;
    if (a[1] == Py_None) codes = (tc = c.empty(cs, at::kByte)).data_ptr();
    if (a[2] == Py_None) scales = (ts = c.empty(ss, at::kByte)).data_ptr();
    s = f_quantize(x->data_ptr(), f32 ? MOE_F32 : MOE_BF16, batch, rows, cols, codes, scales, c.stream());
  }
  return finish(s, [&] {
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, given(a[1], tc));
    PyTuple_SET_ITEM(r, 1, given(a[2], ts));
    return r;
  });
}

// (codes, scales, out or None, 1 for fp32) -> out
PyObject* dequantize(PyObject* const* a) {
  Call c;
  const at::Tensor* q = c.tensor(a[0]);
  if (!c.ok || q->dim() < 2 || q->scalar_type() != at::kByte) return none();
  const int64_t rows = q->size(-2), cols = 2 * q->size(-1);
  if (cols <= 0 || cols % 32) return none();
  std::vector<int64_t> os(q->sizes().begin(), q->sizes().end());
  int64_t batch = 1;
  for (size_t i = 0; i + 2 < os.size(); ++i) batch *= os[i];
  os.back() = cols;
  at::ScalarType type = a[3] == Py_True ? at::kFloat : at::kBFloat16;
  if (a[2] != Py_None) {
    const at::Tensor* o = c.tensor(a[2]);
    if (!c.ok || (o->scalar_type() != at::kFloat && o->scalar_type() != at::kBFloat16)) return none();
    type = o->scalar_type();
  }
  void* scales = c.need(a[1], batch * ((rows + 127) / 128) * ((cols + 127) / 128) * 512, at::kByte, -1);
  void* out = c.need(a[2], batch * rows * cols, type, cols, true);
  if (!c.ok) return none();
  at::Tensor to;
  int s;
  {
    Unlocked u;
    if (a[2] == Py_None) out = (to = c.empty(os, type)).data_ptr();
    s = f_dequantize(q->data_ptr(), scales, batch, rows, cols, type == at::kFloat ? MOE_F32 : MOE_BF16, out,
                     c.stream());
  }
  return finish(s, [&] { return given(a[2], to); });
}

// (problem, x_perm, offs, six weights, scales, y_perm or None, ws or None) -> y_perm
PyObject* expert_ffn(PyObject* const* a) {
  Call c;
  moe_problem p;
  Weights w;
  if (!problem(a[0], &p) || p.T < 0 || p.k <= 0 || !weights(c, p, a + 3, &w)) return none();
  const at::Tensor* tx = c.tensor(a[1]);
  if (!c.ok || tx->dim() != 2) return none();
  const int64_t R = p.T * p.k + (p.I_s > 0 ? p.T : 0);
  void* x = c.need(a[1], R * p.d, at::kBFloat16, p.d);
  void* offs = c.need(a[2], p.E + 2, at::kInt, -1);
  void* y = c.need(a[10], R * p.d, at::kBFloat16, p.d, true);
  const at::Tensor* ws = c.tensor(a[11], true);
  if (!c.ok) return none();
  at::Tensor ty, tw;
  int s;
  {
    Unlocked u;
    if (a[10] == Py_None) y = (ty = c.empty({tx->size(0), p.d}, at::kBFloat16)).data_ptr();
    if (!ws) ws = &(tw = c.empty({(int64_t)std::max<size_t>(f_stage_ws(&p), 1)}, at::kByte));
    s = f_expert_ffn(&p, x, (const int32_t*)offs, w.wg, w.wu, w.wd, w.sg, w.su, w.sd, w.scales, y, ws->data_ptr(),
                     ws->nbytes(), c.stream());
  }
  return finish(s, [&] { return given(a[10], ty); });
}

// (problem, x, w_router, bias or None, six weights, scales, norm_weight or None, eps, shared_gate or None,
//  y or None, topk_ids or None, topk_w or None, ws or None) -> y
PyObject* decode(PyObject* const* a) {
  Call c;
  moe_problem p;
  Weights w;
  if (!problem(a[0], &p) || p.T < 0 || p.k <= 0 || !weights(c, p, a + 4, &w)) return none();
  const int64_t d = p.d;
  void* x = c.need(a[1], p.T * d, at::kBFloat16, d);
  void* wr = c.need(a[2], (int64_t)p.E * d, at::kBFloat16, d);
  void* bias = c.need(a[3], p.E, at::kFloat, -1, true);
  moe_block_options opt;
  opt.norm_weight = c.need(a[11], d, at::kBFloat16, -1, true);
  opt.norm_eps = (float)PyFloat_AsDouble(a[12]);
  opt.shared_gate = c.need(a[13], d, at::kBFloat16, -1, true);
  void* y = c.need(a[14], p.T * d, at::kBFloat16, d, true);
  void* ids = c.need(a[15], p.T * p.k, at::kInt, p.k, true);
  void* tw = c.need(a[16], p.T * p.k, at::kFloat, p.k, true);
  const at::Tensor* ws = c.tensor(a[17], true);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  if (!c.ok) return none();
  at::Tensor ty, tws;
  int s;
  {
    Unlocked u;
    if (a[14] == Py_None) y = (ty = c.empty({p.T, d}, at::kBFloat16)).data_ptr();
    if (!ws) ws = &(tws = c.empty({(int64_t)std::max<size_t>(f_decode_ws(&p), 1)}, at::kByte));
    s = f_decode(&p, &opt, x, wr, (const float*)bias, w.wg, w.wu, w.wd, w.sg, w.su, w.sd, w.scales, y, (int32_t*)ids,
                 (float*)tw, ws->data_ptr(), ws->nbytes(), c.stream());
  }
  return finish(s, [&] { return given(a[14], ty); });
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N || !f_decode) return none();
  try {
    return F(a);
  } catch (...) {  // e.g. a tensor without storage; allocation errors come again from the Python side
    return none();
  }
}

// The addresses of the six entry points above, in their order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[6];
  if (n != 6) return none();
  for (int i = 0; i < 6; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  f_quantize = (decltype(f_quantize))f[0];
  f_dequantize = (decltype(f_dequantize))f[1];
  f_expert_ffn = (decltype(f_expert_ffn))f[2];
  f_stage_ws = (decltype(f_stage_ws))f[3];
  f_decode_ws = (decltype(f_decode_ws))f[4];
  f_decode = (decltype(f_decode))f[5];
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},
                         {"quantize", FAST((call<quantize, 3>))},
                         {"dequantize", FAST((call<dequantize, 4>))},
                         {"expert_ffn", FAST((call<expert_ffn, 12>))},
                         {"decode", FAST((call<decode, 18>))},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__moe_binding(void) { return PyModule_Create(&module); }

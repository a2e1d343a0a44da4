// The Python side of the calls whose kernels run for a few microseconds (the
// expert choice and the 4-bit experts of a decode step): a CPython extension
// that checks the tensors, allocates the outputs and calls the C entry points
// of libmoe_gb300.so on torch's current stream.  What the ctypes functions of
// ops.py spend in the interpreter (9 us of a 12 us call) is most of such a
// step otherwise.  bind() hands over the entry points' addresses, so the
// extension does not link the library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_gb300.h"

namespace {

struct Refused {};   // a Python error is set

decltype(&moe_route_select) f_route_select;
decltype(&moe_route_select_bwd) f_route_select_bwd;
decltype(&moe_route_balance_bias) f_route_balance_bias;
decltype(&moe_w4_gate_up_swiglu) f_w4_gate_up_swiglu;
decltype(&moe_w4_down_workspace_size) f_w4_down_workspace_size;
decltype(&moe_w4_down_combine) f_w4_down_combine;
PyObject* g_check;   // check(name, status) of _lib: raises MoEError

[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
  va_list va;
  va_start(va, format);
  PyErr_FormatV(type, format, va);
  va_end(va);
  throw Refused();
}

void check(const char* name, int rc) {
  if (rc == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "si", name, rc);
  Py_XDECREF(r);
  throw Refused();
}

// A new tensor where `like` is (the allocator's call itself: through the
// dispatcher two of them take 1.7 us more).
at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
}

// A contiguous CUDA tensor of the current device, of the type and number of dimensions.
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type, const char* type_name, int64_t ndim,
                       at::ScalarType or_type = at::ScalarType::Undefined) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor (the path runs only on the GPU)", name);
  const int device = c10::cuda::current_device();
  if (t.get_device() != device)   // the kernels run on the current device and would be handed another GPU's memory
    refuse(PyExc_ValueError, "%s is on cuda:%d but the current device is cuda:%d", name, (int)t.get_device(), device);
  if (t.scalar_type() != type && t.scalar_type() != or_type) refuse(PyExc_TypeError, "%s must be %s", name, type_name);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  if (t.dim() != ndim) refuse(PyExc_ValueError, "%s must have %d dims", name, (int)ndim);
  return t;
}
const at::Tensor& need_f32(PyObject* o, const char* name, int64_t ndim) { return need(o, name, at::kFloat, "torch.float32", ndim); }
const at::Tensor& need_i32(PyObject* o, const char* name, int64_t ndim) { return need(o, name, at::kInt, "torch.int32", ndim); }
const at::Tensor& need_bf16(PyObject* o, const char* name, int64_t ndim) {
  return need(o, name, at::kBFloat16, "torch.bfloat16", ndim);
}
const at::Tensor& need_logits(PyObject* o) {
  return need(o, "logits", at::kFloat, "torch.float32 or torch.bfloat16", 2, at::kBFloat16);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

template <typename T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// Runs f without the GIL (a full launch queue blocks) and checks its status.
template <typename F>
void run(const char* name, F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  check(name, rc);
}

#define BODY_BEGIN \
  HANDLE_TH_ERRORS \
  try {
#define BODY_END             \
  }                          \
  catch (const Refused&) {   \
    return nullptr;          \
  }                          \
  END_HANDLE_TH_ERRORS

#define ARGS(n)                                                                     \
  if (nargs != (n)) {                                                               \
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", (n), nargs);    \
    return nullptr;                                                                 \
  }

// (logits, k, bias, score, n_groups, top_groups, group_score, renorm, scale) -> ids, w
PyObject* route_select(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(9)
  BODY_BEGIN
  const at::Tensor& logits = need_logits(a[0]);
  const int64_t T = logits.size(0), E = logits.size(1), k = integer(a[1]);
  const float* bias = nullptr;
  if (a[2] != Py_None) {
    const at::Tensor& b = need_f32(a[2], "bias", 1);
    if (b.size(0) != E) refuse(PyExc_ValueError, "bias must be [E]");
    bias = ptr<float>(b);
  }
  const int64_t score = integer(a[3]), groups = integer(a[4]), top = integer(a[5]), group_score = integer(a[6]),
                renorm = integer(a[7]);
  const float scale = (float)real(a[8]);
  const at::Tensor ids = fresh({T, k < 0 ? 0 : k}, at::kInt, logits);
  const at::Tensor w = fresh({T, k < 0 ? 0 : k}, at::kFloat, logits);
  void* st = stream();
  run("moe_route_select", [&] {
    return f_route_select(ptr(logits), logits.scalar_type() == at::kBFloat16, bias, T, E, k, (int)score, groups, top,
                          (int)group_score, (int)renorm, scale, ptr<int32_t>(ids), ptr<float>(w), st);
  });
  return pair(ids, w);
  BODY_END
}

// (dw, logits, ids, score, renorm, scale, row_map) -> d_logits, or with row_map d_logits, dw
PyObject* route_select_bwd(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(7)
  BODY_BEGIN
  const at::Tensor& dw = need_f32(a[0], "dw", 2);
  const at::Tensor& logits = need_logits(a[1]);
  const at::Tensor& ids = need_i32(a[2], "ids", 2);
  const int64_t T = logits.size(0), E = logits.size(1), k = ids.size(1);
  if (ids.size(0) != T) refuse(PyExc_ValueError, "ids must be [T, k]");
  const int64_t score = integer(a[3]), renorm = integer(a[4]);
  const float scale = (float)real(a[5]);
  const int32_t* row_map = nullptr;
  int64_t nparts = 1;
  at::Tensor sum;
  if (a[6] != Py_None) {
    const at::Tensor& m = need_i32(a[6], "row_map", 1);
    if (m.size(0) != T * k || dw.size(0) != T * k)
      refuse(PyExc_ValueError, "row_map must hold T*k entries and dw must be [T*k, nparts]");
    row_map = ptr<int32_t>(m);
    nparts = dw.size(1);
    sum = fresh({T, k}, at::kFloat, dw);
  } else if (dw.size(0) != T || dw.size(1) != k) {
    refuse(PyExc_ValueError, "dw must be [T, k]");
  }
  const at::Tensor d_logits = fresh({T, E}, logits.scalar_type(), logits);
  void* st = stream();
  run("moe_route_select_bwd", [&] {
    return f_route_select_bwd(ptr<float>(dw), nparts, row_map, ptr(logits), logits.scalar_type() == at::kBFloat16,
                              ptr<int32_t>(ids), T, E, k, (int)score, (int)renorm, scale, ptr(d_logits),
                              sum.defined() ? ptr<float>(sum) : nullptr, st);
  });
  return sum.defined() ? pair(d_logits, sum) : THPVariable_Wrap(d_logits);
  BODY_END
}

// (bias, counts, rate, out) -> out
PyObject* route_balance_bias(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BODY_BEGIN
  const at::Tensor& bias = need_f32(a[0], "bias", 1);
  const at::Tensor& counts = need_i32(a[1], "counts", 1);
  const int64_t E = bias.size(0);
  if (counts.size(0) != E) refuse(PyExc_ValueError, "counts must be [E]");
  const float rate = (float)real(a[2]);
  const at::Tensor out = a[3] == Py_None ? fresh({E}, at::kFloat, bias) : need_f32(a[3], "out", 1);
  if (out.size(0) != E) refuse(PyExc_ValueError, "out must be [E]");
  void* st = stream();
  run("moe_route_balance_bias", [&] { return f_route_balance_bias(ptr<float>(bias), ptr<int32_t>(counts), E, rate, ptr<float>(out), st); });
  return THPVariable_Wrap(out);
  BODY_END
}

// 4-bit weights with K rows an expert.
struct Weights {
  const uint32_t* q;
  const uint16_t* scales;
  const uint8_t* zeros;
  int64_t E, N, group;
};

Weights weights(PyObject* q, PyObject* scales, PyObject* zeros, int64_t K) {
  const at::Tensor& tq = need_i32(q, "qweight", 2);
  const at::Tensor& ts = need_bf16(scales, "scales", 2);
  const int64_t words = tq.size(0), rows = ts.size(0);
  if (K < 8 || K % 8 != 0 || words % (K / 8) != 0)
    refuse(PyExc_ValueError, "qweight must be [E*K/8, N] with K = %lld", (long long)K);
  Weights w{ptr<uint32_t>(tq), ptr<uint16_t>(ts), nullptr, words / (K / 8), tq.size(1), 0};
  if (ts.size(1) != w.N || w.E == 0 || rows == 0 || rows % w.E != 0 || K % (rows / w.E) != 0)
    refuse(PyExc_ValueError, "scales must be [E*K/group, N]");
  w.group = K / (rows / w.E);
  if (zeros != Py_None) {
    const at::Tensor& tz = need(zeros, "zeros", at::kByte, "torch.uint8", 2);
    if (tz.size(0) != rows || tz.size(1) != w.N) refuse(PyExc_ValueError, "zeros must be [E*K/group, N]");
    w.zeros = ptr<uint8_t>(tz);
  }
  return w;
}

// The slots' experts ids [T, k] and k; None: one dense expert.
const int32_t* slots(PyObject* o, int64_t T, int64_t E, int64_t* k) {
  *k = 1;
  if (o == Py_None) {
    if (E != 1) refuse(PyExc_ValueError, "ids are needed with more than one expert");
    return nullptr;
  }
  const at::Tensor& ids = need_i32(o, "ids", 2);
  if (ids.size(0) != T) refuse(PyExc_ValueError, "ids must be [T, k]");
  *k = ids.size(1);
  return ptr<int32_t>(ids);
}

// (x, ids, qweight, scales, zeros) -> h
PyObject* w4_gate_up_swiglu(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(5)
  BODY_BEGIN
  const at::Tensor& x = need_bf16(a[0], "x", 2);
  const int64_t T = x.size(0), H = x.size(1);
  const Weights w = weights(a[2], a[3], a[4], H);
  if (w.N % 2 != 0) refuse(PyExc_ValueError, "qweight must be [E*H/8, 2I]");
  int64_t k;
  const int32_t* ids = slots(a[1], T, w.E, &k);
  const at::Tensor h = fresh({T, k, w.N / 2}, at::kBFloat16, x);
  void* st = stream();
  run("moe_w4_gate_up_swiglu", [&] {
    return f_w4_gate_up_swiglu(ptr<uint16_t>(x), ids, w.q, w.scales, w.zeros, T, H, w.E, k, w.N / 2, w.group,
                               ptr<uint16_t>(h), st);
  });
  return THPVariable_Wrap(h);
  BODY_END
}

// (h, ids, w, qweight, scales, zeros, y_shared, out) -> y
PyObject* w4_down_combine(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(8)
  BODY_BEGIN
  const at::Tensor& h = need_bf16(a[0], "h", 3);
  const int64_t T = h.size(0), k = h.size(1), I = h.size(2);
  const Weights w = weights(a[3], a[4], a[5], I);
  int64_t slots_k;
  const int32_t* ids = slots(a[1], T, w.E, &slots_k);
  if (slots_k != k) refuse(PyExc_ValueError, "h must be [T, k, I] and ids [T, k]");
  const float* wt = nullptr;
  if (a[2] != Py_None) {
    const at::Tensor& t = need_f32(a[2], "w", 2);
    if (t.size(0) != T || t.size(1) != k) refuse(PyExc_ValueError, "w must be [T, k]");
    wt = ptr<float>(t);
  }
  const uint16_t* shared = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor& t = need_bf16(a[6], "y_shared", 2);
    if (t.size(0) != T || t.size(1) != w.N) refuse(PyExc_ValueError, "y_shared must be [T, H]");
    shared = ptr<uint16_t>(t);
  }
  const at::Tensor y = a[7] == Py_None ? fresh({T, w.N}, at::kBFloat16, h) : need_bf16(a[7], "out", 2);
  if (y.size(0) != T || y.size(1) != w.N) refuse(PyExc_ValueError, "out must be [T, H]");
  size_t bytes = 0;
  check("moe_w4_down_workspace_size", f_w4_down_workspace_size(T, w.N, k, &bytes));
  const at::Tensor ws = fresh({(int64_t)bytes}, at::kByte, h);
  void* st = stream();
  run("moe_w4_down_combine", [&] {
    return f_w4_down_combine(ptr<uint16_t>(h), ids, wt, w.q, w.scales, w.zeros, shared, T, w.N, w.E, k, I, w.group,
                             ptr<uint16_t>(y), ptr(ws), bytes, st);
  });
  return THPVariable_Wrap(y);
  BODY_END
}

// (check, addresses of the entry points in the order below)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(7)
  BODY_BEGIN
  void* at[6];
  for (int i = 0; i < 6; ++i) at[i] = reinterpret_cast<void*>(static_cast<uintptr_t>(integer(a[i + 1])));
  f_route_select = reinterpret_cast<decltype(f_route_select)>(at[0]);
  f_route_select_bwd = reinterpret_cast<decltype(f_route_select_bwd)>(at[1]);
  f_route_balance_bias = reinterpret_cast<decltype(f_route_balance_bias)>(at[2]);
  f_w4_gate_up_swiglu = reinterpret_cast<decltype(f_w4_gate_up_swiglu)>(at[3]);
  f_w4_down_workspace_size = reinterpret_cast<decltype(f_w4_down_workspace_size)>(at[4]);
  f_w4_down_combine = reinterpret_cast<decltype(f_w4_down_combine)>(at[5]);
  Py_INCREF(a[0]);
  Py_XSETREF(g_check, a[0]);
  Py_RETURN_NONE;
  BODY_END
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL

PyMethodDef methods[] = {
    {"bind", FAST(bind), nullptr},
    {"route_select", FAST(route_select), nullptr},
    {"route_select_bwd", FAST(route_select_bwd), nullptr},
    {"route_balance_bias", FAST(route_balance_bias), nullptr},
    {"w4_gate_up_swiglu", FAST(w4_gate_up_swiglu), nullptr},
    {"w4_down_combine", FAST(w4_down_combine), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }

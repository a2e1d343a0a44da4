// The Python side of the calls whose kernels run for a few microseconds (the
// expert choice, the experts of a decode step, a block's norms, the gradients'
// clipping): a CPython extension
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

#include <algorithm>
#include <type_traits>
#include <vector>

#include "../../include/moe_gb300.h"

namespace {

struct Refused {};   // a Python error is set

decltype(&moe_route_select) f_route_select;
decltype(&moe_route_select_bwd) f_route_select_bwd;
decltype(&moe_route_balance_bias) f_route_balance_bias;
decltype(&moe_w4_gate_up_swiglu) f_w4_gate_up_swiglu;
decltype(&moe_w4_down_workspace_size) f_w4_down_workspace_size;
decltype(&moe_w4_down_combine) f_w4_down_combine;
decltype(&moe_few_experts_workspace_size) f_few_experts_workspace_size;
decltype(&moe_few_experts) f_few_experts;
decltype(&moe_few_layer_workspace_size) f_few_layer_workspace_size;
decltype(&moe_few_layer) f_few_layer;
decltype(&moe_block_norm) f_block_norm;
decltype(&moe_block_norm_bwd_workspace_size) f_block_norm_bwd_workspace_size;
decltype(&moe_block_norm_bwd) f_block_norm_bwd;
decltype(&moe_grad_clip_workspace_size) f_grad_clip_workspace_size;
decltype(&moe_grad_clip) f_grad_clip;
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

// A contiguous CUDA tensor of the current device, of the type and number of
// dimensions (-1: any layout of any dimensions that fills its memory).
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type, const char* type_name, int64_t ndim,
                       at::ScalarType or_type = at::ScalarType::Undefined) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor (the path runs only on the GPU)", name);
  const int device = c10::cuda::current_device();
  if (t.get_device() != device)   // the kernels run on the current device and would be handed another GPU's memory
    refuse(PyExc_ValueError, "%s is on cuda:%d but the current device is cuda:%d", name, (int)t.get_device(), device);
  if (t.scalar_type() != type && t.scalar_type() != or_type) refuse(PyExc_TypeError, "%s must be %s", name, type_name);
  if (ndim < 0) {
    if (!t.is_non_overlapping_and_dense()) refuse(PyExc_ValueError, "%s must fill its memory: no gaps, no overlaps", name);
    return t;
  }
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

// After a call that wrote into a tensor it was given: autograd, where it keeps
// the tensor, has to know that it changed.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
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
  if (a[3] != Py_None) written(out);
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
  if (a[7] != Py_None) written(y);
  return THPVariable_Wrap(y);
  BODY_END
}

// bf16 experts gate_up [E*H, 2I], down [E*I, H] for rows of H, E of them (0: as many as gate_up holds).
struct Experts {
  const uint16_t *gate_up, *down;
  int64_t E, I;
};

Experts experts(PyObject* gate_up, PyObject* down, int64_t H, int64_t E, const char* gate_up_name, const char* down_name) {
  const at::Tensor& gu = need_bf16(gate_up, gate_up_name, 2);
  const at::Tensor& dn = need_bf16(down, down_name, 2);
  if (H < 1 || gu.size(0) % H != 0 || gu.size(0) == 0 || gu.size(1) % 2 != 0)
    refuse(PyExc_ValueError, "%s must be [E*H, 2I]", gate_up_name);
  const Experts x{ptr<uint16_t>(gu), ptr<uint16_t>(dn), gu.size(0) / H, gu.size(1) / 2};
  if (E && x.E != E) refuse(PyExc_ValueError, "%s must be [E*H, 2I] with E = %lld", gate_up_name, (long long)E);
  if (dn.size(0) != x.E * x.I || dn.size(1) != H) refuse(PyExc_ValueError, "%s must be [E*I, H]", down_name);
  return x;
}

Experts shared_expert(PyObject* gate_up, PyObject* down, int64_t H) {
  if ((gate_up == Py_None) != (down == Py_None)) refuse(PyExc_ValueError, "sh_gate_up and sh_down go together");
  if (gate_up == Py_None) return Experts{nullptr, nullptr, 1, 0};
  return experts(gate_up, down, H, 1, "sh_gate_up", "sh_down");
}

// Both contiguous.
bool overlap(const at::Tensor& a, const at::Tensor& b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.data_ptr()), q = reinterpret_cast<uintptr_t>(b.data_ptr());
  return a.nbytes() && b.nbytes() && p < q + b.nbytes() && q < p + a.nbytes();
}

// (x, ids, w, gate_up, down, sh_gate_up, sh_down, out) -> y
PyObject* few_experts(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(8)
  BODY_BEGIN
  const at::Tensor& x = need_bf16(a[0], "x", 2);
  const at::Tensor& ids = need_i32(a[1], "ids", 2);
  const at::Tensor& w = need_f32(a[2], "w", 2);
  const int64_t T = x.size(0), H = x.size(1), k = ids.size(1);
  if (ids.size(0) != T || w.size(0) != T || w.size(1) != k) refuse(PyExc_ValueError, "ids and w must be [T, k]");
  const Experts e = experts(a[3], a[4], H, 0, "gate_up", "down"), sh = shared_expert(a[5], a[6], H);
  const at::Tensor y = a[7] == Py_None ? fresh({T, H}, at::kBFloat16, x) : need_bf16(a[7], "out", 2);
  if (y.size(0) != T || y.size(1) != H) refuse(PyExc_ValueError, "out must be [T, H]");
  for (int i = 0; i < 7 && a[7] != Py_None; ++i)
    if (a[i] != Py_None && overlap(y, THPVariable_Unpack(a[i]))) refuse(PyExc_ValueError, "out overlaps an input");
  size_t bytes = 0;
  check("moe_few_experts_workspace_size", f_few_experts_workspace_size(T, H, e.E, k, e.I, sh.I, &bytes));
  const at::Tensor ws = fresh({(int64_t)bytes}, at::kByte, x);
  void* st = stream();
  run("moe_few_experts", [&] {
    return f_few_experts(ptr<uint16_t>(x), ptr<int32_t>(ids), ptr<float>(w), e.gate_up, e.down, sh.gate_up, sh.down, T, H,
                         e.E, k, e.I, sh.I, ptr<uint16_t>(y), ptr(ws), bytes, st);
  });
  if (a[7] != Py_None) written(y);
  return THPVariable_Wrap(y);
  BODY_END
}

// (x, w_router, gate_up, down, k, bias, balance_bias, sh_gate_up, sh_down, score, n_groups, top_groups, group_score,
//  renorm, scale) -> y, ids, w
PyObject* few_layer(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(15)
  BODY_BEGIN
  const at::Tensor& x = need_bf16(a[0], "x", 2);
  const at::Tensor& wr = need_f32(a[1], "w_router", 2);
  const int64_t T = x.size(0), H = x.size(1), E = wr.size(1), k = integer(a[4]);
  if (wr.size(0) != H || E < 1) refuse(PyExc_ValueError, "w_router must be [H, E]");
  const Experts e = experts(a[2], a[3], H, E, "gate_up", "down"), sh = shared_expert(a[7], a[8], H);
  const float* bias[2] = {nullptr, nullptr};
  const char* name[2] = {"bias", "balance_bias"};
  for (int i = 0; i < 2; ++i)
    if (a[5 + i] != Py_None) {
      const at::Tensor& b = need_f32(a[5 + i], name[i], 1);
      if (b.size(0) != E) refuse(PyExc_ValueError, "%s must be [E]", name[i]);
      bias[i] = ptr<float>(b);
    }
  const int64_t score = integer(a[9]), groups = integer(a[10]), top = integer(a[11]), group_score = integer(a[12]),
                renorm = integer(a[13]);
  const float scale = (float)real(a[14]);
  size_t bytes = 0;
  check("moe_few_layer_workspace_size", f_few_layer_workspace_size(T, H, E, k, e.I, sh.I, &bytes));
  const at::Tensor y = fresh({T, H}, at::kBFloat16, x), ids = fresh({T, k}, at::kInt, x), w = fresh({T, k}, at::kFloat, x);
  const at::Tensor ws = fresh({(int64_t)bytes}, at::kByte, x);
  void* st = stream();
  run("moe_few_layer", [&] {
    return f_few_layer(ptr<uint16_t>(x), ptr<float>(wr), bias[0], bias[1], e.gate_up, e.down, sh.gate_up, sh.down, T, H, E,
                       k, e.I, sh.I, (int)score, groups, top, (int)group_score, (int)renorm, scale, ptr<int32_t>(ids),
                       ptr<float>(w), ptr<uint16_t>(y), ptr(ws), bytes, st);
  });
  PyObject* out[3] = {THPVariable_Wrap(y), THPVariable_Wrap(ids), THPVariable_Wrap(w)};
  PyObject* r = PyTuple_Pack(3, out[0], out[1], out[2]);
  for (PyObject* o : out) Py_XDECREF(o);
  return r;
  BODY_END
}

// The operands of block_norm; an absent one is undefined.
struct Norm {
  at::Tensor x, branch, weight, post, gate;
  int types = 0;
  int64_t T, H, gates = 0;
  float a, b;
};

at::Tensor float_or_bf16(PyObject* o, const char* name, int64_t ndim) {
  return need(o, name, at::kFloat, "torch.float32 or torch.bfloat16", ndim, at::kBFloat16);
}

// From a[0..]: x, weight, branch, post_weight, gate, residual_scale, branch_scale.
Norm norm_operands(PyObject* const* a) {
  Norm n;
  n.x = float_or_bf16(a[0], "x", 2);
  n.T = n.x.size(0);
  n.H = n.x.size(1);
  if (n.x.scalar_type() == at::kFloat) n.types |= MOE_NORM_X_F32;
  auto vector = [&](PyObject* o, const char* name, int bit) {
    at::Tensor t;
    if (o == Py_None) return t;
    t = float_or_bf16(o, name, 1);
    if (t.size(0) != n.H) refuse(PyExc_ValueError, "%s must be [H]", name);
    if (t.scalar_type() == at::kFloat) n.types |= bit;
    return t;
  };
  n.weight = vector(a[1], "weight", MOE_NORM_WEIGHT_F32);
  if (a[2] != Py_None) {
    n.branch = need_bf16(a[2], "branch", 2);
    if (n.branch.size(0) != n.T || n.branch.size(1) != n.H) refuse(PyExc_ValueError, "branch must be [T, H]");
  }
  n.post = vector(a[3], "post_weight", MOE_NORM_POST_F32);
  n.a = (float)real(a[5]);
  n.b = (float)real(a[6]);
  if (!n.branch.defined()) {
    if (!n.weight.defined()) refuse(PyExc_ValueError, "block_norm needs branch or weight");
    if (n.post.defined() || a[4] != Py_None || n.a != 1.f || n.b != 1.f)
      refuse(PyExc_ValueError, "post_weight, gate and the scales need branch");
  }
  if (a[4] != Py_None) {
    n.gate = float_or_bf16(a[4], "gate", 2);
    n.gates = n.gate.size(0);
    if (n.gate.size(1) != n.H || n.gates == 0 || n.T % n.gates != 0)
      refuse(PyExc_ValueError, "gate must be [gates, H] with gates a divisor of T");
    if (n.gate.scalar_type() == at::kFloat) n.types |= MOE_NORM_GATE_F32;
  }
  return n;
}

template <typename T = void>
T* maybe(const at::Tensor& t) {
  return t.defined() ? ptr<T>(t) : nullptr;
}
at::Tensor like(const at::Tensor& t) { return t.defined() ? fresh(t.sizes(), t.scalar_type(), t) : at::Tensor(); }
PyObject* wrap_or_none(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// (x, weight, branch, post_weight, gate, residual_scale, branch_scale, eps, save) -> r or None, h or None, stats or None
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(9)
  BODY_BEGIN
  const Norm n = norm_operands(a);
  const float eps = (float)real(a[7]);
  at::Tensor r, h, stats;
  if (n.branch.defined()) r = fresh({n.T, n.H}, n.x.scalar_type(), n.x);
  if (n.weight.defined()) h = fresh({n.T, n.H}, at::kBFloat16, n.x);
  if (integer(a[8])) stats = fresh({2, n.T}, at::kFloat, n.x);
  void* st = stream();
  run("moe_block_norm", [&] {
    return f_block_norm(ptr(n.x), maybe<uint16_t>(n.branch), maybe(n.weight), maybe(n.post), maybe(n.gate), n.types, n.T,
                        n.H, n.gates, n.a, n.b, eps, maybe(r), maybe<uint16_t>(h), maybe<float>(stats), st);
  });
  PyObject* out[3] = {wrap_or_none(r), wrap_or_none(h), wrap_or_none(stats)};
  PyObject* tuple = PyTuple_Pack(3, out[0], out[1], out[2]);
  for (PyObject* o : out) Py_XDECREF(o);
  return tuple;
  BODY_END
}

// (dh, dr, stats, x, weight, branch, post_weight, gate, residual_scale, branch_scale)
//  -> dx, d_branch, d_weight, d_post_weight, d_gate (None where the operand is)
PyObject* block_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(10)
  BODY_BEGIN
  const Norm n = norm_operands(a + 3);
  at::Tensor dh, dr, stats;
  if ((a[0] == Py_None) != !n.weight.defined()) refuse(PyExc_ValueError, "dh and weight go together");
  if (a[0] != Py_None) {
    dh = need_bf16(a[0], "dh", 2);
    if (dh.size(0) != n.T || dh.size(1) != n.H) refuse(PyExc_ValueError, "dh must be [T, H]");
  }
  if (a[1] != Py_None) {
    dr = need(a[1], "dr", n.x.scalar_type(), "of x's type", 2);
    if (dr.size(0) != n.T || dr.size(1) != n.H) refuse(PyExc_ValueError, "dr must be [T, H]");
  }
  if (n.weight.defined() || n.post.defined()) {
    stats = need_f32(a[2], "stats", 2);
    if (stats.size(0) != 2 || stats.size(1) != n.T) refuse(PyExc_ValueError, "stats must be [2, T]");
  }
  const at::Tensor dx = like(n.x), d_branch = like(n.branch), d_weight = like(n.weight), d_post = like(n.post),
                   d_gate = like(n.gate);
  size_t bytes = 0;
  check("moe_block_norm_bwd_workspace_size",
        f_block_norm_bwd_workspace_size(n.T, n.H, n.gates, n.weight.defined(), n.post.defined(), &bytes));
  const at::Tensor ws = fresh({(int64_t)bytes}, at::kByte, n.x);
  void* st = stream();
  run("moe_block_norm_bwd", [&] {
    return f_block_norm_bwd(maybe<uint16_t>(dh), maybe(dr), ptr(n.x), maybe<uint16_t>(n.branch), maybe<float>(stats),
                            maybe(n.weight), maybe(n.post), maybe(n.gate), n.types, n.T, n.H, n.gates, n.a, n.b, ptr(dx),
                            maybe<uint16_t>(d_branch), maybe(d_weight), maybe(d_post), maybe(d_gate), ptr(ws), bytes, st);
  });
  PyObject* out[5] = {wrap_or_none(dx), wrap_or_none(d_branch), wrap_or_none(d_weight), wrap_or_none(d_post),
                      wrap_or_none(d_gate)};
  PyObject* tuple = PyTuple_Pack(5, out[0], out[1], out[2], out[3], out[4]);
  for (PyObject* o : out) Py_XDECREF(o);
  return tuple;
  BODY_END
}

// Elements at the same places of both tensors' memory belong together.
bool same_layout(const at::Tensor& a, const at::Tensor& b) {
  if (a.is_contiguous() && b.is_contiguous()) return true;   // in order, whatever the shapes
  if (a.sizes() != b.sizes()) return false;
  for (int64_t d = 0; d < a.dim(); ++d)
    if (a.size(d) > 1 && a.stride(d) != b.stride(d)) return false;
  return true;
}

// (grads: a list or tuple, outs: the same or None, max_norm, eps) -> norm
PyObject* grad_clip(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4)
  BODY_BEGIN
  const bool clip = a[1] != Py_None;
  if (!(PyList_Check(a[0]) || PyTuple_Check(a[0])) || (clip && !(PyList_Check(a[1]) || PyTuple_Check(a[1]))))
    refuse(PyExc_TypeError, "grads and out must be lists or tuples of tensors");
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[0]);
  if (n == 0) refuse(PyExc_ValueError, "grads must hold a tensor");
  if (clip && PySequence_Fast_GET_SIZE(a[1]) != n) refuse(PyExc_ValueError, "out must hold a tensor for each of grads");
  std::vector<const void*> src(n);
  std::vector<void*> dst(n);
  std::vector<int64_t> size(n);
  std::vector<uint8_t> f32(n);
  struct Span {
    uintptr_t begin, end;
    bool operator<(const Span& o) const { return begin < o.begin; }
  };
  std::vector<Span> reads, writes;   // of what is read alone, and of what is written
  const int device = c10::cuda::current_device();   // need() asks for it each time
  auto tensor = [&](PyObject* o, const char* name, at::ScalarType type, at::ScalarType or_type) -> const at::Tensor& {
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.is_cuda() && t.get_device() == device && (t.scalar_type() == type || t.scalar_type() == or_type) && t.is_non_overlapping_and_dense())
        return t;
    }
    return need(o, name, type, or_type == at::kBFloat16 ? "torch.float32 or torch.bfloat16" : "of its gradient's type", -1, or_type);
  };
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PySequence_Fast_GET_ITEM(a[0], i);
    const at::Tensor& g = tensor(o, "a gradient", at::kFloat, at::kBFloat16);
    src[i] = ptr(g);
    size[i] = g.numel();
    f32[i] = g.scalar_type() == at::kFloat;
    if (!clip) continue;
    dst[i] = const_cast<void*>(src[i]);
    PyObject* q = PySequence_Fast_GET_ITEM(a[1], i);
    if (q != o) {
      const at::Tensor& t = tensor(q, "a tensor of out", g.scalar_type(), at::ScalarType::Undefined);
      if (t.numel() != size[i]) refuse(PyExc_ValueError, "a tensor of out must have its gradient's size");
      if (!same_layout(g, t)) refuse(PyExc_ValueError, "a tensor of out must have its gradient's strides");
      dst[i] = ptr(t);
    }
    const uintptr_t bytes = (uintptr_t)size[i] * (f32[i] ? 4 : 2), from = reinterpret_cast<uintptr_t>(src[i]),
                    to = reinterpret_cast<uintptr_t>(dst[i]);
    if (bytes == 0) continue;
    if (to != from) reads.push_back({from, from + bytes});
    writes.push_back({to, to + bytes});
  }
  // what is written overlaps nothing else: a gradient that is listed twice would be scaled twice
  for (std::vector<Span>* v : {&reads, &writes})
    if (!std::is_sorted(v->begin(), v->end())) std::sort(v->begin(), v->end());
  uintptr_t end = 0;
  auto read = reads.begin();
  for (const Span& s : writes) {
    if (s.begin < end) refuse(PyExc_ValueError, "a tensor of out overlaps another one of out");
    end = s.end;
    while (read != reads.end() && read->end <= s.begin) ++read;
    for (auto r = read; r != reads.end() && r->begin < s.end; ++r)
      if (r->end > s.begin) refuse(PyExc_ValueError, "a tensor of out overlaps a gradient");
  }
  const at::Tensor& first = THPVariable_Unpack(PySequence_Fast_GET_ITEM(a[0], 0));
  const float max_norm = (float)real(a[2]), eps = (float)real(a[3]);
  const at::Tensor norm = fresh({}, at::kFloat, first);
  size_t bytes = 0;
  check("moe_grad_clip_workspace_size", f_grad_clip_workspace_size(src.data(), size.data(), f32.data(), n, &bytes));
  const at::Tensor ws = fresh({(int64_t)bytes}, at::kByte, first);
  void* st = stream();
  run("moe_grad_clip", [&] {
    return f_grad_clip(src.data(), clip ? dst.data() : nullptr, size.data(), f32.data(), n, max_norm, eps, ptr<float>(norm),
                       ptr(ws), bytes, st);
  });
  if (clip)   // the list as it is now: another thread may have changed it meanwhile
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(a[1]); ++i)
      if (THPVariable_Check(PySequence_Fast_GET_ITEM(a[1], i))) written(THPVariable_Unpack(PySequence_Fast_GET_ITEM(a[1], i)));
  return THPVariable_Wrap(norm);
  BODY_END
}

// (check, addresses of the entry points in the order below)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(16)
  BODY_BEGIN
  int next = 1;
  auto take = [&](auto& f) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(static_cast<uintptr_t>(integer(a[next++])));
  };
  take(f_route_select);
  take(f_route_select_bwd);
  take(f_route_balance_bias);
  take(f_w4_gate_up_swiglu);
  take(f_w4_down_workspace_size);
  take(f_w4_down_combine);
  take(f_few_experts_workspace_size);
  take(f_few_experts);
  take(f_few_layer_workspace_size);
  take(f_few_layer);
  take(f_block_norm);
  take(f_block_norm_bwd_workspace_size);
  take(f_block_norm_bwd);
  take(f_grad_clip_workspace_size);
  take(f_grad_clip);
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
    {"few_experts", FAST(few_experts), nullptr},
    {"few_layer", FAST(few_layer), nullptr},
    {"block_norm", FAST(block_norm), nullptr},
    {"block_norm_bwd", FAST(block_norm_bwd), nullptr},
    {"grad_clip", FAST(grad_clip), nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }

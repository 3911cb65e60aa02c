// gdr_binding.cpp -- the torch side of the operators of include/gdr_block.h and gdr_attn.h: checks of shapes, types
// and strides, allocation of outputs and workspace, and the call on the current stream.
//
// A decoding step's kernel runs 2 to 10 us; marshalled in Python a call took 11 to 15 us of host time
// on the GPU's host (attributes of eight tensors, the allocator, the foreign call), here 3 to 5.  The
// library's entry points are bound by address, so this module does not link against it and follows
// the library that the package has open.  Errors: ValueError for what is found here, the status
// number for what the library refuses (the package raises GDRError from it).
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include "../../include/gdr_attn.h"
#include "../../include/gdr_block.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

#define GDR_ENTRIES(X)                                                                                              \
  X(gdr_conv_fwd) X(gdr_conv_bwd) X(gdr_conv_step) X(gdr_conv_fwd_workspace_bytes) X(gdr_conv_bwd_workspace_bytes) \
  X(gdr_ssm_fwd) X(gdr_ssm_bwd) X(gdr_ssm_step) X(gdr_ssm_saved_bytes) X(gdr_ssm_fwd_workspace_bytes)              \
  X(gdr_ssm_bwd_workspace_bytes) X(gdr_norm_fwd) X(gdr_norm_bwd) X(gdr_norm_bwd_workspace_bytes) X(gdr_step) X(gdr_rope) X(gdr_rope_workspace_bytes)              \
  X(gdr_attn_fwd) X(gdr_attn_bwd) X(gdr_attn_fwd_workspace_bytes) X(gdr_attn_bwd_workspace_bytes) X(gdr_attn_step)        \
  X(gdr_attn_step_workspace_bytes) X(gdr_cache_write) X(gdr_cache_write_workspace_bytes)

struct Library {
#define GDR_FIELD(name) decltype(&::name) name;
  GDR_ENTRIES(GDR_FIELD)
#undef GDR_FIELD
} lib;

const Tensor kNone;

const Tensor& tensor(PyObject* o, const char* name) {
  if (o == Py_None) return kNone;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
const Tensor& required(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.defined(), name, ": expected a tensor, got None");
  return t;
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

gdr_dtype type_code(at::ScalarType t) {
  if (t == at::kBFloat16) return GDR_DTYPE_BF16;
  TORCH_CHECK_VALUE(t == at::kFloat, "dtype ", t, ": float32 or bfloat16");
  return GDR_DTYPE_F32;
}

// A size as the library takes it: one that does not fit must not arrive as another.
int size32(const char* name, int64_t v) {
  TORCH_CHECK_VALUE(v <= INT_MAX, name, ": a size of ", v, " does not fit 32 bits");
  return (int)v;
}

// Makes the tensors' device current for a call: the default stream of every device has the same handle, which
// the library would take for the current device's.  Asks first: torch's guard, when there is nothing to change,
// costs a call 0.2 us of host time.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(at::Device dev) {
    if (c10::cuda::current_device() != dev.index()) guard.set_index(dev.index());
  }
};

// A call's tensors lie on one device, that of its first activation: the kernels run there.
void on_device(const char* name, const Tensor& t, at::Device dev) {
  TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", the call's first tensor on ", dev);
}

// An activation of the call: on the GPU, of a shape and type.
void act(const char* name, const Tensor& t, IntArrayRef shape, at::ScalarType type, at::Device dev) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == type && t.sizes() == shape, name, ": expected a CUDA ", type,
                    " tensor of shape ", shape, ", got ", t.scalar_type(), " ", t.sizes(), " on ", t.device());
  on_device(name, t, dev);
}

// A contiguous tensor of a shape and type, or none.
void full(const char* name, const Tensor& t, IntArrayRef shape, at::Device dev, at::ScalarType type = at::kFloat) {
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous(), name,
                    ": expected a contiguous CUDA ", type, " tensor of shape ", shape, ", got ", t.scalar_type(), " ",
                    t.sizes(), ", strides ", t.strides(), ", on ", t.device());
  on_device(name, t, dev);
}

// A parameter or state that the library reads by 16 bytes: itself, or a copy where it is a view that
// begins between them (a parameter in a flat buffer).
Tensor by_16(const Tensor& t) { return ((uintptr_t)ptr(t) & 15u) == 0 ? t : t.detach().clone(); }

// Token stride of a [..., inner dimensions] activation (0: contiguous), -1 if its rows are not
// contiguous and evenly spaced.
long long token_stride(const Tensor& t, int inner) {
  if (t.is_contiguous()) return 0;
  const int64_t n = t.dim();
  int64_t width = 1;
  for (int64_t k = n - 1; k >= n - inner; --k) {
    if (t.size(k) != 1 && t.stride(k) != width) return -1;
    width *= t.size(k);
  }
  int64_t ld = 0, span = 0;  // innermost leading dimension's stride; what the next one's has to be
  for (int64_t k = n - inner - 1; k >= 0; --k) {
    if (t.size(k) == 1) continue;
    if (t.stride(k) < width) return -1;  // rows that overlap: a broadcast dimension's stride is 0
    if (ld == 0)
      ld = t.stride(k);
    else if (t.stride(k) != span)
      return -1;
    span = t.stride(k) * t.size(k);
  }
  return ld;
}
long long strided(const char* name, const Tensor& t, int inner) {
  const long long ld = token_stride(t, inner);
  TORCH_CHECK_VALUE(ld >= 0, name, ": rows must be contiguous and evenly spaced over the batch, got shape ", t.sizes(),
                    ", strides ", t.strides());
  return ld;
}

int sequences(const Tensor& cu, int64_t B, at::Device dev, const char* name = "cu_seqlens") {
  if (!cu.defined()) return size32("x", B);
  TORCH_CHECK_VALUE(cu.is_cuda() && cu.scalar_type() == at::kInt && cu.dim() == 1 && cu.numel() >= 2 && cu.is_contiguous(),
                    name, ": expected a contiguous CUDA int32 vector of at least 2 entries");
  on_device(name, cu, dev);
  TORCH_CHECK_VALUE(B == 1, name, " needs a batch of 1 (the packed tokens)");
  return size32(name, cu.numel()) - 1;
}

void check_slots(const Tensor& slots, const Tensor& state, int64_t B, at::Device dev) {
  if (slots.defined()) {
    TORCH_CHECK_VALUE(slots.is_cuda() && slots.scalar_type() == at::kInt && slots.is_contiguous() && slots.dim() == 1 &&
                          slots.size(0) == B,
                      "slots: expected a contiguous CUDA int32 vector of ", B, " entries");
    on_device("slots", slots, dev);
  } else {
    TORCH_CHECK_VALUE(state.size(0) >= B, "state: ", state.size(0), " states for ", B, " rows");
  }
}

gdr_stream_t stream_of(const Tensor& t) { return (gdr_stream_t)c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

// Uninitialised, on the current stream; without the dispatcher, which takes as long as the allocation.
Tensor fresh_of(IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
Tensor fresh(IntArrayRef shape, const Tensor& like) { return fresh_of(shape, like.scalar_type(), like); }
Tensor fresh_f32(IntArrayRef shape, const Tensor& like) { return fresh_of(shape, at::kFloat, like); }
// The caller's workspace, whose status it can ask for, or one of the bytes that the call needs (torch's
// blocks are 512-byte aligned).  What the caller's holds too little of, the library refuses.
struct Workspace {
  Tensor t;
  size_t bytes;
  Workspace(size_t need, const Tensor& like) : bytes(need) {
    if (need) t = fresh_of({(int64_t)need}, at::kByte, like);
  }
  Workspace(const Tensor& given, size_t need, const Tensor& like) : Workspace(given.defined() ? 0 : need, like) {
    if (!given.defined()) return;
    TORCH_CHECK_VALUE(given.is_cuda() && given.is_contiguous(), "workspace: expected a contiguous CUDA tensor");
    on_device("workspace", given, like.device());
    t = given;
    bytes = given.nbytes();
  }
};

PyObject* answer(gdr_status st, const Tensor& t) { return st == GDR_OK ? THPVariable_Wrap(t) : PyLong_FromLong(st); }
PyObject* answer(gdr_status st, std::initializer_list<Tensor> ts) {
  if (st != GDR_OK) return PyLong_FromLong(st);
  PyObject* tuple = PyTuple_New((Py_ssize_t)ts.size());
  if (!tuple) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(tuple, i++, THPVariable_Wrap(t));
  return tuple;
}

// After a call that changed t in place: its version tells autograd, which may have saved it.  (Tensors of
// inference mode have none.)
gdr_status changed(const Tensor& t, gdr_status st) {
  if (st == GDR_OK && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return st;
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// ---------------------------------------------------------------------------------- convolution
gdr_conv_problem conv_problem(const Tensor& x, const Tensor& w, const Tensor& b, const Tensor& state, const Tensor& cu,
                              long silu, const Tensor& dy) {
  TORCH_CHECK_VALUE(x.dim() == 3, "x: expected [B, T, C], got ", x.sizes());
  const int64_t B = x.size(0), T = x.size(1), C = x.size(2), W = w.size(-1);
  const auto type = x.scalar_type();
  const at::Device dev = x.device();
  gdr_conv_problem p = {};
  p.dtype = type_code(type);
  p.B = size32("x", B);
  p.T = size32("x", T);
  p.C = size32("x", C);
  p.W = size32("weight", W);
  act("x", x, {B, T, C}, type, dev);
  full("weight", w, {C, W}, dev);
  full("bias", b, {C}, dev);
  p.num_seqs = sequences(cu, B, dev);
  full("initial_state", state, {p.num_seqs, W - 1, C}, dev, type);
  p.cu_seqlens = (const int32_t*)ptr(cu);
  p.silu = (int)silu;
  p.ld_x = strided("x", x, 1);
  if (dy.defined()) {
    act("dy", dy, {B, T, C}, type, dev);
    p.ld_dy = strided("dy", dy, 1);
  }
  return p;
}

// x, weight, bias, initial_state, cu_seqlens, silu, output_final_state, workspace
PyObject* conv_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor &x = required(a[0], "x"), &w = required(a[1], "weight"), &b = tensor(a[2], "bias"),
               &state = tensor(a[3], "initial_state"), &cu = tensor(a[4], "cu_seqlens"), &given = tensor(a[7], "workspace");
  const gdr_conv_problem p = conv_problem(x, w, b, state, cu, integer(a[5]), kNone);
  const OnDevice current(x.device());
  const Tensor y = fresh(x.sizes(), x), last = integer(a[6]) ? fresh({p.num_seqs, p.W - 1, p.C}, x) : Tensor();
  const Workspace ws(given, cu.defined() ? lib.gdr_conv_fwd_workspace_bytes(&p) : 0, x);
  return answer(lib.gdr_conv_fwd(&p, ptr(x), (const float*)ptr(w), (const float*)ptr(b), ptr(state), ptr(y), ptr(last),
                                 ptr(ws.t), ws.bytes, stream_of(x)),
                {y, last});
  END_HANDLE_TH_ERRORS
}

// x, weight, bias, dy, initial_state, dfinal_state, cu_seqlens, silu, workspace
PyObject* conv_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor &x = required(a[0], "x"), &w = required(a[1], "weight"), &b = tensor(a[2], "bias"), &dy = required(a[3], "dy"),
               &state = tensor(a[4], "initial_state"), &dlast = tensor(a[5], "dfinal_state"), &cu = tensor(a[6], "cu_seqlens"),
               &given = tensor(a[8], "workspace");
  const gdr_conv_problem p = conv_problem(x, w, b, state, cu, integer(a[7]), dy);
  full("dfinal_state", dlast, {p.num_seqs, p.W - 1, p.C}, x.device(), x.scalar_type());
  const OnDevice current(x.device());
  const Tensor dx = fresh(x.sizes(), x), dw = fresh(w.sizes(), w), db = b.defined() ? fresh(b.sizes(), b) : Tensor(),
               dstate = state.defined() ? fresh(state.sizes(), state) : Tensor();
  const Workspace ws(given, lib.gdr_conv_bwd_workspace_bytes(&p), x);
  return answer(lib.gdr_conv_bwd(&p, ptr(x), (const float*)ptr(w), (const float*)ptr(b), ptr(state), ptr(dy), ptr(dlast),
                                 ptr(dx), (float*)ptr(dw), (float*)ptr(db), ptr(dstate), ptr(ws.t), ws.bytes,
                                 stream_of(x)),
                {dx, dw, db, dstate});
  END_HANDLE_TH_ERRORS
}

// x, state, weight, bias, slots, silu
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Tensor &x = required(a[0], "x"), &state = required(a[1], "state"), &w = required(a[2], "weight"),
               &b = tensor(a[3], "bias"), &slots = tensor(a[4], "slots");
  TORCH_CHECK_VALUE(x.dim() == 2 && state.dim() == 3, "expected x [B, C] and state [num_slots, W - 1, C], got ", x.sizes(),
                    " and ", state.sizes());
  const int64_t B = x.size(0), C = x.size(1), W = w.size(-1);
  const auto type = x.scalar_type();
  const at::Device dev = x.device();
  gdr_conv_problem p = {};
  p.dtype = type_code(type);
  p.B = p.num_seqs = size32("x", B);
  p.T = 1;
  p.C = size32("x", C);
  p.W = size32("weight", W);
  p.num_slots = size32("state", state.size(0));
  act("x", x, {B, C}, type, dev);
  full("weight", w, {C, W}, dev);
  full("bias", b, {C}, dev);
  full("state", state, {state.size(0), W - 1, C}, dev, type);
  check_slots(slots, state, B, dev);
  p.silu = (int)integer(a[5]);
  p.ld_x = strided("x", x, 1);
  const OnDevice current(dev);
  const Tensor y = fresh({B, C}, x);
  return answer(changed(state, lib.gdr_conv_step(&p, ptr(x), (const float*)ptr(w), (const float*)ptr(b), ptr(state),
                                                 (const int32_t*)ptr(slots), ptr(y), stream_of(x))),
                y);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------- selective scan
struct SsmTensors {
  const Tensor &x, &dt, &A, &Bm, &Cm, &D, &bias;
};
// lead: dimensions in front of the channels (2: [B, T, ...], 1: one token of [B, ...])
gdr_ssm_problem ssm_problem(const SsmTensors& t, int lead, const Tensor& cu, long softplus, const Tensor& dy) {
  TORCH_CHECK_VALUE(t.x.dim() == lead + 1 && t.Bm.dim() == lead + 2, "expected x [", lead == 2 ? "B, T" : "B", ", D] and Bm, Cm [",
                    lead == 2 ? "B, T" : "B", ", G, N], got ", t.x.sizes(), " and ", t.Bm.sizes());
  const int64_t B = t.x.size(0), T = lead == 2 ? t.x.size(1) : 1, D = t.x.size(-1), G = t.Bm.size(-2), N = t.Bm.size(-1);
  const auto type = t.x.scalar_type();
  const at::Device dev = t.x.device();
  gdr_ssm_problem p = {};
  p.dtype = type_code(type);
  p.B = size32("x", B);
  p.T = size32("x", T);
  p.D = size32("x", D);
  p.N = size32("Bm", N);
  p.G = size32("Bm", G);
  const std::array<int64_t, 3> row2 = {B, T, D};
  const std::array<int64_t, 4> bc2 = {B, T, G, N};
  const std::array<int64_t, 2> row1 = {B, D};
  const std::array<int64_t, 3> bc1 = {B, G, N};
  const IntArrayRef row = lead == 2 ? IntArrayRef(row2) : IntArrayRef(row1), bc = lead == 2 ? IntArrayRef(bc2) : IntArrayRef(bc1);
  act("x", t.x, row, type, dev);
  act("dt", t.dt, row, type, dev);
  act("Bm", t.Bm, bc, type, dev);
  act("Cm", t.Cm, bc, type, dev);
  full("A", t.A, {D, N}, dev);
  full("D", t.D, {D}, dev);
  full("dt_bias", t.bias, {D}, dev);
  p.num_seqs = sequences(cu, B, dev);
  p.cu_seqlens = (const int32_t*)ptr(cu);
  p.dt_softplus = (int)softplus;
  p.ld_x = strided("x", t.x, 1);
  p.ld_dt = strided("dt", t.dt, 1);
  p.ld_b = strided("Bm", t.Bm, 2);
  p.ld_c = strided("Cm", t.Cm, 2);
  if (dy.defined()) {
    act("dy", dy, row, type, dev);
    p.ld_dy = strided("dy", dy, 1);
  }
  return p;
}

// x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus, output_final_state, save, workspace
PyObject* ssm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 13);
  const SsmTensors t{required(a[0], "x"), required(a[1], "dt"), required(a[2], "A"), required(a[3], "Bm"),
                     required(a[4], "Cm"), tensor(a[5], "D"), tensor(a[6], "dt_bias")};
  const Tensor &S0 = tensor(a[7], "S0"), &cu = tensor(a[8], "cu_seqlens"), &given = tensor(a[12], "workspace");
  const gdr_ssm_problem p = ssm_problem(t, 2, cu, integer(a[9]), kNone);
  full("S0", S0, {p.num_seqs, p.D, p.N}, t.x.device());
  const OnDevice current(t.x.device());
  const Tensor y = fresh(t.x.sizes(), t.x), S_T = integer(a[10]) ? fresh_f32({p.num_seqs, p.D, p.N}, t.x) : Tensor(),
               saved = integer(a[11]) ? fresh_f32({(int64_t)(lib.gdr_ssm_saved_bytes(&p) / 4)}, t.x) : Tensor();
  const Tensor A = by_16(t.A), start = by_16(S0);
  const Workspace ws(given, lib.gdr_ssm_fwd_workspace_bytes(&p), t.x);
  return answer(lib.gdr_ssm_fwd(&p, ptr(t.x), ptr(t.dt), (const float*)ptr(A), ptr(t.Bm), ptr(t.Cm), (const float*)ptr(t.D),
                                (const float*)ptr(t.bias), (const float*)ptr(start), ptr(y), (float*)ptr(S_T), (float*)ptr(saved),
                                ptr(ws.t), ws.bytes, stream_of(t.x)),
                {y, S_T, saved});
  END_HANDLE_TH_ERRORS
}

// x, dt, A, Bm, Cm, h_saved, dy, D, dt_bias, dS_T, cu_seqlens, dt_softplus, want_dS0, workspace
PyObject* ssm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 14);
  const SsmTensors t{required(a[0], "x"), required(a[1], "dt"), required(a[2], "A"), required(a[3], "Bm"),
                     required(a[4], "Cm"), tensor(a[7], "D"), tensor(a[8], "dt_bias")};
  const Tensor &saved = tensor(a[5], "h_saved"), &dy = required(a[6], "dy"), &dS_T = tensor(a[9], "dS_T"),
               &cu = tensor(a[10], "cu_seqlens"), &given = tensor(a[13], "workspace");
  const gdr_ssm_problem p = ssm_problem(t, 2, cu, integer(a[11]), dy);
  full("dS_T", dS_T, {p.num_seqs, p.D, p.N}, t.x.device());
  const int64_t need = (int64_t)(lib.gdr_ssm_saved_bytes(&p) / 4);
  TORCH_CHECK_VALUE(saved.defined() && saved.is_cuda() && saved.scalar_type() == at::kFloat && saved.is_contiguous() &&
                        saved.numel() >= need,
                    "h_saved: expected the ", need, " floats that ssm_forward kept (save=True)");
  on_device("h_saved", saved, t.x.device());
  const OnDevice current(t.x.device());
  const Tensor dx = fresh(t.x.sizes(), t.x), ddt = fresh(t.x.sizes(), t.x), dB = fresh(t.Bm.sizes(), t.x),
               dC = fresh(t.Bm.sizes(), t.x), dA = fresh(t.A.sizes(), t.A),
               dD = t.D.defined() ? fresh(t.D.sizes(), t.D) : Tensor(), db = t.bias.defined() ? fresh(t.bias.sizes(), t.bias) : Tensor(),
               dS0 = integer(a[12]) ? fresh_f32({p.num_seqs, p.D, p.N}, t.x) : Tensor();
  const Tensor A = by_16(t.A), end = by_16(dS_T), states = by_16(saved);
  const Workspace ws(given, lib.gdr_ssm_bwd_workspace_bytes(&p), t.x);
  return answer(lib.gdr_ssm_bwd(&p, ptr(t.x), ptr(t.dt), (const float*)ptr(A), ptr(t.Bm), ptr(t.Cm), (const float*)ptr(t.D),
                                (const float*)ptr(t.bias), (const float*)ptr(states), ptr(dy), (const float*)ptr(end), ptr(dx),
                                ptr(ddt), (float*)ptr(dA), ptr(dB), ptr(dC), (float*)ptr(dD), (float*)ptr(db), (float*)ptr(dS0),
                                ptr(ws.t), ws.bytes, stream_of(t.x)),
                {dx, ddt, dA, dB, dC, dD, db, dS0});
  END_HANDLE_TH_ERRORS
}

// x, dt, A, Bm, Cm, state, D, dt_bias, slots, dt_softplus
PyObject* ssm_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  const SsmTensors t{required(a[0], "x"), required(a[1], "dt"), required(a[2], "A"), required(a[3], "Bm"),
                     required(a[4], "Cm"), tensor(a[6], "D"), tensor(a[7], "dt_bias")};
  const Tensor &state = required(a[5], "state"), &slots = tensor(a[8], "slots");
  gdr_ssm_problem p = ssm_problem(t, 1, kNone, integer(a[9]), kNone);
  TORCH_CHECK_VALUE(state.dim() == 3, "state: expected [num_slots, D, N], got ", state.sizes());
  const at::Device dev = t.x.device();
  full("state", state, {state.size(0), p.D, p.N}, dev);
  check_slots(slots, state, p.B, dev);
  p.num_slots = size32("state", state.size(0));
  const OnDevice current(dev);
  const Tensor A = by_16(t.A), y = fresh({p.B, p.D}, t.x);
  return answer(changed(state, lib.gdr_ssm_step(&p, ptr(t.x), ptr(t.dt), (const float*)ptr(A), ptr(t.Bm), ptr(t.Cm),
                                                (const float*)ptr(t.D), (const float*)ptr(t.bias), (float*)ptr(state),
                                                (const int32_t*)ptr(slots), ptr(y), stream_of(t.x))),
                y);
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------------- block norms
gdr_norm_problem norm_problem(const Tensor& x, const Tensor& post, const Tensor& gate, const Tensor& scale, const Tensor& pre,
                              at::ScalarType stream_type, double eps) {
  TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) > 0, "x: expected [..., D], got ", x.sizes());
  const int64_t D = x.size(-1);
  const auto type = x.scalar_type();
  const at::Device dev = x.device();
  gdr_norm_problem p = {};
  p.dtype = type_code(type);
  p.res_dtype = type_code(stream_type);
  p.D = size32("x", D);
  act("x", x, x.sizes(), type, dev);
  if (gate.defined()) act("gate", gate, x.sizes(), type, dev);
  full("post_weight", post, {D}, dev);
  full("scale", scale, {D}, dev);
  full("pre_weight", pre, {D}, dev);
  p.eps = (float)eps;
  p.heads = 1;
  p.tokens = x.numel() / D;
  // rows one by one; else heads of a token side by side, as in a slice of a wider tensor
  p.ld_x = token_stride(x, 1);
  p.ld_gate = gate.defined() ? token_stride(gate, 1) : 0;
  if ((p.ld_x < 0 || p.ld_gate < 0) && x.dim() > 2) {
    p.heads = size32("x", x.size(-2));
    p.tokens = p.heads ? x.numel() / D / p.heads : 0;
    p.ld_x = strided("x", x, 2);
    p.ld_gate = gate.defined() ? strided("gate", gate, 2) : 0;
  } else {
    strided("x", x, 1);
    if (gate.defined()) strided("gate", gate, 1);
  }
  return p;
}

// x, post_weight, gate, scale, residual, pre_weight, eps
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor &x = required(a[0], "x"), &post = tensor(a[1], "post_weight"), &gate = tensor(a[2], "gate"),
               &scale = tensor(a[3], "scale"), &res = tensor(a[4], "residual"), &pre = tensor(a[5], "pre_weight");
  const auto type = res.defined() ? res.scalar_type() : x.scalar_type();
  const gdr_norm_problem p = norm_problem(x, post, gate, scale, pre, type, number(a[6]));
  full("residual", res, x.sizes(), x.device(), type);
  const OnDevice current(x.device());
  const Tensor r = res.defined() ? fresh(x.sizes(), res) : pre.defined() ? Tensor() : fresh(x.sizes(), x),
               y = pre.defined() ? fresh(x.sizes(), x) : Tensor();
  return answer(lib.gdr_norm_fwd(&p, ptr(x), (const float*)ptr(post), ptr(gate), (const float*)ptr(scale), ptr(res),
                                 (const float*)ptr(pre), ptr(r), ptr(y), stream_of(x)),
                {r, y});
  END_HANDLE_TH_ERRORS
}

// x, post_weight, gate, scale, r (None: no residual), pre_weight, dr, dy, eps
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor &x = required(a[0], "x"), &post = tensor(a[1], "post_weight"), &gate = tensor(a[2], "gate"),
               &scale = tensor(a[3], "scale"), &r = tensor(a[4], "r"), &pre = tensor(a[5], "pre_weight"),
               &dr = tensor(a[6], "dr"), &dy = tensor(a[7], "dy");
  const bool has_residual = r.defined();
  const auto type = has_residual ? r.scalar_type() : x.scalar_type();
  const gdr_norm_problem p = norm_problem(x, post, gate, scale, pre, type, number(a[8]));
  const at::Device dev = x.device();
  full("r", r, x.sizes(), dev, type);
  full("dr", dr, x.sizes(), dev, type);
  full("dy", dy, x.sizes(), dev, x.scalar_type());
  TORCH_CHECK_VALUE(has_residual || !pre.defined() || x.is_contiguous(), "x: a plain norm's backward needs a contiguous x");
  const OnDevice current(dev);
  const Tensor dx = fresh(x.sizes(), x), dgate = gate.defined() ? fresh(x.sizes(), x) : Tensor(),
               dres = has_residual ? fresh(x.sizes(), r) : Tensor(), dpost = post.defined() ? fresh(post.sizes(), post) : Tensor(),
               dscale = scale.defined() ? fresh(scale.sizes(), scale) : Tensor(),
               dpre = pre.defined() ? fresh(pre.sizes(), pre) : Tensor();
  const Workspace ws(lib.gdr_norm_bwd_workspace_bytes(&p), x);
  const void* normed = has_residual ? ptr(r) : pre.defined() ? ptr(x) : nullptr;  // what w_pre was applied to
  return answer(lib.gdr_norm_bwd(&p, ptr(x), (const float*)ptr(post), ptr(gate), (const float*)ptr(scale), normed,
                                 (const float*)ptr(pre), has_residual, ptr(dr), ptr(dy), ptr(dx), ptr(dgate), ptr(dres),
                                 (float*)ptr(dpost), (float*)ptr(dscale), (float*)ptr(dpre), ptr(ws.t), ws.bytes, stream_of(x)),
                {dx, dgate, dres, dpost, dscale, dpre});
  END_HANDLE_TH_ERRORS
}

// ----------------------------------------------------------------- the delta rule, one token each
// q, k, v, g, beta, state, layout, scale, slots, prologue
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  const Tensor &q = required(a[0], "q"), &k = required(a[1], "k"), &v = required(a[2], "v"), &g = required(a[3], "g"),
               &beta = required(a[4], "beta"), &state = required(a[5], "state"), &slots = tensor(a[8], "slots");
  TORCH_CHECK_VALUE(q.dim() == 3 && v.dim() == 3 && state.dim() == 4, "expected q [B, Hk, DK], v [B, Hv, DV] and a state of four dimensions, got ",
                    q.sizes(), ", ", v.sizes(), " and ", state.sizes());
  const auto type = q.scalar_type();
  const at::Device dev = q.device();
  const int64_t B = q.size(0), Hk = q.size(1), DK = q.size(2), Hv = v.size(1), DV = v.size(2);
  gdr_problem p = {};
  p.dtype = type_code(type);
  p.layout = (gdr_state_layout)integer(a[6]);
  p.B = p.num_seqs = size32("q", B);
  p.T = 1;
  p.Hk = size32("q", Hk);
  p.Hv = size32("v", Hv);
  p.DK = size32("q", DK);
  p.DV = size32("v", DV);
  const int num_slots = size32("state", state.size(0));
  full("q", q, {B, Hk, DK}, dev, type);
  full("k", k, {B, Hk, DK}, dev, type);
  full("v", v, {B, Hv, DV}, dev, type);
  full("g", g, {B, Hv}, dev);
  full("beta", beta, {B, Hv}, dev, type);
  const bool kv = p.layout == GDR_STATE_KV;
  full("state", state, {state.size(0), Hv, kv ? DK : DV, kv ? DV : DK}, dev);
  check_slots(slots, state, B, dev);
  p.scale = (float)number(a[7]);
  p.prologue = (unsigned)integer(a[9]);
  const OnDevice current(dev);
  const Tensor o = fresh({B, Hv, DV}, v);
  return answer(changed(state, lib.gdr_step(&p, ptr(q), ptr(k), ptr(v), (const float*)ptr(g), ptr(beta), (float*)ptr(state),
                                            num_slots, (const int32_t*)ptr(slots), ptr(o), stream_of(q))),
                o);
  END_HANDLE_TH_ERRORS
}

// ----------------------------------------------------------------------------- rotary positions
// q, k (or None), freqs, positions, cu_seqlens, interleaved, inverse, scale, workspace
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor &q = required(a[0], "q"), &k = tensor(a[1], "k"), &freqs = required(a[2], "freqs"), &positions = tensor(a[3], "positions"),
               &cu = tensor(a[4], "cu_seqlens"), &given = tensor(a[8], "workspace");
  TORCH_CHECK_VALUE(q.dim() == 4 || q.dim() == 3, "q: expected [B, T, H, D] or [B, H, D], got ", q.sizes());
  const bool rows = q.dim() == 3;
  TORCH_CHECK_VALUE(!rows || positions.defined(), "positions: single tokens [B, H, D] need them");
  const int64_t B = q.size(0), T = rows ? 1 : q.size(1), D = q.size(-1);
  const auto type = q.scalar_type();
  const at::Device dev = q.device();
  gdr_rope_problem p = {};
  p.dtype = type_code(type);
  p.B = size32("q", B);
  p.T = size32("q", T);
  p.Hq = size32("q", q.size(-2));
  p.D = size32("q", D);
  act("q", q, q.sizes(), type, dev);
  p.ld_q = strided("q", q, 2);
  if (k.defined()) {
    TORCH_CHECK_VALUE(k.dim() == q.dim(), "k: expected ", q.dim(), " dimensions, got ", k.sizes());
    p.Hk = size32("k", k.size(-2));
    if (rows)
      act("k", k, {B, k.size(-2), D}, type, dev);
    else
      act("k", k, {B, T, k.size(-2), D}, type, dev);
    p.ld_k = strided("k", k, 2);
  }
  TORCH_CHECK_VALUE(freqs.dim() == 1, "freqs: expected a vector, got ", freqs.sizes());
  full("freqs", freqs, freqs.sizes(), dev, at::kDouble);
  p.R = size32("freqs", 2 * freqs.size(0));
  if (rows)
    full("positions", positions, {B}, dev, at::kInt);
  else
    full("positions", positions, {B, T}, dev, at::kInt);
  p.num_seqs = sequences(cu, B, dev);
  p.cu_seqlens = positions.defined() ? nullptr : (const int32_t*)ptr(cu);
  if (positions.defined()) p.num_seqs = p.B;
  p.interleaved = (int)integer(a[5]);
  p.inverse = (int)integer(a[6]);
  p.scale = (float)number(a[7]);
  const OnDevice current(dev);
  const Tensor q_out = fresh(q.sizes(), q), k_out = k.defined() ? fresh(k.sizes(), k) : Tensor();
  const Workspace ws(given, p.cu_seqlens ? lib.gdr_rope_workspace_bytes(&p) : 0, q);
  return answer(lib.gdr_rope(&p, ptr(q), ptr(k), (const double*)ptr(freqs), (const int32_t*)ptr(positions), ptr(q_out), ptr(k_out),
                             ptr(ws.t), ws.bytes, stream_of(q)),
                {q_out, k_out});
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------------ attention
gdr_attn_problem attn_problem(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, const Tensor& cu_k, long causal,
                              long window, double scale, const Tensor& dout) {
  TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4, "expected q [B, Tq, Hq, D] and k, v [B, Tk, Hk, D], got ", q.sizes(), " and ", k.sizes());
  const int64_t B = q.size(0), D = q.size(3);
  const auto type = q.scalar_type();
  const at::Device dev = q.device();
  gdr_attn_problem p = {};
  p.dtype = type_code(type);
  p.B = size32("q", B);
  p.Tq = size32("q", q.size(1));
  p.Tk = size32("k", k.size(1));
  p.Hq = size32("q", q.size(2));
  p.Hk = size32("k", k.size(2));
  p.D = size32("q", D);
  act("q", q, q.sizes(), type, dev);
  act("k", k, {B, k.size(1), k.size(2), D}, type, dev);
  act("v", v, k.sizes(), type, dev);
  p.ld_q = strided("q", q, 2);
  p.ld_k = strided("k", k, 2);
  p.ld_v = strided("v", v, 2);
  if (dout.defined()) {
    act("do", dout, q.sizes(), type, dev);
    p.ld_do = strided("do", dout, 2);
  }
  p.num_seqs = sequences(cu, B, dev);
  TORCH_CHECK_VALUE(cu.defined() || !cu_k.defined(), "cu_seqlens_k needs cu_seqlens");
  const Tensor& keys = cu_k.defined() ? cu_k : cu;
  if (cu_k.defined())
    TORCH_CHECK_VALUE(sequences(cu_k, B, dev, "cu_seqlens_k") == p.num_seqs, "cu_seqlens_k: expected ", p.num_seqs + 1, " entries, got ", cu_k.numel());
  p.cu_q = (const int32_t*)ptr(cu);
  p.cu_k = (const int32_t*)ptr(keys);
  p.causal = (int)causal;
  TORCH_CHECK_VALUE(window >= 0, "window: ", window, " is negative");
  p.window = window > INT_MAX ? 0 : (int)window;  // wider than any sequence: none
  p.scale = (float)scale;
  return p;
}

// q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace
PyObject* attn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor &q = required(a[0], "q"), &k = required(a[1], "k"), &v = required(a[2], "v"), &cu = tensor(a[3], "cu_seqlens"),
               &cu_k = tensor(a[4], "cu_seqlens_k"), &given = tensor(a[8], "workspace");
  const gdr_attn_problem p = attn_problem(q, k, v, cu, cu_k, integer(a[5]), integer(a[6]), number(a[7]), kNone);
  const OnDevice current(q.device());
  const Tensor o = fresh(q.sizes(), q), lse = fresh_f32({p.B, p.Hq, p.Tq}, q);
  const Workspace ws(given, lib.gdr_attn_fwd_workspace_bytes(&p), q);
  return answer(lib.gdr_attn_fwd(&p, ptr(q), ptr(k), ptr(v), ptr(o), (float*)ptr(lse), ptr(ws.t), ws.bytes, stream_of(q)), {o, lse});
  END_HANDLE_TH_ERRORS
}

// q, k, v, o, lse, do, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace
PyObject* attn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const Tensor &q = required(a[0], "q"), &k = required(a[1], "k"), &v = required(a[2], "v"), &o = required(a[3], "o"),
               &lse = required(a[4], "lse"), &dout = required(a[5], "do"), &cu = tensor(a[6], "cu_seqlens"),
               &cu_k = tensor(a[7], "cu_seqlens_k"), &given = tensor(a[11], "workspace");
  const gdr_attn_problem p = attn_problem(q, k, v, cu, cu_k, integer(a[8]), integer(a[9]), number(a[10]), dout);
  full("o", o, q.sizes(), q.device(), q.scalar_type());
  full("lse", lse, {p.B, p.Hq, p.Tq}, q.device());
  const OnDevice current(q.device());
  const Tensor dq = fresh(q.sizes(), q), dk = fresh(k.sizes(), k), dv = fresh(v.sizes(), v);
  const Workspace ws(given, lib.gdr_attn_bwd_workspace_bytes(&p), q);
  return answer(lib.gdr_attn_bwd(&p, ptr(q), ptr(k), ptr(v), ptr(o), (const float*)ptr(lse), ptr(dout), ptr(dq), ptr(dk), ptr(dv),
                                 ptr(ws.t), ws.bytes, stream_of(q)),
                {dq, dk, dv});
  END_HANDLE_TH_ERRORS
}

// The caches and the block table of B rows of heads [Hk, D].
void cache_pages(gdr_cache_problem* p, const Tensor& k_cache, const Tensor& v_cache, const Tensor& table, int64_t B, int64_t Hk, int64_t D,
                 at::ScalarType type, at::Device dev) {
  TORCH_CHECK_VALUE(k_cache.dim() == 4 && table.dim() == 2, "expected k_cache [num_pages, page_size, Hk, D] and block_table [B, max_pages], got ",
                    k_cache.sizes(), " and ", table.sizes());
  full("k_cache", k_cache, {k_cache.size(0), k_cache.size(1), Hk, D}, dev, type);
  full("v_cache", v_cache, k_cache.sizes(), dev, type);
  full("block_table", table, {B, table.size(1)}, dev, at::kInt);
  p->num_pages = size32("k_cache", k_cache.size(0));
  p->page_size = size32("k_cache", k_cache.size(1));
  p->max_pages = size32("block_table", table.size(1));
}
gdr_status both_changed(const Tensor& k_cache, const Tensor& v_cache, gdr_status st) { return changed(v_cache, changed(k_cache, st)); }

// q, k, v, k_cache, v_cache, block_table, lengths, window, scale, workspace
PyObject* attn_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  const Tensor &q = required(a[0], "q"), &k = required(a[1], "k"), &v = required(a[2], "v"), &kc = required(a[3], "k_cache"),
               &vc = required(a[4], "v_cache"), &table = required(a[5], "block_table"), &lengths = required(a[6], "lengths"),
               &given = tensor(a[9], "workspace");
  TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3, "expected q [B, Hq, D] and k, v [B, Hk, D], got ", q.sizes(), " and ", k.sizes());
  const int64_t B = q.size(0), Hk = k.size(1), D = q.size(2);
  const auto type = q.scalar_type();
  const at::Device dev = q.device();
  gdr_cache_problem p = {};
  p.dtype = type_code(type);
  p.B = size32("q", B);
  p.T = 1;
  p.Hq = size32("q", q.size(1));
  p.Hk = size32("k", Hk);
  p.D = size32("q", D);
  act("q", q, q.sizes(), type, dev);
  act("k", k, {B, Hk, D}, type, dev);
  act("v", v, {B, Hk, D}, type, dev);
  p.ld_q = strided("q", q, 2);
  p.ld_k = strided("k", k, 2);
  p.ld_v = strided("v", v, 2);
  cache_pages(&p, kc, vc, table, B, Hk, D, type, dev);
  full("lengths", lengths, {B}, dev, at::kInt);
  const long window = integer(a[7]);
  TORCH_CHECK_VALUE(window >= 0, "window: ", window, " is negative");
  p.window = window > INT_MAX ? 0 : (int)window;
  p.scale = (float)number(a[8]);
  const OnDevice current(dev);
  const Tensor o = fresh(q.sizes(), q);
  const Workspace ws(given, lib.gdr_attn_step_workspace_bytes(&p), q);
  return answer(both_changed(kc, vc, lib.gdr_attn_step(&p, ptr(q), ptr(k), ptr(v), ptr(kc), ptr(vc), (const int32_t*)ptr(table),
                                                       (const int32_t*)ptr(lengths), ptr(o), ptr(ws.t), ws.bytes, stream_of(q))),
                o);
  END_HANDLE_TH_ERRORS
}

// k, v, k_cache, v_cache, block_table, starts, cu_seqlens, workspace
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor &k = required(a[0], "k"), &v = required(a[1], "v"), &kc = required(a[2], "k_cache"), &vc = required(a[3], "v_cache"),
               &table = required(a[4], "block_table"), &starts = tensor(a[5], "starts"), &cu = tensor(a[6], "cu_seqlens"),
               &given = tensor(a[7], "workspace");
  TORCH_CHECK_VALUE(k.dim() == 4, "k: expected [B, T, Hk, D], got ", k.sizes());
  const int64_t Hk = k.size(2), D = k.size(3);
  const auto type = k.scalar_type();
  const at::Device dev = k.device();
  gdr_cache_problem p = {};
  p.dtype = type_code(type);
  p.T = size32("k", k.size(1));
  p.Hk = size32("k", Hk);
  p.D = size32("k", D);
  act("k", k, k.sizes(), type, dev);
  act("v", v, k.sizes(), type, dev);
  p.ld_k = strided("k", k, 2);
  p.ld_v = strided("v", v, 2);
  p.B = sequences(cu, k.size(0), dev);
  p.cu_seqlens = (const int32_t*)ptr(cu);
  cache_pages(&p, kc, vc, table, p.B, Hk, D, type, dev);
  full("starts", starts, {p.B}, dev, at::kInt);
  const OnDevice current(dev);
  const Workspace ws(given, lib.gdr_cache_write_workspace_bytes(&p), k);
  const gdr_status st = both_changed(kc, vc, lib.gdr_cache_write(&p, ptr(k), ptr(v), ptr(kc), ptr(vc), (const int32_t*)ptr(table),
                                                                 (const int32_t*)ptr(starts), ptr(ws.t), ws.bytes, stream_of(k)));
  if (st != GDR_OK) return PyLong_FromLong(st);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// tensor, inner dimensions: token_stride
PyObject* stride(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 2);
  return PyLong_FromLongLong(token_stride(required(a[0], "tensor"), (int)integer(a[1])));
  END_HANDLE_TH_ERRORS
}

// {entry point's name: address}
PyObject* bind(PyObject*, PyObject* table) {
  HANDLE_TH_ERRORS
  auto address = [&](const char* name) {
    PyObject* v = PyDict_GetItemString(table, name);
    TORCH_CHECK_VALUE(v != nullptr, "no address of ", name);
    void* p = PyLong_AsVoidPtr(v);
    TORCH_CHECK_VALUE(p != nullptr, "no address of ", name);
    return p;
  };
  Library l;
#define GDR_BIND(name) l.name = reinterpret_cast<decltype(l.name)>(address(#name));
  GDR_ENTRIES(GDR_BIND)
#undef GDR_BIND
  lib = l;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define GDR_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDR_METHOD(conv_forward), GDR_METHOD(conv_backward), GDR_METHOD(conv_step), GDR_METHOD(ssm_forward),
                         GDR_METHOD(ssm_backward), GDR_METHOD(ssm_step), GDR_METHOD(norm_forward), GDR_METHOD(norm_backward),
                         GDR_METHOD(step), GDR_METHOD(rope), GDR_METHOD(attn_forward), GDR_METHOD(attn_backward), GDR_METHOD(attn_step),
                         GDR_METHOD(cache_write), GDR_METHOD(stride), {"bind", bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef definition = {PyModuleDef_HEAD_INIT, "gdr_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdr_binding(void) { return PyModule_Create(&definition); }

// zc_torch.cpp -- the operator calls of zipccl.h on torch tensors: checks of
// the tensors, allocation of the results, the call.  It is a Python extension
// because a call on a few tokens is bound by the host: allocating two results
// and launching takes 8 us from Python on the Arm host, all checks included
// 12, and the kernel 3.
//
// Every function takes all its arguments by position (operators.py has the
// keywords and defaults); None stands for what is not given.  It returns the
// results, or the library's status as an int where that is not 0.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "zipccl.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

template <class... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw python_error();
}

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: expected a tensor", what);
  return THPVariable_Unpack(o);
}

int value_type(const Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case ScalarType::Float: return ZIPCCL_TYPE_F32;
    case ScalarType::BFloat16: return ZIPCCL_TYPE_BF16;
    case ScalarType::Half: return ZIPCCL_TYPE_F16;
    default: refuse(PyExc_TypeError, "%s: expected float32, bfloat16 or float16, got %s", what, toString(t.scalar_type()));
  }
}

// The device of a call's tensors: that of the first of them.
c10::Device cuda_device(const Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s: expected a CUDA tensor", what);
  return t.device();
}

// A contiguous tensor of this type and shape on this device: the kernels read
// every operand of a call through plain pointers.
const Tensor& plain(const Tensor& t, ScalarType type, IntArrayRef shape, c10::Device device, const char* what) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s: expected %s, got %s", what, toString(type), toString(t.scalar_type()));
  if (t.sizes() != shape) refuse(PyExc_ValueError, "%s: a tensor of another shape was expected", what);
  if (!t.is_cuda() || !t.is_contiguous()) refuse(PyExc_ValueError, "%s: expected a contiguous CUDA tensor", what);
  if (t.device() != device) refuse(PyExc_ValueError, "%s: expected a tensor on the device of the call's others", what);
  return t;
}

const void* optional(PyObject* o, ScalarType type, IntArrayRef shape, c10::Device device, const char* what) {
  return o == Py_None ? nullptr : plain(tensor(o, what), type, shape, device, what).const_data_ptr();
}

// A warning where autograd would expect to go through the call: results carry
// no gradient, so a training step would leave out what comes before in silence.
void no_autograd(const char* call, std::initializer_list<PyObject*> operands) {
  if (!at::GradMode::is_enabled()) return;
  for (PyObject* o : operands)
    if (THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad()) {
      if (PyErr_WarnFormat(PyExc_UserWarning, 2, "%s: an operand requires a gradient, and the results carry none: the package's "
                           "_backward calls compute it (call under torch.no_grad() or with detached tensors)", call) < 0)
        throw python_error();
      return;
    }
}

void two_dims(const Tensor& t, const char* what) {
  if (t.dim() != 2) refuse(PyExc_ValueError, "%s: expected two dimensions", what);
}

// Values between the rows of a [tokens, values] CUDA tensor whose rows are contiguous.
uint64_t row_stride(const Tensor& t, const char* what) {
  two_dims(t, what);
  if (!t.is_cuda() || (t.stride(1) != 1 && t.size(1) > 1 && t.numel() > 0))
    refuse(PyExc_ValueError, "%s: expected a CUDA tensor with contiguous rows", what);
  return (uint64_t)(t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1)));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// A tensor that the call is about to write through a pointer: autograd, where it
// has saved it, then knows that it has changed.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A call's device, current until the call ends: the launches go to the current
// device, and stream 0 is that device's.  Its stream (None: the current one of
// that device) and the results it allocates.  They come from the memory of the
// stream that writes them: what the current stream has freed it may still be
// reading.  A result is the current stream's to read, so its memory goes back
// only after what that stream has queued when it is freed.
struct Call {
  c10::Device device;
  c10::cuda::OptionalCUDAGuard current_device;  // left alone where the device is current already
  cudaStream_t stream;
  bool other = false;
  Call(c10::Device d, PyObject* s) : device(d) {
    if (c10::cuda::device_count() > 1 && c10::cuda::current_device() != d.index()) current_device.set_device(d);
    const cudaStream_t current = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    stream = current;
    if (s != Py_None) {
      stream = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(s));
      if (PyErr_Occurred()) throw python_error();
      other = stream != current;
    }
  }
  Tensor scratch(IntArrayRef shape, ScalarType type) const {
    if (!other) return at::detail::empty_cuda(shape, type, device, std::nullopt);
    const c10::cuda::CUDAStreamGuard its(c10::cuda::getStreamFromExternal(stream, device.index()));
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }
  Tensor empty(IntArrayRef shape, ScalarType type) const {
    Tensor t = scratch(shape, type);
    if (other)
      c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), c10::cuda::getCurrentCUDAStream(device.index()));
    return t;
  }
  Tensor result(PyObject* o, IntArrayRef shape, ScalarType type, const char* what) const {
    if (o == Py_None) return empty(shape, type);
    const Tensor& t = plain(tensor(o, what), type, shape, device, what);
    written(t);
    return t;
  }
};

// Pairs of a token that no call takes: refused before results of their size are
// allocated or the count is cut to 32 bits.
bool bad_top_k(int64_t k) { return k < 1 || k > 32; }
PyObject* refused() { return PyLong_FromLong(ZIPCCL_ERR_INVALID_ARG); }

PyObject* answer(zipccl_status st, std::initializer_list<Tensor> out) {
  if (st != ZIPCCL_OK) return PyLong_FromLong(st);
  if (out.size() == 1) return THPVariable_Wrap(*out.begin());
  PyObject* all = PyTuple_New((Py_ssize_t)out.size());
  if (!all) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : out) PyTuple_SET_ITEM(all, i++, THPVariable_Wrap(t));
  return all;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
}

// top_k, score, renormalize, scale, groups, groups_kept, group_score
zipccl_route_options route_options(PyObject* const* a) {
  zipccl_route_options o;
  const int64_t k = integer(a[0]), groups = integer(a[4]), kept = integer(a[5]);
  if (k < 1 || groups < 1 || kept < 1) refuse(PyExc_ValueError, "top_k, groups and groups_kept are at least 1");
  o.top_k = (uint32_t)std::min<int64_t>(k, UINT32_MAX);
  o.score = (int32_t)integer(a[1]);
  o.renormalize = (int32_t)integer(a[2]);
  o.scale = (float)real(a[3]);
  o.groups = (uint32_t)std::min<int64_t>(groups, UINT32_MAX);
  o.groups_kept = (uint32_t)std::min<int64_t>(kept, UINT32_MAX);
  o.group_score = (int32_t)integer(a[6]);
  return o;
}

// logits, <route options>, bias, mask, weights, ids, stream
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  no_autograd("moe_route", {a[0]});
  const zipccl_route_options o = route_options(a + 1);
  const Tensor& logits = tensor(a[0], "logits");
  const int type = value_type(logits, "logits");
  const uint64_t stride = row_stride(logits, "logits");
  const int64_t tokens = logits.size(0), experts = logits.size(1), k = o.top_k;
  if (bad_top_k(k)) return refused();
  const c10::Device device = logits.device();
  const void* bias = optional(a[8], ScalarType::Float, {experts}, device, "bias");
  const void* mask = nullptr;
  if (a[9] != Py_None) {
    const Tensor& m = tensor(a[9], "mask");
    mask = plain(m, m.scalar_type() == ScalarType::Byte ? ScalarType::Byte : ScalarType::Bool, {tokens}, device, "mask").const_data_ptr();
  }
  const Call call(device, a[12]);
  const Tensor weights = call.result(a[10], {tokens, k}, ScalarType::Float, "weights");
  const Tensor ids = call.result(a[11], {tokens, k}, ScalarType::Int, "ids");
  return answer(zipccl_moe_route(logits.const_data_ptr(), type, stride, tokens, experts, &o, static_cast<const float*>(bias),
                                 static_cast<const uint8_t*>(mask), static_cast<float*>(weights.data_ptr()),
                                 static_cast<int32_t*>(ids.data_ptr()), call.stream),
                {weights, ids});
  END_HANDLE_TH_ERRORS
}

// grad_weights, logits, ids, score, renormalize, scale, grad_logits, stream
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  no_autograd("moe_route_backward", {a[0], a[1]});
  const Tensor& logits = tensor(a[1], "logits");
  const int type = value_type(logits, "logits");
  const uint64_t stride = row_stride(logits, "logits");
  const Tensor& ids = tensor(a[2], "ids");
  two_dims(ids, "ids");
  const int64_t tokens = logits.size(0), experts = logits.size(1), k = ids.size(1);
  if (bad_top_k(k)) return refused();
  const c10::Device device = logits.device();
  plain(ids, ScalarType::Int, {tokens, k}, device, "ids");
  const Tensor& grad = plain(tensor(a[0], "grad_weights"), ScalarType::Float, {tokens, k}, device, "grad_weights");
  zipccl_route_options o{};
  o.top_k = (uint32_t)k;
  o.score = (int32_t)integer(a[3]);
  o.renormalize = (int32_t)integer(a[4]);
  o.scale = (float)real(a[5]);
  o.groups = o.groups_kept = 1;
  const Call call(device, a[7]);
  const Tensor out = call.result(a[6], {tokens, experts}, logits.scalar_type(), "grad_logits");
  return answer(zipccl_moe_route_backward(static_cast<const float*>(grad.const_data_ptr()), logits.const_data_ptr(), type,
                                          stride, tokens, experts, &o, static_cast<const int32_t*>(ids.const_data_ptr()),
                                          out.data_ptr(), call.stream),
                {out});
  END_HANDLE_TH_ERRORS
}

// ids, n_experts, counts, offsets, slots, ws, stream
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const Tensor& ids = tensor(a[0], "ids");
  const int64_t experts = integer(a[1]);
  plain(ids, ScalarType::Int, ids.sizes(), ids.device(), "ids");
  uint64_t need = 0;
  if (experts < 1 || experts > UINT32_MAX) refuse(PyExc_ValueError, "n_experts is at least 1");
  const zipccl_status st = zipccl_moe_plan_workspace_bytes(ids.numel(), (uint32_t)experts, &need);
  if (st != ZIPCCL_OK) return PyLong_FromLong(st);
  const Call call(ids.device(), a[6]);
  const Tensor counts = call.result(a[2], {experts}, ScalarType::Int, "counts");
  const Tensor offsets = call.result(a[3], {experts + 1}, ScalarType::Int, "offsets");
  const Tensor slots = call.result(a[4], ids.sizes(), ScalarType::Int, "slots");
  Tensor ws;
  if (need) {
    if (a[5] != Py_None) ws = tensor(a[5], "ws");
    if (!ws.defined() || ws.nbytes() < need) ws = call.scratch({(int64_t)need}, ScalarType::Byte);
    plain(ws, ws.scalar_type(), ws.sizes(), call.device, "ws");
  }
  return answer(zipccl_moe_plan(static_cast<const int32_t*>(ids.const_data_ptr()), ids.numel(), (uint32_t)experts,
                                static_cast<int32_t*>(counts.data_ptr()), static_cast<int32_t*>(offsets.data_ptr()),
                                static_cast<int32_t*>(slots.data_ptr()), need ? ws.data_ptr() : nullptr,
                                need ? ws.nbytes() : 0, call.stream),
                {counts, offsets, slots});
  END_HANDLE_TH_ERRORS
}

const int32_t* pair_slots(const Tensor& slots, int64_t tokens, c10::Device device) {
  return static_cast<const int32_t*>(plain(slots, ScalarType::Int, {tokens, slots.size(1)}, device, "slots").const_data_ptr());
}

// x, slots, out, stream
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  no_autograd("moe_dispatch", {a[0]});
  const Tensor &x = tensor(a[0], "x"), &slots = tensor(a[1], "slots");
  const int type = value_type(x, "x");
  const uint64_t stride = row_stride(x, "x");
  const int64_t tokens = x.size(0), hidden = x.size(1);
  two_dims(slots, "slots");
  if (bad_top_k(slots.size(1))) return refused();
  const int32_t* at = pair_slots(slots, tokens, x.device());
  const Call call(x.device(), a[3]);
  const Tensor out = call.result(a[2], {tokens * slots.size(1), hidden}, x.scalar_type(), "out");
  return answer(zipccl_moe_dispatch(x.const_data_ptr(), type, stride, tokens, (uint32_t)slots.size(1), hidden, at,
                                    out.data_ptr(), call.stream),
                {out});
  END_HANDLE_TH_ERRORS
}

// What the calls on the experts' rows share.
struct Pairs {
  const Tensor &rows, &slots;
  int type;
  const int32_t* at;
  int64_t tokens, k, hidden;
  Pairs(PyObject* r, PyObject* s, const char* what) : rows(tensor(r, what)), slots(tensor(s, "slots")) {
    type = value_type(rows, what);
    two_dims(slots, "slots");
    tokens = slots.size(0);
    k = slots.size(1);
    at = pair_slots(slots, tokens, cuda_device(rows, what));
    two_dims(rows, what);
    hidden = rows.size(1);
    plain(rows, rows.scalar_type(), {tokens * k, hidden}, rows.device(), what);
  }
};

// grad_rows, slots, out, stream
PyObject* dispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  no_autograd("moe_dispatch_backward", {a[0]});
  const Pairs p(a[0], a[1], "grad_rows");
  if (bad_top_k(p.k)) return refused();
  const Call call(p.rows.device(), a[3]);
  const Tensor out = call.result(a[2], {p.tokens, p.hidden}, p.rows.scalar_type(), "out");
  return answer(zipccl_moe_dispatch_backward(p.rows.const_data_ptr(), p.type, p.tokens, (uint32_t)p.k, p.hidden, p.at,
                                             out.data_ptr(), call.stream),
                {out});
  END_HANDLE_TH_ERRORS
}

// rows, slots, weights, residual, out, stream
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  no_autograd("moe_combine", {a[0], a[2], a[3]});
  const Pairs p(a[0], a[1], "rows");
  if (bad_top_k(p.k)) return refused();
  const c10::Device device = p.rows.device();
  const void* weights = optional(a[2], ScalarType::Float, {p.tokens, p.k}, device, "weights");
  const void* residual = optional(a[3], p.rows.scalar_type(), {p.tokens, p.hidden}, device, "residual");
  const Call call(device, a[5]);
  const Tensor out = call.result(a[4], {p.tokens, p.hidden}, p.rows.scalar_type(), "out");
  return answer(zipccl_moe_combine(p.rows.const_data_ptr(), p.type, p.tokens, (uint32_t)p.k, p.hidden, p.at,
                                   static_cast<const float*>(weights), residual, out.data_ptr(), call.stream),
                {out});
  END_HANDLE_TH_ERRORS
}

// grad_out, rows, slots, weights, grad_rows, grad_weights, stream
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  no_autograd("moe_combine_backward", {a[0], a[1], a[3]});
  const Pairs p(a[1], a[2], "rows");
  if (bad_top_k(p.k)) return refused();
  const ScalarType type = p.rows.scalar_type();
  const c10::Device device = p.rows.device();
  const Tensor& grad = plain(tensor(a[0], "grad_out"), type, {p.tokens, p.hidden}, device, "grad_out");
  const void* weights = optional(a[3], ScalarType::Float, {p.tokens, p.k}, device, "weights");
  const Call call(device, a[6]);
  const Tensor grad_rows = call.result(a[4], p.rows.sizes(), type, "grad_rows");
  const Tensor grad_weights = call.result(a[5], {p.tokens, p.k}, ScalarType::Float, "grad_weights");
  return answer(zipccl_moe_combine_backward(grad.const_data_ptr(), p.rows.const_data_ptr(), p.type, p.tokens, (uint32_t)p.k,
                                            p.hidden, p.at, static_cast<const float*>(weights), grad_rows.data_ptr(),
                                            static_cast<float*>(grad_weights.data_ptr()), call.stream),
                {grad_rows, grad_weights});
  END_HANDLE_TH_ERRORS
}

// A list of tensors, read once (it may be an iterator) and held with its
// tensors until it goes; None: an empty one.
struct Sequence {
  PyObject* o;
  Py_ssize_t n;
  explicit Sequence(PyObject* s) : o(s == Py_None ? PyTuple_New(0) : PySequence_Fast(s, "expected a sequence of tensors")) {
    if (!o) throw python_error();
    n = PySequence_Fast_GET_SIZE(o);
  }
  Sequence(const Sequence&) = delete;
  ~Sequence() { Py_DECREF(o); }
  const Tensor& at(Py_ssize_t i, const char* what) const { return tensor(PySequence_Fast_GET_ITEM(o, i), what); }
};

// The addresses of one list of tensors, into one field of the records.
void column(const Sequence& s, std::vector<zipccl_adamw_tensor>& records, bool scales, ScalarType type, c10::Device device,
            bool writes, const char* what, void (*set)(zipccl_adamw_tensor&, void*)) {
  if (s.n != (Py_ssize_t)records.size())
    refuse(PyExc_ValueError, "%s: expected %zd tensors, got %zd", what, (Py_ssize_t)records.size(), s.n);
  for (Py_ssize_t i = 0; i < s.n; ++i) {
    const Tensor& t = s.at(i, what);
    const uint64_t want = scales ? (records[i].n + ZIPCCL_ADAMW_BLOCK - 1) / ZIPCCL_ADAMW_BLOCK : records[i].n;
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s: expected %s, got %s", what, toString(type), toString(t.scalar_type()));
    if (t.device() != device || !t.is_contiguous())
      refuse(PyExc_ValueError, "%s: expected contiguous tensors on the device of the first parameter", what);
    if ((uint64_t)t.numel() != want) refuse(PyExc_ValueError, "%s: a tensor of another size was expected", what);
    set(records[i], t.data_ptr());
    if (writes) written(t);
  }
}

// params, grads, exp_avgs, exp_avg_sqs, avg_scales, sq_scales, copies, grad_scale,
// lr, beta1, beta2, eps, weight_decay, step, stream
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const Sequence p(a[0]), g(a[1]), m(a[2]), v(a[3]), ms(a[4]), vs(a[5]), copies(a[6]);
  if (p.n == 0) Py_RETURN_NONE;
  if (g.n != p.n) refuse(PyExc_ValueError, "grads: expected %zd tensors, got %zd", p.n, g.n);
  const Tensor &p0 = p.at(0, "params"), &g0 = g.at(0, "grads");
  const ScalarType ptype = p0.scalar_type(), gtype = g0.scalar_type();
  for (ScalarType t : {ptype, gtype})
    if (t != ScalarType::Float && t != ScalarType::BFloat16)
      refuse(PyExc_TypeError, "params and grads: expected float32 or bfloat16, got %s", toString(t));
  const c10::Device device = cuda_device(p0, "params");
  std::vector<zipccl_adamw_tensor> records(p.n);
  for (Py_ssize_t i = 0; i < p.n; ++i) records[i].n = (uint64_t)p.at(i, "params").numel();
  const bool small = a[4] != Py_None;
  const ScalarType state = small ? ScalarType::Float8_e4m3fn : ScalarType::Float;
  column(p, records, false, ptype, device, true, "params", [](zipccl_adamw_tensor& r, void* at) { r.d_param = at; });
  column(g, records, false, gtype, device, false, "grads", [](zipccl_adamw_tensor& r, void* at) { r.d_grad = at; });
  column(m, records, false, state, device, true, "exp_avgs", [](zipccl_adamw_tensor& r, void* at) { r.d_exp_avg = at; });
  column(v, records, false, state, device, true, "exp_avg_sqs", [](zipccl_adamw_tensor& r, void* at) { r.d_exp_avg_sq = at; });
  if (small) {
    column(ms, records, true, ScalarType::Float, device, true, "scales", [](zipccl_adamw_tensor& r, void* at) { r.d_avg_scale = (float*)at; });
    column(vs, records, true, ScalarType::Float, device, true, "scales", [](zipccl_adamw_tensor& r, void* at) { r.d_sq_scale = (float*)at; });
  }
  if (a[6] != Py_None)
    column(copies, records, false, ScalarType::BFloat16, device, true, "copies", [](zipccl_adamw_tensor& r, void* at) { r.d_copy = at; });
  const float* scale = nullptr;
  if (a[7] != Py_None) {
    const Tensor& t = tensor(a[7], "grad_scale");
    if (t.numel() != 1) refuse(PyExc_ValueError, "grad_scale: expected one value");
    scale = static_cast<const float*>(plain(t, ScalarType::Float, t.sizes(), device, "grad_scale").const_data_ptr());
  }
  const int64_t step = integer(a[13]);
  const zipccl_adamw_options o = {real(a[8]), real(a[9]), real(a[10]), real(a[11]), real(a[12]), (uint64_t)std::max<int64_t>(step, 0)};
  const Call call(device, a[14]);
  const zipccl_status st =
      zipccl_adamw_step(records.data(), (uint32_t)records.size(), ptype == ScalarType::Float ? ZIPCCL_TYPE_F32 : ZIPCCL_TYPE_BF16,
                        gtype == ScalarType::Float ? ZIPCCL_TYPE_F32 : ZIPCCL_TYPE_BF16, small ? 8 : 32, &o, scale, call.stream);
  if (st != ZIPCCL_OK) return PyLong_FromLong(st);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// ---- 8-bit blocks: a pair (codes, scales)
uint8_t* bytes(const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

struct Blocks {
  Tensor codes, scales;
};

// (codes, scales) of an argument.
Blocks blocks(PyObject* o, const char* what) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) refuse(PyExc_TypeError, "%s: expected Fp8Blocks (codes, scales)", what);
  Blocks b{tensor(PyTuple_GET_ITEM(o, 0), what), tensor(PyTuple_GET_ITEM(o, 1), what)};
  if (b.codes.scalar_type() != ScalarType::Float8_e4m3fn)
    refuse(PyExc_TypeError, "%s: expected codes of Float8_e4m3fn, got %s", what, toString(b.codes.scalar_type()));
  if (b.scales.scalar_type() != ScalarType::Float8_e8m0fnu)
    refuse(PyExc_TypeError, "%s: expected scales of Float8_e8m0fnu, got %s", what, toString(b.scales.scalar_type()));
  return b;
}

// Bytes between rows of codes [.., rows, cols], whose matrices lie rows apart.
uint64_t code_stride(const Tensor& t, const char* what) {
  const int64_t d = t.dim(), rows = t.size(d - 2), cols = t.size(d - 1);
  if (t.numel() == 0) return (uint64_t)((cols + 15) / 16 * 16);
  const bool apart = rows > 1 || (d == 3 && t.size(0) > 1);
  const int64_t stride = rows > 1 ? t.stride(d - 2) : d == 3 && t.size(0) > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
  if (!t.is_cuda() || (cols > 1 && t.stride(d - 1) != 1) || (apart && (stride % 16 || stride < cols)) ||
      (d == 3 && t.size(0) > 1 && t.stride(0) != stride * rows))
    refuse(PyExc_ValueError, "%s: expected CUDA codes whose rows are contiguous and a multiple of 16 bytes apart", what);
  return (uint64_t)stride;
}

int64_t block_count(int64_t n) { return (n + ZIPCCL_FP8_BLOCK - 1) / ZIPCCL_FP8_BLOCK; }

// Blocks that a call fills: given, or allocated with rows of a multiple of 16 bytes.
Blocks new_blocks(const Call& call, PyObject* o, IntArrayRef shape, IntArrayRef scale_shape, const char* what) {
  if (o != Py_None) {
    Blocks b = blocks(o, what);
    if (b.codes.sizes() != shape) refuse(PyExc_ValueError, "%s: codes of another shape were expected", what);
    if (b.codes.device() != call.device) refuse(PyExc_ValueError, "%s: expected tensors on the device of the call's others", what);
    plain(b.scales, ScalarType::Float8_e8m0fnu, scale_shape, call.device, what);
    code_stride(b.codes, what);
    written(b.codes);
    written(b.scales);
    return b;
  }
  std::vector<int64_t> held(shape.begin(), shape.end());
  const int64_t cols = held.back();
  held.back() = (cols + 15) / 16 * 16;
  Tensor codes = call.empty(held, ScalarType::Float8_e4m3fn);
  if (held.back() != cols) codes = codes.slice(-1, 0, cols);
  return {codes, call.empty(scale_shape, ScalarType::Float8_e8m0fnu)};
}

PyObject* pair(const Blocks& b) {
  PyObject* both = PyTuple_New(2);
  if (!both) throw python_error();
  PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(b.codes));
  PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(b.scales));
  return both;
}

// Offsets of the chunks (None: one chunk) and how many chunks there are.
const int32_t* chunk_offsets(PyObject* o, c10::Device device, int64_t* experts) {
  *experts = 1;
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "offsets");
  if (t.dim() != 1 || t.numel() < 2) refuse(PyExc_ValueError, "offsets: expected one dimension, one value more than there are experts");
  *experts = t.numel() - 1;
  return static_cast<const int32_t*>(plain(t, ScalarType::Int, t.sizes(), device, "offsets").const_data_ptr());
}

bool bad_chunks(int64_t experts) { return experts > 1024; }
bool bad_widths(int64_t a, int64_t b = 1) { return a > 1 << 22 || b > 1 << 22; }

// rows, out, stream
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 3);
  no_autograd("moe_quantize", {a[0]});
  const Tensor& x = tensor(a[0], "rows");
  const int type = value_type(x, "rows");
  const uint64_t stride = row_stride(x, "rows");
  const int64_t rows = x.size(0), cols = x.size(1);
  if (bad_widths(cols)) return refused();
  const Call call(x.device(), a[2]);
  const Blocks b = new_blocks(call, a[1], {rows, cols}, {rows, block_count(cols)}, "out");
  const zipccl_status st = zipccl_moe_quantize(x.const_data_ptr(), type, stride, rows, cols, bytes(b.codes), code_stride(b.codes, "out"),
                                               bytes(b.scales), call.stream);
  return st == ZIPCCL_OK ? pair(b) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// rows, offsets, by_rows, out, rows_out, stream
PyObject* quantize_columns(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  no_autograd("moe_quantize_columns", {a[0]});
  const Tensor& x = tensor(a[0], "rows");
  const int type = value_type(x, "rows");
  const uint64_t stride = row_stride(x, "rows");
  const int64_t rows = x.size(0), cols = x.size(1);
  int64_t experts;
  const int32_t* offsets = chunk_offsets(a[1], x.device(), &experts);
  if (bad_widths(cols) || bad_chunks(experts)) return refused();
  const int asked = PyObject_IsTrue(a[2]);
  if (asked < 0) throw python_error();
  const bool both = asked == 1;
  if (!both && a[4] != Py_None) refuse(PyExc_ValueError, "rows_out is given and by_rows is not");
  const Call call(x.device(), a[5]);
  const Blocks b = new_blocks(call, a[3], {rows, cols}, {rows / (int64_t)ZIPCCL_FP8_BLOCK + experts, cols}, "out");
  Blocks r;
  if (both) r = new_blocks(call, a[4], {rows, cols}, {rows, block_count(cols)}, "rows_out");
  const zipccl_status st = zipccl_moe_quantize_columns(
      x.const_data_ptr(), type, stride, rows, cols, offsets, (uint32_t)experts, bytes(b.codes), code_stride(b.codes, "out"),
      bytes(b.scales), both ? bytes(r.codes) : nullptr, both ? code_stride(r.codes, "rows_out") : 0, both ? bytes(r.scales) : nullptr,
      call.stream);
  if (st != ZIPCCL_OK) return PyLong_FromLong(st);
  if (!both) return pair(b);
  PyObject* out = PyTuple_New(2);
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out, 0, pair(r));
  PyTuple_SET_ITEM(out, 1, pair(b));
  return out;
  END_HANDLE_TH_ERRORS
}

// weights, out, stream
PyObject* quantize_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 3);
  no_autograd("moe_quantize_weights", {a[0]});
  const Tensor& w = tensor(a[0], "weights");
  const int type = value_type(w, "weights");
  if (w.dim() != 2 && w.dim() != 3) refuse(PyExc_ValueError, "weights: expected two or three dimensions");
  plain(w, w.scalar_type(), w.sizes(), cuda_device(w, "weights"), "weights");
  const int64_t experts = w.dim() == 3 ? w.size(0) : 1, rows = w.size(-2), cols = w.size(-1);
  if (bad_widths(rows, cols) || bad_chunks(experts)) return refused();
  const Call call(w.device(), a[2]);
  std::vector<int64_t> scales = {block_count(rows), block_count(cols)};
  if (w.dim() == 3) scales.insert(scales.begin(), experts);
  const Blocks b = new_blocks(call, a[1], w.sizes(), scales, "out");
  const zipccl_status st = zipccl_moe_quantize_weights(w.const_data_ptr(), type, (uint32_t)experts, rows, cols, bytes(b.codes),
                                                       code_stride(b.codes, "out"), bytes(b.scales), call.stream);
  return st == ZIPCCL_OK ? pair(b) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// form, a, b, offsets, type, out, stream
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const int form = (int)integer(a[0]);
  const bool by_weights = form == ZIPCCL_MATMUL_WEIGHTS, forward = form == ZIPCCL_MATMUL_FORWARD;
  const char* names[2] = {forward ? "rows" : by_weights ? "grad_columns" : "grad_rows", by_weights ? "columns" : "weights"};
  const Blocks x = blocks(a[1], names[0]), w = blocks(a[2], names[1]);
  const c10::Device device = cuda_device(x.codes, names[0]);
  int64_t experts;
  const int32_t* offsets = chunk_offsets(a[3], device, &experts);
  two_dims(x.codes, names[0]);
  if (by_weights) two_dims(w.codes, names[1]);
  else if (w.codes.dim() != (offsets ? 3 : 2))
    refuse(PyExc_ValueError, "%s: expected %s dimensions", names[1], offsets ? "three" : "two");
  const int64_t rows = x.codes.size(0), inner = w.codes.size(-1), outer = by_weights ? x.codes.size(1) : w.codes.size(-2);
  if (!by_weights && offsets && w.codes.size(0) != experts) refuse(PyExc_ValueError, "%s: a matrix for each chunk was expected", names[1]);
  if (by_weights ? w.codes.size(0) != rows : x.codes.size(1) != (forward ? inner : outer))
    refuse(PyExc_ValueError, "%s and %s: sizes that fit each other were expected", names[0], names[1]);
  if (bad_widths(inner, outer) || bad_chunks(experts)) return refused();
  if (w.codes.device() != device) refuse(PyExc_ValueError, "%s: expected a tensor on the device of the call's others", names[1]);
  constexpr ScalarType scale = ScalarType::Float8_e8m0fnu;
  if (by_weights) {
    const int64_t blocks = rows / (int64_t)ZIPCCL_FP8_BLOCK + experts;
    plain(x.scales, scale, {blocks, outer}, device, names[0]);
    plain(w.scales, scale, {blocks, inner}, device, names[1]);
  } else {
    plain(x.scales, scale, {rows, block_count(x.codes.size(1))}, device, names[0]);
    if (offsets) plain(w.scales, scale, {experts, block_count(outer), block_count(inner)}, device, names[1]);
    else plain(w.scales, scale, {block_count(outer), block_count(inner)}, device, names[1]);
  }
  const int type = (int)integer(a[4]);
  const ScalarType to = type == ZIPCCL_TYPE_F32 ? ScalarType::Float : type == ZIPCCL_TYPE_BF16 ? ScalarType::BFloat16 : ScalarType::Half;
  const zipccl_fp8_blocks xa = {bytes(x.codes), bytes(x.scales), code_stride(x.codes, names[0])};
  const zipccl_fp8_blocks wb = {bytes(w.codes), bytes(w.scales), code_stride(w.codes, names[1])};
  const Call call(device, a[6]);
  std::vector<int64_t> shape = by_weights ? std::vector<int64_t>{outer, inner} : std::vector<int64_t>{rows, forward ? outer : inner};
  if (by_weights && offsets) shape.insert(shape.begin(), experts);
  Tensor out = call.result(a[5], shape, to, "out");
  if (inner == 0 || outer == 0) {  // sums of nothing
    const c10::cuda::CUDAStreamGuard its(c10::cuda::getStreamFromExternal(call.stream, device.index()));
    if (out.numel()) out.zero_();
    return answer(ZIPCCL_OK, {out});
  }
  return answer(zipccl_moe_matmul(form, &xa, &wb, rows, inner, outer, offsets, (uint32_t)experts, out.data_ptr(), type, shape.back(),
                                  call.stream),
                {out});
  END_HANDLE_TH_ERRORS
}

// A matrix of weights for each expert: plain, or 8-bit blocks.
struct Matrices {
  const void* at;
  const uint8_t* scales = nullptr;
  uint64_t stride;
  IntArrayRef shape;
  bool small;
  Tensor held, held_scales;
  Matrices(PyObject* o, ScalarType type, c10::Device device, const char* what) {
    small = PyTuple_Check(o);
    if (small) {
      const Blocks b = blocks(o, what);
      if (b.codes.dim() != 3) refuse(PyExc_ValueError, "%s: expected three dimensions", what);
      if (!b.codes.is_cuda() || b.codes.device() != device) refuse(PyExc_ValueError, "%s: expected a tensor on the device of the call's others", what);
      plain(b.scales, ScalarType::Float8_e8m0fnu, {b.codes.size(0), block_count(b.codes.size(1)), block_count(b.codes.size(2))}, device, what);
      held = b.codes;
      held_scales = b.scales;
      stride = code_stride(held, what);
      scales = bytes(held_scales);
    } else {
      held = tensor(o, what);
      plain(held, type, held.sizes(), device, what);
      if (held.dim() != 3) refuse(PyExc_ValueError, "%s: expected three dimensions", what);
      stride = (uint64_t)held.size(2);
    }
    at = held.const_data_ptr();
    shape = held.sizes();
  }
};

// x, router, up, down, <route options>, bias, mask, activation, residual, out, weights, ids, ws, stream
PyObject* layer(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 20);
  no_autograd("moe_layer", {a[0], a[1], a[2], a[3], a[14]});
  const zipccl_route_options o = route_options(a + 4);
  const Tensor &x = tensor(a[0], "x"), &router = tensor(a[1], "router");
  zipccl_moe_layer_args l{};
  l.type = value_type(x, "x");
  l.router_type = value_type(router, "router");
  l.x_stride = row_stride(x, "x");
  const int64_t tokens = x.size(0), hidden = x.size(1), k = o.top_k;
  if (bad_top_k(k)) return refused();
  const c10::Device device = x.device();
  two_dims(router, "router");
  const int64_t experts = router.size(0);
  plain(router, router.scalar_type(), {experts, hidden}, device, "router");
  if (router.scalar_type() != x.scalar_type() && router.scalar_type() != ScalarType::Float)
    refuse(PyExc_TypeError, "router: expected the type of x or float32");
  const Matrices up(a[2], x.scalar_type(), device, "up"), down(a[3], x.scalar_type(), device, "down");
  if (up.small != down.small) refuse(PyExc_TypeError, "up and down: expected both in 8-bit blocks or neither");
  const int64_t inner = down.shape[2], rows = up.shape[1];
  if (up.shape[0] != experts || down.shape[0] != experts || up.shape[2] != hidden || down.shape[1] != hidden ||
      (rows != inner && rows != 2 * inner))
    refuse(PyExc_ValueError, "up and down: expected [experts, inner or 2 inner, hidden] and [experts, hidden, inner]");
  l.gated = rows != inner;
  l.weight_bits = up.small ? 8 : 8 * (int)x.element_size();
  l.d_bias = static_cast<const float*>(optional(a[11], ScalarType::Float, {experts}, device, "bias"));
  if (a[12] != Py_None) {
    const Tensor& m = tensor(a[12], "mask");
    l.d_mask = static_cast<const uint8_t*>(plain(m, m.scalar_type() == ScalarType::Byte ? ScalarType::Byte : ScalarType::Bool, {tokens}, device, "mask").const_data_ptr());
  }
  l.activation = (int32_t)integer(a[13]);
  l.d_residual = optional(a[14], x.scalar_type(), {tokens, hidden}, device, "residual");
  uint64_t need = 0;
  const zipccl_status sized = zipccl_moe_layer_workspace_bytes((uint64_t)tokens, (uint32_t)k, (uint64_t)inner, &need);
  if (sized != ZIPCCL_OK) return PyLong_FromLong(sized);
  const Call call(device, a[19]);
  const Tensor y = call.result(a[15], {tokens, hidden}, x.scalar_type(), "out");
  const Tensor weights = call.result(a[16], {tokens, k}, ScalarType::Float, "weights");
  const Tensor ids = call.result(a[17], {tokens, k}, ScalarType::Int, "ids");
  Tensor ws;
  if (a[18] != Py_None) ws = tensor(a[18], "ws");
  if (!ws.defined() || ws.nbytes() < need) ws = call.scratch({(int64_t)need}, ScalarType::Byte);
  plain(ws, ws.scalar_type(), ws.sizes(), device, "ws");
  l.d_x = x.const_data_ptr();
  l.d_router = router.const_data_ptr();
  l.d_up = up.at;
  l.d_down = down.at;
  l.d_up_scales = up.scales;
  l.d_down_scales = down.scales;
  l.d_y = y.data_ptr();
  l.d_weights = static_cast<float*>(weights.data_ptr());
  l.d_ids = static_cast<int32_t*>(ids.data_ptr());
  l.tokens = (uint64_t)tokens;
  l.hidden = (uint64_t)hidden;
  l.inner = (uint64_t)inner;
  l.up_stride = up.stride;
  l.down_stride = down.stride;
  l.experts = (uint32_t)std::min<int64_t>(experts, UINT32_MAX);
  return answer(zipccl_moe_layer(&l, &o, ws.data_ptr(), ws.nbytes(), call.stream), {y, weights, ids});
  END_HANDLE_TH_ERRORS
}

#define ZC_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ZC_METHOD(route),             ZC_METHOD(route_backward), ZC_METHOD(plan),
                         ZC_METHOD(dispatch),          ZC_METHOD(dispatch_backward), ZC_METHOD(combine),
                         ZC_METHOD(combine_backward),  ZC_METHOD(adamw),          ZC_METHOD(quantize),
                         ZC_METHOD(quantize_columns),  ZC_METHOD(quantize_weights), ZC_METHOD(matmul),            ZC_METHOD(layer),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_zipccl_torch", "Operator calls of libzipccl on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__zipccl_torch() { return PyModule_Create(&module); }

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
  if (!t.is_cuda() || (t.stride(1) != 1 && t.size(1) > 1))
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

#define ZC_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ZC_METHOD(route),             ZC_METHOD(route_backward), ZC_METHOD(plan),
                         ZC_METHOD(dispatch),          ZC_METHOD(dispatch_backward), ZC_METHOD(combine),
                         ZC_METHOD(combine_backward),  ZC_METHOD(adamw),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_zipccl_torch", "Operator calls of libzipccl on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__zipccl_torch() { return PyModule_Create(&module); }

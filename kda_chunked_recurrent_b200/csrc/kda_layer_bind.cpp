// kda_layer_bind.cpp — the Python side of the layer operators (include/kda_layer.h): checks of
// the tensors, allocation of outputs, and the call of the C entry point.
//
// A token call's kernel takes a few microseconds; checking a dozen tensors from Python takes
// several times that, so it is done here.  The functions take positional arguments (layer.py
// has the signatures and their documentation).  What does not fit raises ValueError; a code
// other than KDA_OK goes to the Python function given to set_fail, which raises.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/torch.h>

#include <optional>
#include <utility>

#include "kda_layer.h"

namespace {

using at::Tensor;
using Shape = c10::SmallVector<int64_t, 4>;

PyObject* g_fail = nullptr;

// ---- arguments
const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, ": a tensor expected");
  return &THPVariable_Unpack(o);
}
const Tensor& need(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  TORCH_CHECK_VALUE(t != nullptr, name, ": a tensor expected, got None");
  return *t;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
int32_t int32(int64_t v, const char* name) {
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, ": ", v, " is out of range");
  return static_cast<int32_t>(v);
}

int dtype_code(const Tensor& x) {
  switch (x.scalar_type()) {
    case at::kBFloat16: return KDA_DTYPE_BF16;
    case at::kHalf: return KDA_DTYPE_F16;
    case at::kFloat: return KDA_DTYPE_F32;
    default:
      TORCH_CHECK_VALUE(false, "x: bfloat16, float16 or float32 expected, got ", x.scalar_type());
  }
  return -1;
}
// Asked last, when all else fits (so that the checks can be tested where there is no GPU), or
// where a tensor lies elsewhere than x.
void on_gpu(at::Device dev) {
  TORCH_CHECK_VALUE(dev.is_cuda(), "x: a CUDA tensor expected, got one on ", dev);
}
bool same_device(const Tensor& t, at::Device dev) {
  if (t.device() == dev) return true;
  on_gpu(dev);
  return false;
}

// A contiguous tensor of this type, shape and device: its address; NULL for none.
void* like(const Tensor* t, const char* name, at::ScalarType type, at::IntArrayRef shape,
           at::Device dev) {
  if (t == nullptr) return nullptr;
  TORCH_CHECK_VALUE(t->scalar_type() == type && t->sizes() == shape && t->is_contiguous() &&
                        same_device(*t, dev),
                    name, ": a contiguous ", type, " tensor of shape ", shape, " on ", dev,
                    " expected, got ", t->scalar_type(), " ", t->sizes(), " on ", t->device(),
                    ", strides ", t->strides());
  return t->data_ptr();
}
// n contiguous values of one of two types.
void* values(const Tensor* t, const char* name, at::ScalarType a, at::ScalarType b, int64_t n,
             at::Device dev) {
  if (t == nullptr) return nullptr;
  TORCH_CHECK_VALUE((t->scalar_type() == a || t->scalar_type() == b) && t->numel() == n &&
                        t->is_contiguous() && same_device(*t, dev),
                    name, ": ", n, " contiguous ", a, " values on ", dev, " expected, got ",
                    t->numel(), " of ", t->scalar_type(), " on ", t->device());
  return t->data_ptr();
}
// Elements between the rows of a tensor [..., row] whose last `tail` dimensions are a
// contiguous row and whose leading dimensions step through rows at one distance.
int64_t rows(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
             at::Device dev, int tail = 1) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && same_device(t, dev), name,
                    ": a ", type, " tensor of shape ", shape, " on ", dev, " expected, got ",
                    t.scalar_type(), " ", t.sizes(), " on ", t.device());
  const auto st = t.strides();
  const int dims = static_cast<int>(shape.size());
  int64_t n = 1;
  for (int i = dims - 1; i >= dims - tail; --i) {
    TORCH_CHECK_VALUE(shape[i] == 1 || st[i] == n, name,
                      ": the elements of a row must be adjacent, strides ", st);
    n *= shape[i];
  }
  int64_t row = -1, step = 1;
  for (int i = dims - tail - 1; i >= 0; --i) {
    if (shape[i] == 1) continue;
    if (row < 0) row = st[i];
    TORCH_CHECK_VALUE(st[i] == row * step, name, ": rows must lie at one distance, strides ", st);
    step *= shape[i];
  }
  if (row < 0 || t.numel() == 0) return n;
  TORCH_CHECK_VALUE(row >= n, name, ": rows must not overlap, strides ", st);
  return row;
}
// An output: the caller's, checked, or a new one, allocated when the call is made.
class Output {
 public:
  Output(PyObject* given, const char* name, at::ScalarType type, Shape shape, const Tensor& x)
      : type_(type), shape_(std::move(shape)) {
    const Tensor* t = tensor(given, name);
    if (t == nullptr) return;
    like(t, name, type, shape_, x.device());
    given_ = *t;
  }
  bool given() const { return given_.has_value(); }
  Tensor make(const Tensor& x) const {
    return given_ ? *given_ : at::empty(shape_, x.options().dtype(type_));
  }

 private:
  at::ScalarType type_;
  Shape shape_;
  std::optional<Tensor> given_;
};

struct Seqs {
  int64_t num;
  uint32_t flags = 0;
  void *cu = nullptr, *slots, *has, *status;
};
Seqs seqs(int64_t n_rows, PyObject* cu_o, PyObject* num_o, const Tensor* state, PyObject* slots_o,
          PyObject* has_o, PyObject* status_o, at::Device dev) {
  Seqs s;
  const Tensor* cu = tensor(cu_o, "cu_seqlens");
  const int64_t num = num_o == Py_None ? -1 : integer(num_o);
  if (cu != nullptr) {
    s.num = cu->numel() - 1;
    TORCH_CHECK_VALUE(s.num >= 1, "cu_seqlens: at least two offsets expected");
    s.cu = values(cu, "cu_seqlens", at::kInt, at::kLong, s.num + 1, dev);
    if (cu->scalar_type() == at::kLong) s.flags = KDA_LAYER_CU_SEQLENS_I64;
    TORCH_CHECK_VALUE(num_o == Py_None || num == s.num, "num_seqs does not agree with cu_seqlens");
  } else {
    s.num = num_o == Py_None ? 1 : num;
    TORCH_CHECK_VALUE(s.num >= 1 && n_rows % s.num == 0,
                      "without cu_seqlens the rows are num_seqs sequences of one length");
  }
  const Tensor *slots = tensor(slots_o, "state_indices"), *has = tensor(has_o, "has_state");
  TORCH_CHECK_VALUE(state != nullptr || (slots == nullptr && has == nullptr),
                    "state_indices and has_state need a state");
  s.slots = values(slots, "state_indices", at::kInt, at::kInt, s.num, dev);
  s.has = values(has, "has_state", at::kBool, at::kByte, s.num, dev);
  s.status = values(tensor(status_o, "device_status"), "device_status", at::kInt, at::kInt, 1, dev);
  return s;
}

// ---- the call: on the tensors' device, its current stream unless one is given.  Made behind the
// checks and before the outputs: they are then allocated on the stream that writes them, as under
// torch.cuda.stream(); memory of another stream may still be in use there.
class Call {
 public:
  Call(at::Device dev, PyObject* stream) : device_((on_gpu(dev), dev)) {
    if (stream == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
    if (stream_ == nullptr && PyErr_Occurred()) throw python_error();
    given_.reset_stream(c10::cuda::getStreamFromExternal(stream_, dev.index()));
  }
  template <typename F>
  void launch(const char* where, F&& call) const;

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard given_;
  cudaStream_t stream_;
};
template <typename F>
void Call::launch(const char* where, F&& call) const {
  // Other Python threads run meanwhile: a launch into a full queue waits until there is room.
  PyThreadState* const thread = PyEval_SaveThread();
  const kda_status_t rc = call(static_cast<void*>(stream_));
  PyEval_RestoreThread(thread);
  if (rc == KDA_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "is", static_cast<int>(rc), where);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw python_error();
}

template <typename T>
T* as(void* p) {
  return static_cast<T*>(p);
}
PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap_or_none(const std::optional<Tensor>& t) {
  if (t) return wrap(*t);
  Py_RETURN_NONE;
}
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = (a != nullptr && b != nullptr) ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

#define KDA_ARGS(n)                                                                   \
  if (nargs != (n)) {                                                                 \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");                    \
    return nullptr;                                                                   \
  }

// ---- short convolution
struct Conv {
  int64_t ch, width, parts, slots = 0;
  void *weight, *bias, *state;
  Shape out;
};
Conv conv_args(const Tensor& x, PyObject* weight_o, PyObject* bias_o, const Tensor* state,
               PyObject* parts_o) {
  Conv c;
  const at::Device dev = x.device();
  const Tensor& weight = need(weight_o, "weight");
  c.ch = x.size(-1);
  c.parts = integer(parts_o);
  TORCH_CHECK_VALUE(weight.dim() == 2, "weight: [channels, width] expected");
  c.width = weight.size(1);
  c.weight = like(&weight, "weight", at::kFloat, {c.ch, c.width}, dev);
  c.bias = like(tensor(bias_o, "bias"), "bias", at::kFloat, {c.ch}, dev);
  if (state != nullptr) {
    TORCH_CHECK_VALUE(state->dim() == 3 && state->size(0) >= 1,
                      "state: [slots, width - 1, channels] expected, with a slot at least");
    c.slots = state->size(0);
  }
  c.state = like(state, "state", x.scalar_type(), {c.slots, c.width - 1, c.ch}, dev);
  TORCH_CHECK_VALUE(c.parts >= 1 && c.ch % c.parts == 0, "parts must divide the channels");
  if (c.parts > 1) c.out.push_back(c.parts);
  for (int i = 0; i + 1 < x.dim(); ++i) c.out.push_back(x.size(i));
  c.out.push_back(c.ch / c.parts);
  return c;
}
kda_conv_shape_t conv_shape(const Conv& c, int64_t num, int64_t tokens, const Tensor& x) {
  kda_conv_shape_t s{};
  s.num_seqs = int32(num, "sequences");
  s.tokens = int32(tokens, "tokens");
  s.channels = int32(c.ch, "channels");
  s.width = int32(c.width, "width");
  s.parts = int32(c.parts, "parts");
  s.pool_size = int32(c.slots, "slots");
  s.dtype = dtype_code(x);
  s.x_stride = rows(x, "x", x.scalar_type(), x.sizes(), x.device());
  return s;
}

// x, weight, bias, state, state_indices, has_state, cu_seqlens, num_seqs, parts, silu, out,
// device_status, stream
PyObject* conv_prefill(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KDA_ARGS(13)
  const Tensor& x = need(a[0], "x");
  TORCH_CHECK_VALUE(x.dim() == 2, "x: [T, C] expected");
  const Tensor* state = tensor(a[3], "state");
  const Conv c = conv_args(x, a[1], a[2], state, a[8]);
  const Seqs s = seqs(x.size(0), a[6], a[7], state, a[4], a[5], a[11], x.device());
  const kda_conv_shape_t shape = conv_shape(c, s.num, x.size(0), x);
  const Output output(a[10], "out", x.scalar_type(), c.out, x);
  const Call call(x.device(), a[12]);
  const Tensor out = output.make(x);
  const uint32_t flags = s.flags | (truth(a[9]) ? KDA_CONV_SILU : 0u);
  call.launch("kda_conv_prefill", [&](void* stream) {
    return kda_conv_prefill(x.data_ptr(), as<float>(c.weight), as<float>(c.bias), c.state,
                            as<int32_t>(s.slots), as<uint8_t>(s.has), s.cu, &shape,
                            out.data_ptr(), as<int32_t>(s.status), flags, stream);
  });
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// x, weight, bias, state, state_indices, parts, silu, out, step_states, return_step_states,
// keep_state, device_status, stream
PyObject* conv_decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KDA_ARGS(13)
  const Tensor& x = need(a[0], "x");
  TORCH_CHECK_VALUE(x.dim() == 3, "x: [N, T, C] expected");
  const at::Device dev = x.device();
  const int64_t N = x.size(0), T = x.size(1);
  const Tensor& state = need(a[3], "state");
  const Conv c = conv_args(x, a[1], a[2], &state, a[5]);
  const kda_conv_shape_t shape = conv_shape(c, N, T, x);
  void* slots = values(tensor(a[4], "state_indices"), "state_indices", at::kInt, at::kInt, N, dev);
  void* status = values(tensor(a[11], "device_status"), "device_status", at::kInt, at::kInt, 1, dev);
  const Output output(a[7], "out", x.scalar_type(), c.out, x);
  const Output step_output(a[8], "step_states", x.scalar_type(), {N, T, c.width - 1, c.ch}, x);
  const Call call(dev, a[12]);
  const Tensor out = output.make(x);
  std::optional<Tensor> steps;
  if (step_output.given() || truth(a[9])) steps = step_output.make(x);
  const uint32_t flags =
      (truth(a[6]) ? KDA_CONV_SILU : 0u) | (truth(a[10]) ? KDA_LAYER_KEEP_STATE : 0u);
  call.launch("kda_conv_decode", [&](void* stream) {
    return kda_conv_decode(x.data_ptr(), as<float>(c.weight), as<float>(c.bias), c.state,
                           as<int32_t>(slots), &shape, out.data_ptr(),
                           steps ? steps->data_ptr() : nullptr, as<int32_t>(status), flags,
                           stream);
  });
  return pair(wrap(out), wrap_or_none(steps));
  END_HANDLE_TH_ERRORS
}

// ---- selective scan
struct Scan {
  kda_scan_shape_t shape{};
  void *x, *dt, *A_log, *B, *C, *D, *z, *bias, *state;
};
// a: x, dt, A_log, B, C, D, z, dt_bias, state
Scan scan_args(PyObject* const* a) {
  Scan s;
  const Tensor &x = need(a[0], "x"), &dt = need(a[1], "dt"), &A = need(a[2], "A_log"),
               &B = need(a[3], "B"), &C = need(a[4], "C");
  const Tensor *D = tensor(a[5], "D"), *z = tensor(a[6], "z"), *bias = tensor(a[7], "dt_bias"),
               *state = tensor(a[8], "state");
  const at::Device dev = x.device();
  const at::ScalarType type = x.scalar_type();
  const int64_t ch = x.size(-1);
  TORCH_CHECK_VALUE(A.dim() == 2 && B.dim() == x.dim() + 1,
                    "A_log: [D, N] and B, C: [..., G, N] expected");
  const int64_t size = A.size(1), groups = B.size(-2);
  Shape bc(x.sizes().begin(), x.sizes().end() - 1);
  bc.push_back(groups);
  bc.push_back(size);
  kda_scan_shape_t& sh = s.shape;
  sh.channels = int32(ch, "channels");
  sh.state_size = int32(size, "state size");
  sh.groups = int32(groups, "groups");
  sh.dtype = dtype_code(x);
  sh.x_stride = rows(x, "x", type, x.sizes(), dev);
  sh.dt_stride = rows(dt, "dt", type, x.sizes(), dev);
  sh.z_stride = z != nullptr ? rows(*z, "z", type, x.sizes(), dev) : 0;
  sh.b_stride = rows(B, "B", type, bc, dev, 2);
  sh.c_stride = rows(C, "C", type, bc, dev, 2);
  if (state != nullptr) {
    TORCH_CHECK_VALUE(state->dim() == 3 && state->size(0) >= 1,
                      "state: [slots, channels, state size] expected, with a slot at least");
    sh.pool_size = int32(state->size(0), "slots");
  }
  s.x = x.data_ptr();
  s.dt = dt.data_ptr();
  s.A_log = like(&A, "A_log", at::kFloat, {ch, size}, dev);
  s.B = B.data_ptr();
  s.C = C.data_ptr();
  s.D = like(D, "D", at::kFloat, {ch}, dev);
  s.z = z != nullptr ? z->data_ptr() : nullptr;
  s.bias = like(bias, "dt_bias", at::kFloat, {ch}, dev);
  s.state = like(state, "state", at::kFloat, {sh.pool_size, ch, size}, dev);
  return s;
}

// x, dt, A_log, B, C, D, z, dt_bias, state, state_indices, has_state, cu_seqlens, num_seqs,
// max_seqlen, softplus, out, device_status, stream
PyObject* scan_prefill(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KDA_ARGS(18)
  const Tensor& x = need(a[0], "x");
  TORCH_CHECK_VALUE(x.dim() == 2, "x: [T, D] expected");
  Scan c = scan_args(a);
  const Seqs s = seqs(x.size(0), a[11], a[12], tensor(a[8], "state"), a[9], a[10], a[16],
                      x.device());
  c.shape.num_seqs = int32(s.num, "sequences");
  c.shape.tokens = int32(x.size(0), "tokens");
  c.shape.max_seqlen = int32(integer(a[13]), "max_seqlen");
  const Output output(a[15], "out", x.scalar_type(), Shape(x.sizes()), x);
  const Call call(x.device(), a[17]);
  const Tensor out = output.make(x);
  const uint32_t flags = s.flags | (truth(a[14]) ? KDA_SCAN_SOFTPLUS : 0u);
  call.launch("kda_scan_prefill", [&](void* stream) {
    return kda_scan_prefill(c.x, c.dt, as<float>(c.A_log), c.B, c.C, as<float>(c.D), c.z,
                            as<float>(c.bias), as<float>(c.state), as<int32_t>(s.slots),
                            as<uint8_t>(s.has), s.cu, &c.shape, out.data_ptr(),
                            as<int32_t>(s.status), flags, stream);
  });
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// x, dt, A_log, B, C, D, z, dt_bias, state, state_indices, softplus, out, step_states,
// return_step_states, keep_state, device_status, stream
PyObject* scan_decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KDA_ARGS(17)
  const Tensor& x = need(a[0], "x");
  TORCH_CHECK_VALUE(x.dim() == 3, "x: [N, T, D] expected");
  need(a[8], "state");
  const at::Device dev = x.device();
  const int64_t N = x.size(0), T = x.size(1);
  Scan c = scan_args(a);
  c.shape.num_seqs = int32(N, "sequences");
  c.shape.tokens = int32(T, "tokens");
  void* slots = values(tensor(a[9], "state_indices"), "state_indices", at::kInt, at::kInt, N, dev);
  void* status = values(tensor(a[15], "device_status"), "device_status", at::kInt, at::kInt, 1, dev);
  const Output output(a[11], "out", x.scalar_type(), Shape(x.sizes()), x);
  const Output step_output(a[12], "step_states", at::kFloat,
                           {N, T, x.size(2), static_cast<int64_t>(c.shape.state_size)}, x);
  const Call call(dev, a[16]);
  const Tensor out = output.make(x);
  std::optional<Tensor> steps;
  if (step_output.given() || truth(a[13])) steps = step_output.make(x);
  const uint32_t flags =
      (truth(a[10]) ? KDA_SCAN_SOFTPLUS : 0u) | (truth(a[14]) ? KDA_LAYER_KEEP_STATE : 0u);
  call.launch("kda_scan_decode", [&](void* stream) {
    return kda_scan_decode(c.x, c.dt, as<float>(c.A_log), c.B, c.C, as<float>(c.D), c.z,
                           as<float>(c.bias), as<float>(c.state), as<int32_t>(slots), &c.shape,
                           out.data_ptr(), steps ? as<float>(steps->data_ptr()) : nullptr,
                           as<int32_t>(status), flags, stream);
  });
  return pair(wrap(out), wrap_or_none(steps));
  END_HANDLE_TH_ERRORS
}

// ---- norm
// x, weight, eps, residual, gate, flags, bits8, group, out, residual_out, scales, stream
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KDA_ARGS(12)
  const Tensor& x = need(a[0], "x");
  const int dims = static_cast<int>(x.dim()), tail = dims - 1;
  TORCH_CHECK_VALUE(dims == 2 || dims == 3, "x: [T, W] or [T, H, W] expected");
  const at::Device dev = x.device();
  const at::ScalarType type = x.scalar_type();
  const Tensor *res = tensor(a[3], "residual"), *gate = tensor(a[4], "gate"),
               *res_out_in = tensor(a[9], "residual_out"), *scales_in = tensor(a[10], "scales");
  const bool bits8 = truth(a[6]);
  const int64_t group = integer(a[7]), W = x.size(-1);
  TORCH_CHECK_VALUE(group == 0 || (group == 128 && bits8),
                    "group: 0, or 128 with an 8-bit output");
  TORCH_CHECK_VALUE(bits8 || scales_in == nullptr, "scales belong to an 8-bit output");
  TORCH_CHECK_VALUE(res != nullptr || res_out_in == nullptr, "residual_out needs a residual");
  kda_norm_shape_t sh{};
  sh.tokens = int32(x.size(0), "tokens");
  sh.heads = dims == 3 ? int32(x.size(1), "heads") : 1;
  sh.width = int32(W, "width");
  sh.group = static_cast<int32_t>(group);
  sh.dtype = dtype_code(x);
  sh.out_dtype = bits8 ? KDA_DTYPE_E4M3 : sh.dtype;
  sh.eps = static_cast<float>(PyFloat_AsDouble(a[2]));
  if (PyErr_Occurred()) throw python_error();
  sh.x_stride = rows(x, "x", type, x.sizes(), dev, tail);
  if (res != nullptr) sh.residual_stride = rows(*res, "residual", type, x.sizes(), dev, tail);
  if (gate != nullptr) sh.gate_stride = rows(*gate, "gate", type, x.sizes(), dev, tail);
  void* weight = like(tensor(a[1], "weight"), "weight", at::kFloat, {W}, dev);
  const Output output(a[8], "out", bits8 ? at::kFloat8_e4m3fn : type, Shape(x.sizes()), x);
  sh.residual_out_stride =
      res_out_in != nullptr ? rows(*res_out_in, "residual_out", type, x.sizes(), dev, tail)
                            : sh.heads * W;
  Shape per_row(x.sizes().begin(), x.sizes().end() - 1);
  per_row.push_back(group == 0 ? 1 : (W + 127) / 128);
  const Output scale_output(a[10], "scales", at::kFloat, per_row, x);
  const Call call(dev, a[11]);
  const Tensor out = output.make(x);
  std::optional<Tensor> res_out, scales;
  if (res_out_in != nullptr) res_out = *res_out_in;
  else if (res != nullptr) res_out = at::empty(x.sizes(), x.options());
  if (bits8) scales = scale_output.make(x);
  const uint32_t flags = static_cast<uint32_t>(integer(a[5]));
  call.launch("kda_rms_norm", [&](void* stream) {
    return kda_rms_norm(x.data_ptr(), as<float>(weight), res ? res->data_ptr() : nullptr,
                        gate ? gate->data_ptr() : nullptr, &sh, out.data_ptr(),
                        res_out ? res_out->data_ptr() : nullptr,
                        scales ? as<float>(scales->data_ptr()) : nullptr, flags, stream);
  });
  PyObject *o = wrap(out), *r = wrap_or_none(res_out), *s = wrap_or_none(scales);
  PyObject* all = (o && r && s) ? PyTuple_Pack(3, o, r, s) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(r);
  Py_XDECREF(s);
  return all;
  END_HANDLE_TH_ERRORS
}

PyObject* set_fail(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_fail, f);
  Py_RETURN_NONE;
}

#define KDA_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_METHOD(conv_prefill), KDA_METHOD(conv_decode),
                         KDA_METHOD(scan_prefill), KDA_METHOD(scan_decode),
                         KDA_METHOD(rms_norm),     {"set_fail", set_fail, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_bind", nullptr, -1, methods,
                      nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_bind() { return PyModule_Create(&module); }

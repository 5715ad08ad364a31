// marshal.cpp -- Python binding of the training operators' frequent calls.
//
// What the rest of the binding does in Python through ctypes -- checking each
// tensor before its pointer crosses the C ABI, allocating outputs, filling
// the argument struct -- done in compiled code: a recurrence step of 64 x 256
// takes the GPU 2 us, and the same checks in Python took ten times that.  The
// C ABI is reached through the addresses that init() is given, so this module
// needs nothing of libtbe.so at link time.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "tbe.h"

namespace {

// The C ABI's functions, in the order of kNames.
struct Abi {
  decltype(&tbe_gated_scan) scan;
  decltype(&tbe_gated_scan_backward) scan_backward;
  decltype(&tbe_gated_scan_step) scan_step;
  decltype(&tbe_gated_scan_states) scan_states;
  decltype(&tbe_gated_scan_workspace_bytes) scan_workspace;
  decltype(&tbe_preference_loss) preference;
  decltype(&tbe_preference_loss_backward_low) preference_backward;
  decltype(&tbe_preference_workspace_bytes) preference_workspace;
  decltype(&tbe_catalogue_loss) catalogue;
  decltype(&tbe_catalogue_loss_backward_full) catalogue_backward;
  decltype(&tbe_catalogue_workspace_bytes) catalogue_workspace;
  decltype(&tbe_linear_attention) linear;
  decltype(&tbe_linear_attention_backward) linear_backward;
  decltype(&tbe_linear_attention_step) linear_step;
  decltype(&tbe_linear_attention_workspace_bytes) linear_workspace;
  decltype(&tbe_status_string) status_string;
} abi = {};
const char* const kNames[] = {"tbe_gated_scan",
                              "tbe_gated_scan_backward",
                              "tbe_gated_scan_step",
                              "tbe_gated_scan_states",
                              "tbe_gated_scan_workspace_bytes",
                              "tbe_preference_loss",
                              "tbe_preference_loss_backward_low",
                              "tbe_preference_workspace_bytes",
                              "tbe_catalogue_loss",
                              "tbe_catalogue_loss_backward_full",
                              "tbe_catalogue_workspace_bytes",
                              "tbe_linear_attention",
                              "tbe_linear_attention_backward",
                              "tbe_linear_attention_step",
                              "tbe_linear_attention_workspace_bytes",
                              "tbe_status_string"};
PyObject* error_type = nullptr;

struct Refused {
  std::string what;
};

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (void)std::initializer_list<int>{((s << a), 0)...};
  throw Refused{s.str()};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(what, " must be a tensor");
  return THPVariable_Unpack(o);
}

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? TBE_F32 : t == at::kHalf ? TBE_F16 : t == at::kBFloat16 ? TBE_BF16 : -1;
}

// A [rows, cols] argument with consecutive columns; its row stride.
int64_t rows_of(const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, at::Device dev, const char* what) {
  if (t.device() != dev || !dev.is_cuda())
    refuse(what, " must be a CUDA tensor on the device of the other arguments (got ", t.device(), ")");
  if (t.scalar_type() != type) refuse(what, " has dtype ", t.scalar_type(), "; expected ", type);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(what, " has shape ", t.sizes(), "; expected [", rows, ", ", cols, "]");
  const int64_t stride = rows > 1 ? t.stride(0) : cols;
  if ((cols > 1 && rows > 0 && t.stride(1) != 1) || stride < cols)
    refuse(what, " must have consecutive columns and rows that do not overlap");
  return stride;
}

// A contiguous argument of exactly `shape`; its address.
void* vector_of(PyObject* o, at::IntArrayRef shape, at::ScalarType type, at::ScalarType other, at::Device dev,
                const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.device() != dev || (t.scalar_type() != type && t.scalar_type() != other) || t.sizes() != shape ||
      !t.is_contiguous())
    refuse(what, " must be a contiguous ", type, " tensor of shape ", shape, " on ", dev, " (got ", t.scalar_type(), ", ",
           t.sizes(), ", ", t.device(), ")");
  return t.data_ptr();
}
template <typename T>
T* floats_of(PyObject* o, at::IntArrayRef shape, at::Device dev, const char* what) {
  return o == Py_None ? nullptr : static_cast<T*>(vector_of(o, shape, at::kFloat, at::kFloat, dev, what));
}
int32_t* status_of(PyObject* o, at::Device dev) {
  return o == Py_None ? nullptr : static_cast<int32_t*>(vector_of(o, {1}, at::kInt, at::kInt, dev, "dev_status"));
}

double number_of(PyObject* o) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) throw Refused{""};
  return d;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

bool truth_of(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw Refused{""};
  return t != 0;
}

// Where a call's kernels go: the stream of a handle (an integer), or the
// current one for None.  It is made current while the call allocates, so that
// new memory is the stream's own: a workspace that goes back at the end of the
// call is then only handed out again behind the kernels that use it.
class Stream {
 public:
  Stream(PyObject* o, at::Device dev) : device_(dev), caller_(c10::cuda::getCurrentCUDAStream(dev.index())), s_(caller_) {
    if (o == Py_None) return;
    void* handle = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused{""};
    if (handle == caller_.stream()) return;
    s_ = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), dev.index());
    use_.reset_stream(s_);
  }
  void* handle() const { return s_.stream(); }
  // A result.  The caller's own stream is as likely to use it, so that its
  // memory is not handed out again before that one is through with it either.
  at::Tensor result(at::IntArrayRef shape, at::ScalarType type) const {
    at::Tensor t = empty(shape, type, caller_.device());
    if (handle() != caller_.stream()) t.record_stream(caller_.unwrap());
    return t;
  }
  at::Tensor workspace(size_t bytes) const { return empty({(int64_t)bytes}, at::kByte, caller_.device()); }

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::CUDAStream caller_, s_;
  c10::cuda::OptionalCUDAStreamGuard use_;
};

void check(int rc, const char* what) {
  if (rc != TBE_OK) refuse(what, " failed: ", abi.status_string(rc), " (", rc, ")");
}

// Arguments that the three scan calls share.
struct Scan {
  tbe_scan_inputs in;
  at::ScalarType type;
  at::Device dev{at::kCPU};
};
Scan scan_of(PyObject* x_, PyObject* r_, PyObject* g_, PyObject* decay_, PyObject* offsets_, PyObject* h0_,
             PyObject* sharpness) {
  const at::Tensor& x = tensor(x_, "x");
  Scan s = {};
  s.type = x.scalar_type();
  s.dev = x.device();
  s.in.dtype = dtype_code(s.type);
  if (x.dim() != 2 || s.in.dtype < 0)
    refuse("x must be a [tokens, channels] tensor of float32, float16 or bfloat16 (got ", s.type, ", ", x.sizes(), ")");
  const int64_t N = x.size(0), C = x.size(1);
  const at::Tensor &r = tensor(r_, "recur"), &g = tensor(g_, "gate");
  s.in.x_stride = rows_of(x, N, C, s.type, s.dev, "x");
  s.in.recur_stride = rows_of(r, N, C, s.type, s.dev, "recur");
  s.in.gate_stride = rows_of(g, N, C, s.type, s.dev, "gate");
  int64_t S = N;
  if (offsets_ != nullptr) {
    const at::Tensor& o = tensor(offsets_, "offsets");
    S = o.numel() - 1;
    if (S < 0) refuse("offsets must hold at least one entry");
    s.in.offsets = vector_of(offsets_, {S + 1}, at::kLong, at::kInt, s.dev, "offsets");
    s.in.offsets_i32 = o.scalar_type() == at::kInt;
  }
  if (C > INT32_MAX || S > INT32_MAX) refuse("too many channels or sequences");
  if (decay_ == Py_None) refuse("decay is required");
  s.in.decay = floats_of<const float>(decay_, {C}, s.dev, "decay");
  s.in.h0 = h0_ == nullptr ? nullptr : floats_of<const float>(h0_, {S, C}, s.dev, "h0");
  s.in.tokens = N;
  s.in.sequences = (int32_t)S;
  s.in.channels = (int32_t)C;
  s.in.x = x.data_ptr();
  s.in.recur = r.data_ptr();
  s.in.gate = g.data_ptr();
  s.in.sharpness = (float)number_of(sharpness);
  return s;
}

// An output: the given tensor, or a new one.  Returns its row stride.
int64_t output(PyObject* given, int64_t rows, int64_t cols, const Scan& s, const Stream& stream, const char* what,
               at::Tensor& t) {
  if (given == Py_None) {
    t = stream.result({rows, cols}, s.type);
    return cols;
  }
  t = tensor(given, what);
  return rows_of(t, rows, cols, s.type, s.dev, what);
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* items[] = {wrap(t)...};
  PyObject* r = PyTuple_New(sizeof...(T));
  for (size_t i = 0; i < sizeof...(T); ++i) {
    if (!items[i]) Py_CLEAR(r);
    if (r) PyTuple_SET_ITEM(r, i, items[i]);
  }
  return r;
}

// (x, recur, gate, decay, offsets, h0, sharpness, want_states, out, dev_status, stream)
PyObject* scan(PyObject* const* a) {
  const Scan s = scan_of(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
  const int64_t N = s.in.tokens, C = s.in.channels, S = s.in.sequences;
  const Stream stream(a[10], s.dev);
  at::Tensor h, states, ws;
  const int64_t stride = output(a[8], N, C, s, stream, "out", h);
  at::Tensor h_last = stream.result({S, C}, at::kFloat);
  if (truth_of(a[7])) states = stream.result({abi.scan_states(N), C}, at::kFloat);
  const size_t bytes = abi.scan_workspace(N, s.in.channels, s.in.dtype, 0);
  if (bytes) ws = stream.workspace(bytes);
  check(abi.scan(&s.in, h.data_ptr(), stride, static_cast<float*>(h_last.data_ptr()),
                 states.defined() ? static_cast<float*>(states.data_ptr()) : nullptr, bytes ? ws.data_ptr() : nullptr, bytes,
                 status_of(a[9], s.dev), stream.handle()),
        "tbe_gated_scan");
  return tuple(h, h_last, states);
}

// (dh, x, recur, gate, decay, offsets, states, h0, dh_last, sharpness, out, dev_status, stream)
PyObject* scan_backward(PyObject* const* a) {
  const Scan s = scan_of(a[1], a[2], a[3], a[4], a[5], a[7], a[9]);
  const int64_t N = s.in.tokens, C = s.in.channels, S = s.in.sequences;
  const Stream stream(a[12], s.dev);
  const at::Tensor& dh = tensor(a[0], "dh");
  const int64_t dh_stride = rows_of(dh, N, C, s.type, s.dev, "dh");
  if (a[6] == Py_None) refuse("states is required");
  const float* states = floats_of<const float>(a[6], {abi.scan_states(N), C}, s.dev, "states");
  const float* dh_last = floats_of<const float>(a[8], {S, C}, s.dev, "dh_last");
  PyObject* given[3] = {Py_None, Py_None, Py_None};
  if (a[10] != Py_None) {
    if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 3) refuse("out must be a tuple of three tensors");
    for (int i = 0; i < 3; ++i) given[i] = PyTuple_GET_ITEM(a[10], i);
  }
  at::Tensor dx, dr, dg, dh0, ws;
  tbe_scan_grads g = {};
  g.dx_stride = output(given[0], N, C, s, stream, "dx", dx);
  g.drecur_stride = output(given[1], N, C, s, stream, "drecur", dr);
  g.dgate_stride = output(given[2], N, C, s, stream, "dgate", dg);
  at::Tensor ddecay = stream.result({C}, at::kFloat);
  if (a[7] != Py_None) dh0 = stream.result({S, C}, at::kFloat);
  g.dx = dx.data_ptr();
  g.drecur = dr.data_ptr();
  g.dgate = dg.data_ptr();
  g.ddecay = static_cast<float*>(ddecay.data_ptr());
  g.dh0 = dh0.defined() ? static_cast<float*>(dh0.data_ptr()) : nullptr;
  const size_t bytes = abi.scan_workspace(N, s.in.channels, s.in.dtype, 1);
  if (bytes) ws = stream.workspace(bytes);
  check(abi.scan_backward(&s.in, dh.data_ptr(), dh_stride, dh_last, states, &g, bytes ? ws.data_ptr() : nullptr, bytes,
                          status_of(a[11], s.dev), stream.handle()),
        "tbe_gated_scan_backward");
  return tuple(dx, dr, dg, ddecay, dh0);
}

// (x, recur, gate, decay, state, sharpness, out, stream)
PyObject* scan_step(PyObject* const* a) {
  const Scan s = scan_of(a[0], a[1], a[2], a[3], nullptr, nullptr, a[5]);
  const int64_t S = s.in.tokens, C = s.in.channels;
  const Stream stream(a[7], s.dev);
  if (a[4] == Py_None) refuse("state is required");
  float* state = floats_of<float>(a[4], {S, C}, s.dev, "state");
  at::Tensor h;
  const int64_t stride = output(a[6], S, C, s, stream, "out", h);
  check(abi.scan_step(&s.in, state, h.data_ptr(), stride, stream.handle()), "tbe_gated_scan_step");
  return wrap(h);
}

struct Preference {
  tbe_preference_inputs in;
  at::ScalarType type;
  at::Device dev{at::kCPU};
  at::Tensor dlogits;
};
Preference preference_of(PyObject* const* a, double beta, double smoothing) {
  const at::Tensor& x = tensor(a[0], "logits");
  Preference p = {};
  p.type = x.scalar_type();
  p.dev = x.device();
  p.in.dtype = dtype_code(p.type);
  if (x.dim() != 2 || p.in.dtype < 0)
    refuse("logits must be a [tokens, vocab] tensor of float32, float16 or bfloat16 (got ", p.type, ", ", x.sizes(), ")");
  const int64_t N = x.size(0), V = x.size(1);
  p.in.logits_stride = rows_of(x, N, V, p.type, p.dev, "logits");
  if (N < 1 || V < 1 || V > INT32_MAX)
    refuse("logits must have at least one row and one column (and fewer than 2^31 columns)");
  const int64_t Q = tensor(a[3], "ref_logps").numel();
  if (Q < 2 || Q % 2 || Q / 2 > INT32_MAX) refuse("ref_logps must hold two sequences per pair");
  p.in.labels = static_cast<const int64_t*>(vector_of(a[1], {N}, at::kLong, at::kLong, p.dev, "labels"));
  p.in.offsets = static_cast<const int64_t*>(vector_of(a[2], {Q + 1}, at::kLong, at::kLong, p.dev, "offsets"));
  p.in.ref_logps = floats_of<const float>(a[3], {Q}, p.dev, "ref_logps");
  p.in.logits = x.data_ptr();
  p.in.tokens = N;
  p.in.vocab = (int32_t)V;
  p.in.pairs = (int32_t)(Q / 2);
  p.in.beta = (float)beta;
  p.in.label_smoothing = (float)smoothing;
  return p;
}
// The gradient's room: the given tensor, or a new one with the logits' row
// stride.  Rows of a narrow view of a wide tensor (more than twice their
// length, and 64 elements, apart) are put as close together as leaves each its
// place in a 16-byte piece.  The first row starts at the same place of a piece
// as the logits' (which may be columns from an odd one on of a wider tensor),
// so that all rows do: only then are they read and written by whole pieces
// (loss and gradient, 2,000 rows of 10,000 bf16 that start on an odd column:
// 29.7 us, an element at a time 49.1 us).
int64_t gradient_room(Preference& p, PyObject* given, const Stream& s) {
  const int64_t N = p.in.tokens, V = p.in.vocab, piece = p.in.dtype == TBE_F32 ? 4 : 8;
  if (given != Py_None) {
    p.dlogits = tensor(given, "dlogits");
    return rows_of(p.dlogits, N, V, p.type, p.dev, "dlogits");
  }
  int64_t stride = p.in.logits_stride;
  if (stride > 2 * V + 64) stride = V + (stride - V) % piece;
  const int64_t first = (int64_t)((uintptr_t)p.in.logits % 16) * piece / 16;
  if (first == 0 && stride == V) p.dlogits = s.result({N, V}, p.type);
  else p.dlogits = s.result({N * stride + first}, p.type).as_strided({N, V}, {stride, 1}, first);
  return stride;
}

// (logits, labels, offsets, ref_logps, beta, label_smoothing, want_grad, grad_scale, dlogits, dev_status, stream)
// -> (one fp32 buffer: loss, seq_logps, margins, lse, coef and the workspace, which begins with lse_low; dlogits)
PyObject* preference(PyObject* const* a) {
  Preference p = preference_of(a, number_of(a[4]), number_of(a[5]));
  const double scale = number_of(a[7]);
  const Stream stream(a[10], p.dev);
  int64_t d_stride = 0;
  if (a[8] != Py_None || truth_of(a[6])) d_stride = gradient_room(p, a[8], stream);
  const int64_t N = p.in.tokens, P = p.in.pairs;
  const int64_t start = (4 * (1 + 3 * P + 2 * N) + 255) / 256 * 256;
  const size_t bytes = abi.preference_workspace(N, p.in.vocab, p.in.pairs, p.in.dtype);
  at::Tensor room = stream.result({(start + (int64_t)bytes) / 4}, at::kFloat);
  float* f = static_cast<float*>(room.data_ptr());
  check(abi.preference(&p.in, f, f + 1, f + 1 + 2 * P, f + 1 + 3 * P, f + 1 + 3 * P + N,
                       p.dlogits.defined() ? p.dlogits.data_ptr() : nullptr, d_stride, (float)scale, f + start / 4, bytes,
                       status_of(a[9], p.dev), stream.handle()),
        "tbe_preference_loss");
  return tuple(room, p.dlogits);
}

// (logits, labels, offsets, ref_logps, lse, lse_low, coef, grad_scale, dlogits, stream) -> dlogits
PyObject* preference_backward(PyObject* const* a) {
  Preference p = preference_of(a, 1.0, 0.0);
  const double scale = number_of(a[7]);
  const Stream stream(a[9], p.dev);
  const int64_t N = p.in.tokens;
  for (int i = 4; i < 7; ++i)
    if (a[i] == Py_None) refuse("lse, lse_low and coef are required");
  const float* lse = floats_of<const float>(a[4], {N}, p.dev, "lse");
  const float* low = floats_of<const float>(a[5], {N}, p.dev, "lse_low");
  const float* coef = floats_of<const float>(a[6], {N}, p.dev, "coef");
  const int64_t stride = gradient_room(p, a[8], stream);
  check(abi.preference_backward(&p.in, lse, low, coef, (float)scale, p.dlogits.data_ptr(), stride, stream.handle()),
        "tbe_preference_loss_backward");
  return wrap(p.dlogits);
}

// What the two catalogue calls share.
struct Catalogue {
  tbe_catalogue_inputs in;
  at::ScalarType type;
  at::Device dev{at::kCPU};
  at::Tensor dhidden, dweights;
  int64_t dhidden_stride, dweights_stride;
};
Catalogue catalogue_of(PyObject* hidden, PyObject* weights, PyObject* labels, PyObject* logit_scale) {
  const at::Tensor &h = tensor(hidden, "hidden"), &w = tensor(weights, "weights");
  Catalogue c = {};
  c.type = h.scalar_type();
  c.dev = h.device();
  c.in.dtype = dtype_code(c.type);
  if (h.dim() != 2 || (c.in.dtype != TBE_F16 && c.in.dtype != TBE_BF16))
    refuse("hidden must be a [tokens, width] tensor of float16 or bfloat16 (got ", c.type, ", ", h.sizes(), ")");
  if (w.dim() != 2) refuse("weights must be a [vocab, width] tensor (got ", w.sizes(), ")");
  const int64_t N = h.size(0), D = h.size(1), V = w.size(0);
  if (N < 1 || D < 1 || V < 1 || D > INT32_MAX || V > INT32_MAX)
    refuse("hidden and weights must have at least one row and one column (and fewer than 2^31)");
  c.in.hidden_stride = rows_of(h, N, D, c.type, c.dev, "hidden");
  c.in.weights_stride = rows_of(w, V, D, c.type, c.dev, "weights");
  c.in.labels = static_cast<const int64_t*>(vector_of(labels, {N}, at::kLong, at::kLong, c.dev, "labels"));
  c.in.hidden = h.data_ptr();
  c.in.weights = w.data_ptr();
  c.in.tokens = N;
  c.in.vocab = (int32_t)V;
  c.in.width = (int32_t)D;
  c.in.logit_scale = (float)number_of(logit_scale);
  return c;
}
void catalogue_grads(Catalogue& c, PyObject* dhidden, PyObject* dweights, const Stream& s) {
  auto one = [&](PyObject* given, int64_t rows, const char* what, at::Tensor& t) {
    t = given == Py_None ? s.result({rows, c.in.width}, c.type) : tensor(given, what);
    return rows_of(t, rows, c.in.width, c.type, c.dev, what);
  };
  c.dhidden_stride = one(dhidden, c.in.tokens, "dhidden", c.dhidden);
  c.dweights_stride = one(dweights, c.in.vocab, "dweights", c.dweights);
}

// (hidden, weights, labels, logit_scale, want_grad, grad_scale, dhidden, dweights, dev_status, stream)
// -> (loss, token_loss, lse, dhidden, dweights)
PyObject* catalogue(PyObject* const* a) {
  Catalogue c = catalogue_of(a[0], a[1], a[2], a[3]);
  const double scale = number_of(a[5]);
  const Stream stream(a[9], c.dev);
  const bool grad = truth_of(a[4]) || a[6] != Py_None || a[7] != Py_None;
  if (grad) catalogue_grads(c, a[6], a[7], stream);
  at::Tensor loss = stream.result({}, at::kFloat), token_loss = stream.result({c.in.tokens}, at::kFloat),
             lse = stream.result({c.in.tokens}, at::kFloat);
  const size_t bytes = abi.catalogue_workspace(&c.in, grad);
  at::Tensor ws = stream.workspace(bytes);
  check(abi.catalogue(&c.in, static_cast<float*>(loss.data_ptr()), static_cast<float*>(token_loss.data_ptr()),
                      static_cast<float*>(lse.data_ptr()), grad ? c.dhidden.data_ptr() : nullptr, c.dhidden_stride,
                      grad ? c.dweights.data_ptr() : nullptr, c.dweights_stride, (float)scale, ws.data_ptr(), bytes,
                      status_of(a[8], c.dev), stream.handle()),
        "tbe_catalogue_loss");
  return tuple(loss, token_loss, lse, c.dhidden, c.dweights);
}

// (hidden, weights, labels, lse, logit_scale, grad_scale, dhidden, dweights, dev_status, stream, token_loss)
// -> (dhidden, dweights)
PyObject* catalogue_backward(PyObject* const* a) {
  Catalogue c = catalogue_of(a[0], a[1], a[2], a[4]);
  const double scale = number_of(a[5]);
  const Stream stream(a[9], c.dev);
  if (a[3] == Py_None) refuse("lse is required");
  const float* lse = floats_of<const float>(a[3], {c.in.tokens}, c.dev, "lse");
  const float* token_loss = floats_of<const float>(a[10], {c.in.tokens}, c.dev, "token_loss");
  catalogue_grads(c, a[6], a[7], stream);
  const size_t bytes = abi.catalogue_workspace(&c.in, 1);
  at::Tensor ws = stream.workspace(bytes);
  check(abi.catalogue_backward(&c.in, lse, token_loss, c.dhidden.data_ptr(), c.dhidden_stride, c.dweights.data_ptr(),
                               c.dweights_stride, (float)scale, ws.data_ptr(), bytes, status_of(a[8], c.dev), stream.handle()),
        "tbe_catalogue_loss_backward");
  return tuple(c.dhidden, c.dweights);
}

// What the three linear attention calls share.
struct Linear {
  tbe_linear_attention_inputs in;
  at::ScalarType type;
  at::Device dev{at::kCPU};
  int64_t S;
};
// A [tokens, heads, head_dim] argument; its token and head strides.
void heads_of(const at::Tensor& t, const Linear& l, const char* what, int64_t& stride, int64_t& head) {
  const int64_t N = l.in.tokens, H = l.in.heads, d = l.in.head_dim;
  if (t.device() != l.dev || !l.dev.is_cuda())
    refuse(what, " must be a CUDA tensor on the device of the other arguments (got ", t.device(), ")");
  if (t.scalar_type() != l.type) refuse(what, " has dtype ", t.scalar_type(), "; expected ", l.type);
  if (t.dim() != 3 || t.size(0) != N || t.size(1) != H || t.size(2) != d)
    refuse(what, " has shape ", t.sizes(), "; expected [", N, ", ", H, ", ", d, "]");
  head = H > 1 ? t.stride(1) : d;
  stride = N > 1 ? t.stride(0) : H * head;
  if ((d > 1 && N > 0 && t.stride(2) != 1) || head < d || stride < d ||
      (stride < (H - 1) * head + d && head < (N - 1) * stride + d))
    refuse(what, " must be consecutive along its last dimension, with tokens and heads that do not overlap");
}
Linear linear_of(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* decay, PyObject* offsets, PyObject* s0,
                 PyObject* scale) {
  const at::Tensor& q = tensor(q_, "q");
  Linear l = {};
  l.type = q.scalar_type();
  l.dev = q.device();
  l.in.dtype = dtype_code(l.type);
  if (q.dim() != 3 || (l.in.dtype != TBE_F16 && l.in.dtype != TBE_BF16))
    refuse("q must be a [tokens, heads, head_dim] tensor of float16 or bfloat16 (got ", l.type, ", ", q.sizes(), ")");
  if (q.size(1) < 1 || q.size(1) > (1 << 16) || q.size(2) < 1 || q.size(2) > TBE_LINEAR_MAX_HEAD_DIM)
    refuse("heads must be 1 to 65536 and head_dim 1 to ", TBE_LINEAR_MAX_HEAD_DIM, " (got ", q.size(1), " and ", q.size(2), ")");
  l.in.tokens = q.size(0);
  l.in.heads = (int32_t)q.size(1);
  l.in.head_dim = (int32_t)q.size(2);
  const at::Tensor &k = tensor(k_, "k"), &v = tensor(v_, "v");
  heads_of(q, l, "q", l.in.q_stride, l.in.q_head_stride);
  heads_of(k, l, "k", l.in.k_stride, l.in.k_head_stride);
  heads_of(v, l, "v", l.in.v_stride, l.in.v_head_stride);
  l.S = l.in.tokens;
  if (offsets != nullptr) {
    const at::Tensor& o = tensor(offsets, "offsets");
    l.S = o.numel() - 1;
    if (l.S < 0) refuse("offsets must hold at least one entry");
    l.in.offsets = vector_of(offsets, {l.S + 1}, at::kLong, at::kInt, l.dev, "offsets");
    l.in.offsets_i32 = o.scalar_type() == at::kInt;
  }
  if (l.S > INT32_MAX) refuse("too many sequences");
  if (decay == Py_None) refuse("decay is required");
  l.in.decay = floats_of<const float>(decay, {l.in.heads}, l.dev, "decay");
  l.in.sequences = (int32_t)l.S;
  if (s0 != nullptr) l.in.s0 = floats_of<const float>(s0, {l.S, l.in.heads, l.in.head_dim, l.in.head_dim}, l.dev, "s0");
  l.in.q = q.data_ptr();
  l.in.k = k.data_ptr();
  l.in.v = v.data_ptr();
  l.in.scale = (float)number_of(scale);
  return l;
}
at::Tensor linear_output(PyObject* given, const Linear& l, const Stream& s, const char* what, int64_t& stride, int64_t& head) {
  at::Tensor t = given == Py_None ? s.result({l.in.tokens, l.in.heads, l.in.head_dim}, l.type) : tensor(given, what);
  heads_of(t, l, what, stride, head);
  return t;
}

// (q, k, v, decay, offsets, s0, scale, want_last, out, dev_status, stream) -> (o, s_last)
PyObject* linear(PyObject* const* a) {
  const Linear l = linear_of(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
  const Stream stream(a[10], l.dev);
  int64_t stride, head;
  at::Tensor o = linear_output(a[8], l, stream, "out", stride, head), last, ws;
  if (truth_of(a[7])) last = stream.result({l.S, l.in.heads, l.in.head_dim, l.in.head_dim}, at::kFloat);
  const size_t bytes = abi.linear_workspace(l.in.tokens, l.in.heads, l.in.head_dim, 0);
  if (bytes) ws = stream.workspace(bytes);
  check(abi.linear(&l.in, o.data_ptr(), stride, head, last.defined() ? static_cast<float*>(last.data_ptr()) : nullptr,
                   bytes ? ws.data_ptr() : nullptr, bytes, status_of(a[9], l.dev), stream.handle()),
        "tbe_linear_attention");
  return tuple(o, last);
}

// (do, q, k, v, decay, offsets, s0, ds_last, scale, out, dev_status, stream) -> (dq, dk, dv, ds0)
PyObject* linear_backward(PyObject* const* a) {
  const Linear l = linear_of(a[1], a[2], a[3], a[4], a[5], a[6], a[8]);
  const Stream stream(a[11], l.dev);
  const at::Tensor& d = tensor(a[0], "do");
  int64_t stride, head;
  heads_of(d, l, "do", stride, head);
  const int64_t shape[4] = {l.S, l.in.heads, l.in.head_dim, l.in.head_dim};
  const float* ds_last = floats_of<const float>(a[7], shape, l.dev, "ds_last");
  PyObject* given[3] = {Py_None, Py_None, Py_None};
  if (a[9] != Py_None) {
    if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 3) refuse("out must be a tuple of three tensors");
    for (int i = 0; i < 3; ++i) given[i] = PyTuple_GET_ITEM(a[9], i);
  }
  tbe_linear_attention_grads g = {};
  at::Tensor dq = linear_output(given[0], l, stream, "dq", g.dq_stride, g.dq_head_stride),
             dk = linear_output(given[1], l, stream, "dk", g.dk_stride, g.dk_head_stride),
             dv = linear_output(given[2], l, stream, "dv", g.dv_stride, g.dv_head_stride), ds0, ws;
  g.dq = dq.data_ptr();
  g.dk = dk.data_ptr();
  g.dv = dv.data_ptr();
  if (a[6] != Py_None) {
    ds0 = stream.result(shape, at::kFloat);
    g.ds0 = static_cast<float*>(ds0.data_ptr());
  }
  const size_t bytes = abi.linear_workspace(l.in.tokens, l.in.heads, l.in.head_dim, 1);
  if (bytes) ws = stream.workspace(bytes);
  check(abi.linear_backward(&l.in, d.data_ptr(), stride, head, ds_last, &g, bytes ? ws.data_ptr() : nullptr, bytes,
                            status_of(a[10], l.dev), stream.handle()),
        "tbe_linear_attention_backward");
  return tuple(dq, dk, dv, ds0);
}

// (q, k, v, decay, state, scale, out, stream) -> o
PyObject* linear_step(PyObject* const* a) {
  const Linear l = linear_of(a[0], a[1], a[2], a[3], nullptr, nullptr, a[5]);
  const Stream stream(a[7], l.dev);
  if (a[4] == Py_None) refuse("state is required");
  float* state = floats_of<float>(a[4], {l.S, l.in.heads, l.in.head_dim, l.in.head_dim}, l.dev, "state");
  int64_t stride, head;
  at::Tensor o = linear_output(a[6], l, stream, "out", stride, head);
  check(abi.linear_step(&l.in, state, o.data_ptr(), stride, head, stream.handle()), "tbe_linear_attention_step");
  return wrap(o);
}

// Calls F with its arguments, with refusals as TBEError and memory that runs
// out as PyTorch's own error.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t COUNT>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != COUNT) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", COUNT, n);
    return nullptr;
  }
  if (!error_type) {
    PyErr_SetString(PyExc_RuntimeError, "init() has not been called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(error_type, e.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    if (PyErr_Occurred()) return nullptr;
    if (PyObject* torch = PyImport_ImportModule("torch")) {
      if (PyObject* type = PyObject_GetAttrString(torch, "OutOfMemoryError")) {
        PyErr_SetString(type, e.what_without_backtrace());
        Py_DECREF(type);
      }
      Py_DECREF(torch);
    }
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// init(error type, {name: address of the C ABI's function})
PyObject* init(PyObject*, PyObject* args) {
  PyObject *type, *table;
  if (!PyArg_ParseTuple(args, "OO!", &type, &PyDict_Type, &table)) return nullptr;
  void* found[sizeof(kNames) / sizeof(kNames[0])];
  static_assert(sizeof(found) == sizeof(Abi), "one name per function");
  for (size_t i = 0; i < sizeof(kNames) / sizeof(kNames[0]); ++i) {
    PyObject* address = PyDict_GetItemString(table, kNames[i]);
    if (!address) return PyErr_Format(PyExc_KeyError, "%s", kNames[i]);
    found[i] = PyLong_AsVoidPtr(address);
    if (PyErr_Occurred()) return nullptr;
  }
  memcpy(&abi, found, sizeof(abi));
  Py_INCREF(type);
  Py_XSETREF(error_type, type);
  Py_RETURN_NONE;
}

#define FAST(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<f, n>)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         {"gated_scan", FAST(scan, 11)},
                         {"gated_scan_backward", FAST(scan_backward, 13)},
                         {"gated_scan_step", FAST(scan_step, 8)},
                         {"preference_loss", FAST(preference, 11)},
                         {"preference_loss_backward", FAST(preference_backward, 10)},
                         {"catalogue_loss", FAST(catalogue, 10)},
                         {"linear_attention", FAST(linear, 11)},
                         {"linear_attention_backward", FAST(linear_backward, 12)},
                         {"linear_attention_step", FAST(linear_step, 8)},
                         {"catalogue_loss_backward", FAST(catalogue_backward, 11)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }

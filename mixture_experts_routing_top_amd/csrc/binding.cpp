// The binding of the gate, layer norm, clipping and microscaled-block calls: argument
// checks, output allocation and the C call in one native function each.
//
// These operators take a few microseconds on the GPU for a small batch, less than
// an interpreter needs to check a call's arguments and allocate its outputs one
// by one.  The functions here take their arguments by position, all given, from
// the documented Python functions; they raise TypeError or ValueError, or return
// the C call's non-zero status, which the caller turns into MoEError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cstdint>
#include <vector>

#include "moe.h"

namespace {

using Args = PyObject* const*;

const at::Tensor& tensor(PyObject* o) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), "expected a torch tensor");
  return THPVariable_Unpack(o);
}

// checks that hold for every tensor of a call
const at::Tensor& on_gpu(const at::Tensor& t) {
  TORCH_CHECK_VALUE(t.is_cuda(), "tensors passed to the MoE library must live on the GPU");
  TORCH_CHECK_VALUE(t.is_contiguous(), "tensors passed to the MoE library must be contiguous");
  return t;
}

moe_dtype dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return MOE_F32;
  TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, "activations must be bfloat16 or float32, got ", t.scalar_type());
  return MOE_BF16;
}

void expect(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev, const char* name) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.device() == dev && t.sizes() == shape, name, ": expected ", type, " ",
                    shape, " on ", dev, ", got ", t.scalar_type(), " ", t.sizes(), " on ", t.device());
  on_gpu(t);
}

// a given tensor's address, or null for None
void* given(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  expect(t, shape, type, dev, name);
  return t.data_ptr();
}

at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev, const char* name) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  const at::Tensor& t = tensor(o);
  expect(t, shape, type, dev, name);
  return t;
}

// A call's stream.  One that the caller gave is the current one while the call
// allocates: what is allocated then belongs to it in torch's allocator, which hands the
// memory of a workspace dropped on return, or of an output dropped early, only to later
// work of the same stream, and takes none that another stream still uses.
struct Stream {
  void* raw;
  c10::OptionalStreamGuard current;
};

// None (the current stream), a torch stream, its handle as an integer, or any
// object with the handle as `cuda_stream`
Stream stream_of(PyObject* o, const at::Device& dev) {
  if (o == Py_None) return {c10::hip::getCurrentHIPStream(dev.index()).stream(), c10::OptionalStreamGuard()};
  THPObjectPtr handle(PyIndex_Check(o) ? PyNumber_Index(o) : PyObject_GetAttrString(o, "cuda_stream"));
  TORCH_CHECK_TYPE(handle, "stream: expected a torch stream, its handle or an object with a cuda_stream");
  void* raw = PyLong_AsVoidPtr(handle.get());
  if (PyErr_Occurred()) throw python_error();
  if (PyObject_IsInstance(o, reinterpret_cast<PyObject*>(THPStreamClass)) == 1) {
    const auto* s = reinterpret_cast<THPStream*>(o);
    const c10::Stream st = c10::Stream::unpack3(s->stream_id, static_cast<c10::DeviceIndex>(s->device_index),
                                                static_cast<c10::DeviceType>(s->device_type));
    TORCH_CHECK_VALUE(st.device_index() == dev.index(), "the stream belongs to another device than the tensors");
    return {raw, c10::OptionalStreamGuard(st)};
  }
  // torch's streams carry the device type of its tensors, which an external HIP stream's does not
  const auto id = c10::hip::getStreamFromExternal(static_cast<hipStream_t>(raw), dev.index()).id();
  return {raw, c10::OptionalStreamGuard(c10::Stream(c10::Stream::UNSAFE, dev, id))};
}

// A given workspace, checked, or one for this call.
at::Tensor workspace_of(PyObject* o, size_t need, const at::Device& dev, const char* name) {
  if (o != Py_None) {
    const at::Tensor& t = tensor(o);
    on_gpu(t);
    TORCH_CHECK_VALUE(t.device() == dev, name, ": on another device than the call's tensors");
    TORCH_CHECK_VALUE(t.nbytes() >= need, name, ": needs ", need, " bytes, got ", t.nbytes());
    return t;
  }
  return at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(dev));
}

int32_t* check_word(PyObject* o, const at::Device& dev) {
  return static_cast<int32_t*>(given(o, {1}, at::kInt, dev, "check"));
}

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int small(PyObject* o) {
  const int64_t v = whole(o);
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, "integer out of range: ", v);
  return static_cast<int>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* none() { Py_RETURN_NONE; }

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = (a && b) ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

template <typename F>
int without_gil(const at::Device& dev, F call) {
  const c10::DeviceGuard guard(dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call();
  Py_END_ALLOW_THREADS;
  return rc;
}

// logits, k, score, bias, n_groups, keep_groups (None: all), group_score, renorm, scale, topk_idx, topk_w, stream, check
PyObject* gate(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const at::Tensor& lg = tensor(a[0]);
  const moe_dtype dt = dtype_code(lg);
  TORCH_CHECK_VALUE(lg.dim() == 2, "router logits must be [T, E]");
  on_gpu(lg);
  const at::Device dev = lg.device();
  const int64_t T = lg.size(0), E = lg.size(1), k = small(a[1]);
  TORCH_CHECK_VALUE(E <= INT32_MAX && k >= 0, "k or E out of range");
  auto* bias = static_cast<const float*>(given(a[3], {E}, at::kFloat, dev, "bias"));
  const Stream s = stream_of(a[11], dev);
  const at::Tensor idx = output(a[9], {T, k}, at::kInt, dev, "topk_idx");
  const at::Tensor w = output(a[10], {T, k}, at::kFloat, dev, "topk_w");
  int32_t* check = check_word(a[12], dev);
  const int groups = small(a[4]), keep = a[5] == Py_None ? groups : small(a[5]), score = small(a[2]), gs = small(a[6]);
  const int renorm = PyObject_IsTrue(a[7]);
  const float scale = real(a[8]);
  const int rc = without_gil(dev, [&] {
    return moe_gate(lg.data_ptr(), dt, T, static_cast<int>(E), static_cast<int>(k), static_cast<moe_score>(score), bias,
                    groups, keep, static_cast<moe_group_score>(gs), renorm, scale, idx.data_ptr<int32_t>(),
                    w.data_ptr<float>(), check, s.raw);
  });
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return pair(wrap(idx), wrap(w));
  END_HANDLE_TH_ERRORS
}

// logits, topk_idx, d_topk_w, score, renorm, scale, d_logits, stream, check
PyObject* gate_backward(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const at::Tensor& lg = tensor(a[0]);
  const moe_dtype dt = dtype_code(lg);
  TORCH_CHECK_VALUE(lg.dim() == 2, "router logits must be [T, E]");
  on_gpu(lg);
  const at::Device dev = lg.device();
  const at::Tensor& idx = tensor(a[1]);
  TORCH_CHECK_VALUE(idx.dim() == 2, "topk_idx must be [T, k]");
  const int64_t T = lg.size(0), E = lg.size(1), k = idx.size(1);
  TORCH_CHECK_VALUE(E <= INT32_MAX && k <= INT32_MAX, "k or E out of range");
  expect(idx, {T, k}, at::kInt, dev, "topk_idx");
  const at::Tensor& g = tensor(a[2]);
  expect(g, {T, k}, at::kFloat, dev, "d_topk_w");
  const Stream s = stream_of(a[7], dev);
  const at::Tensor d = output(a[6], {T, E}, lg.scalar_type(), dev, "d_logits");
  int32_t* check = check_word(a[8], dev);
  const int score = small(a[3]), renorm = PyObject_IsTrue(a[4]);
  const float scale = real(a[5]);
  const int rc = without_gil(dev, [&] {
    return moe_gate_backward(lg.data_ptr(), dt, T, static_cast<int>(E), static_cast<int>(k),
                             static_cast<moe_score>(score), renorm, scale, idx.data_ptr<int32_t>(),
                             g.data_ptr<float>(), d.data_ptr(), check, s.raw);
  });
  return rc != MOE_OK ? PyLong_FromLong(rc) : wrap(d);
  END_HANDLE_TH_ERRORS
}

struct Vectors {
  void *weight, *bias;
  at::ScalarType type;
  moe_dtype code;
};

// weight and bias of a norm: both float32 or of the rows' dtype
Vectors norm_vectors(const at::Tensor& x, PyObject* weight, PyObject* bias) {
  TORCH_CHECK_VALUE(x.dim() == 2, "layer norm takes rows [T, H]");
  at::ScalarType type = x.scalar_type();
  if (weight != Py_None) type = tensor(weight).scalar_type();
  else if (bias != Py_None) type = tensor(bias).scalar_type();
  TORCH_CHECK_TYPE(type == at::kFloat || type == x.scalar_type(),
                   "weight and bias must be float32 or of the rows' dtype");
  return {given(weight, {x.size(1)}, type, x.device(), "weight"), given(bias, {x.size(1)}, type, x.device(), "bias"),
          type, type == at::kFloat ? MOE_F32 : MOE_BF16};
}

// x, weight, bias, eps, residual, y, x_sum, stream
PyObject* layer_norm(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const at::Tensor& x = tensor(a[0]);
  const moe_dtype dt = dtype_code(x);
  on_gpu(x);
  const at::Device dev = x.device();
  const Vectors v = norm_vectors(x, a[1], a[2]);
  const int64_t T = x.size(0), H = x.size(1);
  TORCH_CHECK_VALUE(H <= INT32_MAX, "H out of range");
  const void* residual = given(a[4], x.sizes(), x.scalar_type(), dev, "residual");
  const bool sums = a[4] != Py_None;
  TORCH_CHECK_VALUE(sums || a[6] == Py_None, "x_sum is written with a residual only");
  const Stream s = stream_of(a[7], dev);
  const at::Tensor y = output(a[5], {T, H}, x.scalar_type(), dev, "y");
  const at::Tensor x_sum = sums ? output(a[6], {T, H}, x.scalar_type(), dev, "x_sum") : at::Tensor();
  const float eps = real(a[3]);
  const int rc = without_gil(dev, [&] {
    return moe_layer_norm(x.data_ptr(), residual, dt, T, static_cast<int>(H), v.weight, v.bias, v.code, eps,
                          sums ? x_sum.data_ptr() : nullptr, y.data_ptr(), s.raw);
  });
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return pair(wrap(y), sums ? wrap(x_sum) : none());
  END_HANDLE_TH_ERRORS
}

// d_y, x, weight, bias, eps, d_skip, d_x, d_weight, d_bias, workspace, stream
PyObject* layer_norm_backward(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const at::Tensor& x = tensor(a[1]);
  const moe_dtype dt = dtype_code(x);
  on_gpu(x);
  const at::Device dev = x.device();
  const Vectors v = norm_vectors(x, a[2], a[3]);
  const int64_t T = x.size(0), H = x.size(1);
  TORCH_CHECK_VALUE(H <= INT32_MAX, "H out of range");
  const at::Tensor& dy = tensor(a[0]);
  expect(dy, x.sizes(), x.scalar_type(), dev, "d_y");
  const void* skip = given(a[5], x.sizes(), x.scalar_type(), dev, "d_skip");
  TORCH_CHECK_VALUE(a[2] != Py_None || a[7] == Py_None, "d_weight: there is no such parameter");
  TORCH_CHECK_VALUE(a[3] != Py_None || a[8] == Py_None, "d_bias: there is no such parameter");
  const Stream s = stream_of(a[10], dev);
  const at::Tensor dx = output(a[6], {T, H}, x.scalar_type(), dev, "d_x");
  const at::Tensor dw = a[2] == Py_None ? at::Tensor() : output(a[7], {H}, v.type, dev, "d_weight");
  const at::Tensor db = a[3] == Py_None ? at::Tensor() : output(a[8], {H}, v.type, dev, "d_bias");
  const size_t need = dw.defined() || db.defined()
                          ? moe_layer_norm_backward_workspace_bytes(T, static_cast<int>(H)) : 0;
  const at::Tensor ws = need ? workspace_of(a[9], need, dev, "layer norm workspace") : at::Tensor();
  const float eps = real(a[4]);
  const int rc = without_gil(dev, [&] {
    return moe_layer_norm_backward(dy.data_ptr(), x.data_ptr(), dt, T, static_cast<int>(H), v.weight, v.code, eps, skip,
                                   dx.data_ptr(), dw.defined() ? dw.data_ptr() : nullptr,
                                   db.defined() ? db.data_ptr() : nullptr, ws.defined() ? ws.data_ptr() : nullptr, need,
                                   s.raw);
  });
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  PyObject *pw = dw.defined() ? wrap(dw) : none(), *pb = db.defined() ? wrap(db) : none(), *px = wrap(dx);
  PyObject* r = px && pw && pb ? PyTuple_Pack(3, px, pw, pb) : nullptr;
  Py_XDECREF(px);
  Py_XDECREF(pw);
  Py_XDECREF(pb);
  return r;
  END_HANDLE_TH_ERRORS
}

struct GradLists {
  std::vector<const void*> grads;
  std::vector<void*> out;
  std::vector<int64_t> numel;
  std::vector<moe_dtype> dt;
};

// grads, out (None: in place), max_norm (None: the norm alone), eps, norm, workspace, stream, check
PyObject* clip_grads(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  THPObjectPtr list(PySequence_Fast(a[0], "grads: expected a list of torch tensors"));
  if (!list) throw python_error();
  const Py_ssize_t m = PySequence_Fast_GET_SIZE(list.get());
  PyObject** items = PySequence_Fast_ITEMS(list.get());
  TORCH_CHECK_VALUE(m <= INT32_MAX, "too many gradients");
  TORCH_CHECK_VALUE(m > 0 || a[4] != Py_None, "an empty list of gradients names no device: pass norm");
  const at::Device dev = a[4] != Py_None ? tensor(a[4]).device() : tensor(items[0]).device();
  TORCH_CHECK_VALUE(dev.is_cuda(), "tensors passed to the MoE library must live on the GPU");
  THPObjectPtr outs;
  PyObject** out_items = nullptr;
  if (a[1] != Py_None) {
    outs = THPObjectPtr(PySequence_Fast(a[1], "out: expected a list of torch tensors"));
    if (!outs) throw python_error();
    TORCH_CHECK_VALUE(PySequence_Fast_GET_SIZE(outs.get()) == m, "out: one tensor for each gradient");
    out_items = PySequence_Fast_ITEMS(outs.get());
  }
  GradLists l;
  l.grads.reserve(m);
  l.out.reserve(m);
  l.numel.reserve(m);
  l.dt.reserve(m);
  for (Py_ssize_t i = 0; i < m; ++i) {
    const at::Tensor& g = tensor(items[i]);
    l.dt.push_back(dtype_code(g));
    TORCH_CHECK_VALUE(g.device() == dev && g.is_contiguous(), "grads[", i, "]: must be contiguous and on ", dev);
    l.grads.push_back(g.data_ptr());
    l.numel.push_back(g.numel());
    if (out_items) {
      const at::Tensor& o = tensor(out_items[i]);
      TORCH_CHECK_VALUE(o.scalar_type() == g.scalar_type() && o.device() == dev && o.sizes() == g.sizes() &&
                            o.is_contiguous(),
                        "out[", i, "]: must be like grads[", i, "] and contiguous");
      l.out.push_back(o.data_ptr());
    } else {
      l.out.push_back(g.data_ptr());
    }
  }
  const Stream s = stream_of(a[6], dev);
  const at::Tensor norm = output(a[4], {1}, at::kFloat, dev, "norm");
  int32_t* check = check_word(a[7], dev);
  const size_t need = moe_grad_norm_workspace_bytes();
  const at::Tensor ws = workspace_of(a[5], need, dev, "gradient norm workspace");
  const bool clips = a[2] != Py_None;
  const float max_norm = clips ? real(a[2]) : 0.f, eps = clips ? real(a[3]) : 0.f;
  const int rc = without_gil(dev, [&] {
    return clips ? moe_clip_grads(l.grads.data(), l.out.data(), l.numel.data(), l.dt.data(), static_cast<int>(m),
                                  max_norm, eps, norm.data_ptr<float>(), ws.data_ptr(), need, check, s.raw)
                 : moe_grad_norm(l.grads.data(), l.numel.data(), l.dt.data(), static_cast<int>(m),
                                 norm.data_ptr<float>(), ws.data_ptr(), need, check, s.raw);
  });
  return rc != MOE_OK ? PyLong_FromLong(rc) : wrap(norm);
  END_HANDLE_TH_ERRORS
}

int64_t blocks_of(int64_t K) { return (K + 31) / 32; }

moe_mx_format format_code(PyObject* o) { return static_cast<moe_mx_format>(small(o)); }

// bits of a code, and the bytes of a row of K
int64_t code_bits(moe_mx_format fmt) { return fmt == MOE_MX_FP8 ? 8 : fmt == MOE_MX_FP6 ? 6 : 4; }
int64_t code_bytes(moe_mx_format fmt, int64_t K) { return (K * code_bits(fmt) + 7) / 8; }

// x, format, q, scale, stream, check
PyObject* mx_quantize(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  const at::Tensor& x = tensor(a[0]);
  const moe_dtype dt = dtype_code(x);
  on_gpu(x);
  TORCH_CHECK_VALUE(x.dim() >= 1, "rows of at least one dimension are quantised");
  const at::Device dev = x.device();
  const moe_mx_format fmt = format_code(a[1]);
  const int64_t K = x.size(-1);
  TORCH_CHECK_VALUE(K >= 1, "rows of no values have no blocks");
  const int64_t R = x.numel() / K;
  std::vector<int64_t> shape = x.sizes().vec(), blocks = shape;
  shape.back() = code_bytes(fmt, K);
  blocks.back() = blocks_of(K);
  const Stream s = stream_of(a[4], dev);
  const at::Tensor q = output(a[2], shape, at::kByte, dev, "q");
  const at::Tensor scale = output(a[3], blocks, at::kByte, dev, "scale");
  int32_t* check = check_word(a[5], dev);
  const int rc = without_gil(dev, [&] {
    return moe_mx_quantize(x.data_ptr(), dt, R, K, fmt, q.data_ptr<uint8_t>(), scale.data_ptr<uint8_t>(), check, s.raw);
  });
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return pair(wrap(q), wrap(scale));
  END_HANDLE_TH_ERRORS
}

// q, scale, format, dtype (0 float32, 1 bfloat16), cols (None: the codes' own), rows, out, stream, check
PyObject* mx_dequantize(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const at::Tensor& q = tensor(a[0]);
  on_gpu(q);
  const at::Device dev = q.device();
  const moe_mx_format fmt = format_code(a[2]);
  TORCH_CHECK_VALUE(q.dim() >= 1 && q.scalar_type() == at::kByte, "q: expected uint8 codes");
  const int64_t bytes = q.size(-1);
  const int64_t K = a[4] == Py_None ? bytes * 8 / code_bits(fmt) : whole(a[4]);
  // (bounded first: of 2^61 values the bytes would come to 0, those of rows that hold none)
  TORCH_CHECK_VALUE(K >= 1 && K < INT64_MAX / 8 && code_bytes(fmt, K) == bytes, "q: rows of ", bytes, " bytes do not hold ", K, " values");
  const int64_t R = q.numel() / bytes;
  std::vector<int64_t> shape = q.sizes().vec(), blocks = shape;
  blocks.back() = blocks_of(K);
  const at::Tensor& scale = tensor(a[1]);
  expect(scale, blocks, at::kByte, dev, "scale");
  shape.back() = K;
  const int32_t* rows = nullptr;
  int64_t n_rows = R;
  if (a[5] != Py_None) {
    const at::Tensor& r = tensor(a[5]);
    TORCH_CHECK_VALUE(r.dim() == 1, "rows must be int32 [n]");
    n_rows = r.size(0);
    rows = static_cast<const int32_t*>(given(a[5], {n_rows}, at::kInt, dev, "rows"));
    shape = {n_rows, K};
  }
  const int code = small(a[3]);
  const Stream s = stream_of(a[7], dev);
  const at::Tensor out = output(a[6], shape, code == MOE_BF16 ? at::kBFloat16 : at::kFloat, dev, "out");
  int32_t* check = check_word(a[8], dev);
  if (n_rows == 0) return wrap(out);   // (an empty row map may have no address)
  const int rc = without_gil(dev, [&] {
    return moe_mx_dequantize(q.data_ptr<uint8_t>(), scale.data_ptr<uint8_t>(), fmt, R, K, rows, n_rows,
                             static_cast<moe_dtype>(code), out.data_ptr(), check, s.raw);
  });
  return rc != MOE_OK ? PyLong_FromLong(rc) : wrap(out);
  END_HANDLE_TH_ERRORS
}

// d_out, y, y_scale (None: y in the dtype), inv_pos, topk_w, d_y, d_topk_w, stream, check
PyObject* combine_backward(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const at::Tensor& d_out = tensor(a[0]);
  const moe_dtype dt = dtype_code(d_out);
  on_gpu(d_out);
  const at::Device dev = d_out.device();
  TORCH_CHECK_VALUE(d_out.dim() == 2, "d_out must be [T, H]");
  const at::Tensor& y = tensor(a[1]);
  TORCH_CHECK_VALUE(y.dim() == 2, "y_perm must be [M, H]");
  const int64_t T = d_out.size(0), H = d_out.size(1), M = y.size(0);
  TORCH_CHECK_VALUE(H <= INT32_MAX, "H out of range");
  const bool kept = a[2] != Py_None;
  expect(y, {M, H}, kept ? at::kByte : d_out.scalar_type(), dev, "y_perm");
  const void* y_scale = given(a[2], {M, blocks_of(H)}, at::kByte, dev, "y_perm's scale");
  const at::Tensor& w = tensor(a[4]);
  TORCH_CHECK_VALUE(w.dim() == 2, "topk_w must be [T, k]");
  const int64_t k = w.size(1);
  TORCH_CHECK_VALUE(k <= INT32_MAX, "k out of range");
  expect(w, {T, k}, at::kFloat, dev, "topk_w");
  const at::Tensor& inv = tensor(a[3]);
  expect(inv, {T, k}, at::kInt, dev, "inv_pos");
  const Stream s = stream_of(a[7], dev);
  const at::Tensor d_y = output(a[5], {M, H}, d_out.scalar_type(), dev, "d_y");
  const at::Tensor d_w = output(a[6], {T, k}, at::kFloat, dev, "d_topk_w");
  int32_t* check = check_word(a[8], dev);
  // an empty scale has no address, and no row to read either
  const uint8_t none_kept = 0;
  const auto* scales = kept && M == 0 ? &none_kept : static_cast<const uint8_t*>(y_scale);
  const int rc = without_gil(dev, [&] {
    return moe_combine_backward(d_out.data_ptr(), dt, y.data_ptr(), scales, M, inv.data_ptr<int32_t>(),
                                w.data_ptr<float>(), T, static_cast<int>(k), static_cast<int>(H), d_y.data_ptr(),
                                d_w.data_ptr<float>(), check, s.raw);
  });
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return pair(wrap(d_y), wrap(d_w));
  END_HANDLE_TH_ERRORS
}

struct Weights {
  const uint8_t *codes, *scale;
};

// one of an FFN's matrices: codes [E, N, K / 2] and scale [E, N, K / 32]
Weights mx_weights(PyObject* codes, PyObject* scale, int64_t E, int64_t N, int64_t K, const at::Device& dev,
                   const char* name) {
  return {static_cast<const uint8_t*>(given(codes, {E, N, K / 2}, at::kByte, dev, name)),
          static_cast<const uint8_t*>(given(scale, {E, N, K / 32}, at::kByte, dev, name))};
}

// x, slot_off, slot_expert, n_slots, gate codes, gate scale, up codes, up scale, down codes, down scale, act, x_format,
// y_perm, workspace, stream, check, row_src
PyObject* mx_expert_ffn(PyObject*, Args a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 17);
  const at::Tensor& x = tensor(a[0]);
  const moe_dtype dt = dtype_code(x);
  on_gpu(x);
  const at::Device dev = x.device();
  TORCH_CHECK_VALUE(x.dim() == 2, "x must be [rows, H]");
  const int64_t n_src = x.size(0), H = x.size(1);
  int64_t M = n_src;
  const int32_t* row_src = nullptr;
  if (a[16] != Py_None) {
    const at::Tensor& r = tensor(a[16]);
    TORCH_CHECK_VALUE(r.dim() == 1, "row_src must be int32 [M]");
    M = r.size(0);
    row_src = static_cast<const int32_t*>(given(a[16], {M}, at::kInt, dev, "row_src"));
  }
  const at::Tensor& gate = tensor(a[4]);
  TORCH_CHECK_VALUE(gate.dim() == 3, "w_gate: expected codes [E, I, H / 2]");
  const int64_t E = gate.size(0), I = gate.size(1);
  TORCH_CHECK_VALUE(H <= INT32_MAX && I <= INT32_MAX && E <= INT32_MAX, "H, I or E out of range");
  const Weights wg = mx_weights(a[4], a[5], E, I, H, dev, "w_gate"), wu = mx_weights(a[6], a[7], E, I, H, dev, "w_up"),
                wd = mx_weights(a[8], a[9], E, H, I, dev, "w_down");
  const at::Tensor& slots = tensor(a[2]);
  const int64_t max_slots = slots.numel();
  TORCH_CHECK_VALUE(max_slots < INT32_MAX, "too many slots");
  expect(slots, {max_slots}, at::kInt, dev, "slot_expert");
  const at::Tensor& off = tensor(a[1]);
  expect(off, {max_slots + 1}, at::kInt, dev, "slot_off");
  const at::Tensor& n_slots = tensor(a[3]);
  expect(n_slots, {1}, at::kInt, dev, "n_slots");
  const int act = small(a[10]);
  const moe_mx_format fmt = format_code(a[11]);
  const Stream s = stream_of(a[14], dev);
  const at::Tensor y = output(a[12], {M, H}, x.scalar_type(), dev, "y_perm");
  const int h = static_cast<int>(H), i = static_cast<int>(I), ms = static_cast<int>(max_slots);
  const at::Tensor ws =
      workspace_of(a[13], moe_mx_expert_ffn_workspace_bytes(M, h, i, ms, fmt), dev, "FFN workspace");
  int32_t* check = check_word(a[15], dev);
  const int rc = without_gil(dev, [&] {
    return moe_mx_expert_ffn(x.data_ptr(), row_src, n_src, dt, M, h, i, static_cast<int>(E), off.data_ptr<int32_t>(),
                             slots.data_ptr<int32_t>(), n_slots.data_ptr<int32_t>(), ms, wg.codes, wg.scale, wu.codes,
                             wu.scale, wd.codes, wd.scale, static_cast<moe_act>(act), fmt, y.data_ptr(), ws.data_ptr(),
                             ws.nbytes(), check, s.raw);
  });
  return rc != MOE_OK ? PyLong_FromLong(rc) : wrap(y);
  END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(gate), METHOD(gate_backward), METHOD(layer_norm), METHOD(layer_norm_backward),
                         METHOD(clip_grads), METHOD(mx_quantize), METHOD(mx_dequantize), METHOD(combine_backward),
                         METHOD(mx_expert_ffn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }

// Python module _binding: the entry points of include/dpg.h for expert layers and
// what stands between a block's projections, for torch tensors.  It checks the
// arguments, allocates the outputs a caller does not give, and launches on the
// current stream of the tensors' device; no arithmetic.  Compiled, because the
// same work through ctypes costs about 10 us a call, and 90 us for an optimizer
// step over 48 tensors, where the kernels of one token take 2 to 6 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>
#include <vector>

#include "dpg.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // the package's DpgError

struct Status {  // a status of the C ABI on its way to DpgError
  int code;
  const char* where;
};

struct Refusal {  // a TypeError or ValueError on its way
  PyObject* type;
  std::string text;
};

[[noreturn]] void type_error(const std::string& m) { throw Refusal{PyExc_TypeError, m}; }
[[noreturn]] void value_error(const std::string& m) { throw Refusal{PyExc_ValueError, m}; }

void check_status(int code, const char* where) {
  if (code != DPG_OK) throw Status{code, where};
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const char* dtype_text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

const Tensor& input(PyObject* o, at::ScalarType dtype, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype) type_error(std::string(name) + " must be " + dtype_text(dtype));
  if (!t.is_cuda()) value_error(std::string(name) + " must be a device tensor");
  return t;
}

// BF16 or FP32 rows
const Tensor& rows_input(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    type_error(std::string(name) + " must be torch.bfloat16 or torch.float32");
  if (!t.is_cuda()) value_error(std::string(name) + " must be a device tensor");
  if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
  return t;
}

void same_device(const Tensor& first, const Tensor& t, const char* name) {
  if (t.device() != first.device())
    value_error(std::string(name) + " is on " + t.device().str() + ", expected " + first.device().str());
}

void check_shape(const Tensor& t, at::IntArrayRef shape, const char* name) {
  if (t.sizes() != shape)
    value_error(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}

// contiguous int32 or FP32 tensors
const Tensor& packed(PyObject* o, at::ScalarType dtype, const char* name) {
  const Tensor& t = input(o, dtype, name);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}

const Tensor& floats(PyObject* o, at::IntArrayRef shape, const char* name) {
  const Tensor& t = packed(o, at::kFloat, name);
  check_shape(t, shape, name);
  return t;
}

// int32 [E + 1], E where known
const Tensor& offsets_of(PyObject* o, int64_t experts) {
  const Tensor& t = packed(o, at::kInt, "offsets");
  if (t.dim() != 1 || t.size(0) < 1 || (experts >= 0 && t.size(0) != experts + 1))
    value_error("offsets must be [E + 1]" + (experts < 0 ? std::string() : " with E = " + std::to_string(experts)) +
                ", got " + shape_text(t.sizes()));
  return t;
}

const Tensor& slots_of(PyObject* o) {
  const Tensor& t = packed(o, at::kInt, "positions");
  if (t.dim() != 2 || t.size(1) < 1) value_error("positions must be [T, top_k]");
  return t;
}

// Row stride in elements.  A matrix with at most one row never steps to a next
// one: its stride is reported as the column count rounded up to 8.
int64_t row_stride(const Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
  const int64_t rows = t.size(0), cols = t.size(1);
  if (rows > 0 && cols > 1 && t.stride(1) != 1) value_error(std::string(name) + " must have unit column stride");
  return rows <= 1 ? std::max<int64_t>(8, (cols + 7) / 8 * 8) : t.stride(0);
}

// Strides of one matrix per group.
struct Groups {
  int64_t group, row;
};
Groups group_strides(const Tensor& t, const char* name) {
  const int64_t e = t.size(0), rows = t.size(1), cols = t.size(2), wide = (cols + 7) / 8 * 8;
  if (t.numel() == 0) return {rows * wide, wide};
  if (cols > 1 && t.stride(2) != 1) value_error(std::string(name) + ": the last dimension must be contiguous");
  return {e > 1 ? t.stride(0) : 0, rows > 1 ? t.stride(1) : wide};
}

at::ScalarType dtype_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) type_error("output dtype must be torch.bfloat16 or torch.float32");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

dpg_dtype code_of(at::ScalarType t) {
  if (t == at::kBFloat16) return DPG_BF16;
  if (t == at::kFloat) return DPG_F32;
  type_error("output dtype must be torch.bfloat16 or torch.float32");
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}

// Several contiguous outputs in one block of memory, each at a multiple of 16
// bytes: an allocation costs 1 us, a tensor over a part of one a tenth of that.
class Block {
 public:
  Block(int64_t bytes, const Tensor& like) : all_(fresh({bytes}, at::kByte, like)) {}
  static int64_t padded(int64_t bytes) { return (bytes + 15) & ~(int64_t)15; }
  Tensor part(at::IntArrayRef shape, at::ScalarType dtype) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all_.storage()), all_.key_set(),
                                                        c10::scalarTypeToTypeMeta(dtype));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at_ / (int64_t)t.itemsize());
    at_ += padded((int64_t)t.nbytes());
    return t;
  }

 private:
  Tensor all_;
  int64_t at_ = 0;
};

// the caller's output, checked, or a new one
Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  if (o == Py_None) {
    code_of(dtype);
    return fresh(shape, dtype, like);
  }
  const Tensor& t = tensor(o, "out");
  if (!t.is_cuda()) value_error("out must be a device tensor");
  same_device(like, t, "out");
  check_shape(t, shape, "out");
  return t;
}

hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

template <class T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// A call has written to a caller's tensor: its version goes up, as after torch's
// own in-place operations, so that a backward pass that saved it says so
// instead of computing with the new values.  Inference tensors have no version
// and are never saved.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject* given, const Tensor& out) {
  if (given != Py_None) written(out);
}

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a number");
  }
  return v;
}

// the caller's workspace, or a new one of `need` bytes (undefined for none)
Tensor workspace_of(PyObject* o, size_t need, const Tensor& like) {
  if (o == Py_None) return need > 0 ? fresh({(int64_t)need}, at::kByte, like) : Tensor();
  const Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.device() != like.device())
    value_error("workspace must be a device tensor on " + like.device().str());
  // its bytes are counted from its first one: of a view with gaps they would be
  // others' memory, of an expanded one no memory at all
  if (!t.is_contiguous()) value_error("workspace must be contiguous");
  return t;
}
void* workspace_data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t workspace_bytes(const Tensor& t) { return t.defined() ? t.nbytes() : 0; }

// ---------------------------------------------------------------- entries --
// forward (x, w), input gradient (dy, w): a, w, offsets, out, out_dtype, workspace
PyObject* grouped_rows(PyObject* const* a, bool forward) {
  const char* an = forward ? "x" : "dy";
  const Tensor& x = input(a[0], at::kBFloat16, an);
  const Tensor& w = input(a[1], at::kBFloat16, "w");
  if (x.dim() != 2) value_error(std::string(an) + " must be 2-D");
  const int64_t R = x.size(0);
  if (w.dim() != 3 || w.size(forward ? 2 : 1) != x.size(1)) value_error("w must be [E, N, K]");
  const int64_t E = w.size(0), N = w.size(1), K = w.size(2);
  const Tensor& off = offsets_of(a[2], E);
  same_device(x, w, "w");
  same_device(x, off, "offsets");
  const c10::DeviceGuard guard(x.device());
  Tensor out = output(a[3], {R, forward ? N : K}, dtype_of(a[4], at::kBFloat16), x);
  const Groups g = group_strides(w, "w");
  const Tensor ws = workspace_of(
      a[5], dpg_grouped_workspace_size(forward ? DPG_PASS_FORWARD : DPG_PASS_DGRAD, E, R, N, K), x);
  const auto fn = forward ? &dpg_grouped_forward : &dpg_grouped_dgrad;
  check_status(fn(x.data_ptr(), row_stride(x, an), w.data_ptr(), g.row, g.group, out.data_ptr(),
                  row_stride(out, "out"), code_of(out.scalar_type()), data<int32_t>(off), E, R, N, K,
                  workspace_data(ws), workspace_bytes(ws), stream_of(x)),
               forward ? "dpg_grouped_forward" : "dpg_grouped_dgrad");
  written(a[3], out);
  return wrap(std::move(out));
}
PyObject* grouped_forward(PyObject* const* a) { return grouped_rows(a, true); }
PyObject* grouped_dgrad(PyObject* const* a) { return grouped_rows(a, false); }

// dy, x, offsets, out, out_dtype, workspace
PyObject* grouped_wgrad(PyObject* const* a) {
  const Tensor& dy = input(a[0], at::kBFloat16, "dy");
  const Tensor& x = input(a[1], at::kBFloat16, "x");
  if (dy.dim() != 2) value_error("dy must be 2-D");
  if (x.dim() != 2 || x.size(0) != dy.size(0)) value_error("x must be [R, K]");
  const Tensor& off = offsets_of(a[2], -1);
  const int64_t E = off.size(0) - 1, R = dy.size(0), N = dy.size(1), K = x.size(1);
  same_device(dy, x, "x");
  same_device(dy, off, "offsets");
  const c10::DeviceGuard guard(dy.device());
  Tensor out = output(a[3], {E, N, K}, dtype_of(a[4], at::kBFloat16), dy);
  const Groups g = group_strides(out, "out");
  const Tensor ws = workspace_of(a[5], dpg_grouped_workspace_size(DPG_PASS_WGRAD, E, R, N, K), dy);
  check_status(dpg_grouped_wgrad(dy.data_ptr(), row_stride(dy, "dy"), x.data_ptr(), row_stride(x, "x"),
                                 out.data_ptr(), g.row, g.group, code_of(out.scalar_type()), data<int32_t>(off), E, R,
                                 N, K, workspace_data(ws), workspace_bytes(ws), stream_of(dy)),
               "dpg_grouped_wgrad");
  written(a[3], out);
  return wrap(std::move(out));
}

struct Logits {
  int64_t T, E, ld;
};
Logits logits_of(const Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
  const int64_t T = t.size(0), E = t.size(1);
  if (E > 1 && T > 0 && t.stride(1) != 1) value_error(std::string(name) + " must have unit column stride");
  return {T, E, T > 1 ? t.stride(0) : E};
}

// logits, top_k, renormalize, workspace
PyObject* route(PyObject* const* a) {
  const Tensor& logits = input(a[0], at::kFloat, "logits");
  const Logits l = logits_of(logits, "logits");
  const int64_t k = integer(a[1], "top_k");
  const int renorm = PyObject_IsTrue(a[2]);
  if (renorm < 0) {
    PyErr_Clear();
    type_error("renormalize must be a truth value");
  }
  const size_t need = dpg_route_workspace_size(l.T, l.E, k);
  if (need == (size_t)-1) throw Status{1 <= k && k <= l.E ? DPG_ERR_UNSUPPORTED : DPG_ERR_INVALID_ARG, "dpg_route"};
  const c10::DeviceGuard guard(logits.device());
  const Tensor ws = workspace_of(a[3], need, logits);
  const int64_t n = l.T * k;
  Block block(4 * Block::padded(4 * n) + Block::padded(4 * (l.E + 1)), logits);
  Tensor experts = block.part({l.T, k}, at::kInt), weights = block.part({l.T, k}, at::kFloat);
  Tensor offsets = block.part({l.E + 1}, at::kInt), rows = block.part({n}, at::kInt);
  Tensor positions = block.part({l.T, k}, at::kInt);
  check_status(dpg_route(data<float>(logits), l.ld, l.T, l.E, k, renorm, data<int32_t>(experts), data<float>(weights),
                         data<int32_t>(offsets), data<int32_t>(rows), data<int32_t>(positions),
                         workspace_data(ws), workspace_bytes(ws), stream_of(logits)),
               "dpg_route");
  PyObject* r = PyTuple_New(5);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(std::move(experts)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(weights)));
  PyTuple_SET_ITEM(r, 2, wrap(std::move(offsets)));
  PyTuple_SET_ITEM(r, 3, wrap(std::move(rows)));
  PyTuple_SET_ITEM(r, 4, wrap(std::move(positions)));
  return r;
}

// logits, experts, weights, dweights, renormalize, out
PyObject* route_dgrad(PyObject* const* a) {
  const Tensor& logits = input(a[0], at::kFloat, "logits");
  const Logits l = logits_of(logits, "logits");
  const Tensor& experts = packed(a[1], at::kInt, "experts");
  if (experts.dim() != 2 || experts.size(0) != l.T) value_error("experts must be [T, top_k]");
  const int64_t k = experts.size(1);
  const Tensor& weights = floats(a[2], {l.T, k}, "weights");
  const Tensor& dweights = floats(a[3], {l.T, k}, "dweights");
  same_device(logits, experts, "experts");
  same_device(logits, weights, "weights");
  same_device(logits, dweights, "dweights");
  const int renorm = PyObject_IsTrue(a[4]);
  if (renorm < 0) {
    PyErr_Clear();
    type_error("renormalize must be a truth value");
  }
  const c10::DeviceGuard guard(logits.device());
  Tensor out = output(a[5], {l.T, l.E}, at::kFloat, logits);
  if (out.scalar_type() != at::kFloat) type_error("out must be torch.float32");
  const Logits o = logits_of(out, "out");
  check_status(dpg_route_dgrad(data<float>(logits), l.ld, data<int32_t>(experts), data<float>(weights),
                               data<float>(dweights), data<float>(out), o.ld, l.T, l.E, k, renorm,
                               stream_of(logits)),
               "dpg_route_dgrad");
  written(a[5], out);
  return wrap(std::move(out));
}

// x, positions, offsets, out
PyObject* dispatch(PyObject* const* a) {
  const Tensor& x = rows_input(a[0], "x");
  const Tensor& pos = slots_of(a[1]);
  const int64_t T = pos.size(0), k = pos.size(1);
  if (x.size(0) != T) value_error("x must be [T, H]");
  const int64_t H = x.size(1);
  const Tensor& off = offsets_of(a[2], -1);
  same_device(x, pos, "positions");
  same_device(x, off, "offsets");
  const c10::DeviceGuard guard(x.device());
  Tensor out = output(a[3], {T * k, H}, x.scalar_type(), x);
  if (out.scalar_type() != x.scalar_type()) type_error(std::string("out must be ") + dtype_text(x.scalar_type()));
  check_status(dpg_dispatch(x.data_ptr(), row_stride(x, "x"), data<int32_t>(pos), data<int32_t>(off), out.data_ptr(),
                            row_stride(out, "out"), code_of(x.scalar_type()), T, T * k, H, off.size(0) - 1, k,
                            stream_of(x)),
               "dpg_dispatch");
  written(a[3], out);
  return wrap(std::move(out));
}

// ys, positions, offsets, weights, out, out_dtype
PyObject* combine(PyObject* const* a) {
  const Tensor& ys = rows_input(a[0], "ys");
  const Tensor& pos = slots_of(a[1]);
  const int64_t T = pos.size(0), k = pos.size(1), R = ys.size(0), H = ys.size(1);
  if (R != T * k) value_error("ys must be [T * top_k, H]");
  const Tensor& off = offsets_of(a[2], -1);
  same_device(ys, pos, "positions");
  same_device(ys, off, "offsets");
  const float* w = nullptr;
  if (a[3] != Py_None) {
    const Tensor& weights = floats(a[3], {T, k}, "weights");
    same_device(ys, weights, "weights");
    w = data<float>(weights);
  }
  const c10::DeviceGuard guard(ys.device());
  Tensor out = output(a[4], {T, H}, dtype_of(a[5], ys.scalar_type()), ys);
  check_status(dpg_combine(ys.data_ptr(), row_stride(ys, "ys"), code_of(ys.scalar_type()), data<int32_t>(pos),
                           data<int32_t>(off), w, out.data_ptr(), row_stride(out, "out"), code_of(out.scalar_type()),
                           T, R, H, off.size(0) - 1, k, stream_of(ys)),
               "dpg_combine");
  written(a[4], out);
  return wrap(std::move(out));
}

// dy, ys, positions, offsets, weights
PyObject* combine_dgrad(PyObject* const* a) {
  const Tensor& dy = rows_input(a[0], "dy");
  const Tensor& ys = input(a[1], dy.scalar_type(), "ys");
  const Tensor& pos = slots_of(a[2]);
  const int64_t T = pos.size(0), k = pos.size(1), H = dy.size(1);
  if (dy.size(0) != T || ys.dim() != 2 || ys.size(0) != T * k || ys.size(1) != H)
    value_error("dy must be [T, H] and ys [T * top_k, H]");
  const Tensor& off = offsets_of(a[3], -1);
  const Tensor& weights = floats(a[4], {T, k}, "weights");
  same_device(dy, ys, "ys");
  same_device(dy, pos, "positions");
  same_device(dy, off, "offsets");
  same_device(dy, weights, "weights");
  const c10::DeviceGuard guard(dy.device());
  Tensor dys = fresh({T * k, H}, ys.scalar_type(), dy), dweights = fresh({T, k}, at::kFloat, dy);
  check_status(dpg_combine_dgrad(dy.data_ptr(), row_stride(dy, "dy"), ys.data_ptr(), row_stride(ys, "ys"),
                                 data<int32_t>(pos), data<int32_t>(off), data<float>(weights), dys.data_ptr(),
                                 row_stride(dys, "dys"), data<float>(dweights), code_of(dy.scalar_type()), T, T * k,
                                 H, off.size(0) - 1, k, stream_of(dy)),
               "dpg_combine_dgrad");
  return Py_BuildValue("(NN)", wrap(std::move(dys)), wrap(std::move(dweights)));
}

// One list of an optimizer step: contiguous tensors of one type, with the
// parameters' sizes (or their blocks' count).
class Column {
 public:
  Column(PyObject* list, const char* name) : name_(name) {
    if (list == Py_None) return;
    seq_ = PySequence_Fast(list, "");
    if (!seq_) {
      PyErr_Clear();
      type_error(std::string(name) + " must be a list of tensors");
    }
  }
  ~Column() { Py_XDECREF(seq_); }
  Column(const Column&) = delete;
  Column& operator=(const Column&) = delete;
  bool given() const { return seq_ != nullptr; }
  int64_t size() const { return seq_ ? PySequence_Fast_GET_SIZE(seq_) : 0; }
  const Tensor& at(int64_t i) const { return tensor(PySequence_Fast_GET_ITEM(seq_, i), name_); }
  void check_size(int64_t n) const {
    if (seq_ && size() != n) value_error(std::string(name_) + " must hold one tensor per parameter");
  }
  // the data of tensor i; one that the step writes is added to `outputs`
  void* pointer(int64_t i, at::ScalarType dtype, at::Device device, int64_t numel,
                std::vector<c10::TensorImpl*>* outputs = nullptr) const {
    if (!seq_) return nullptr;
    const Tensor& t = at(i);
    if (outputs) outputs->push_back(t.unsafeGetTensorImpl());
    if (t.scalar_type() != dtype) type_error(std::string(name_) + " must be " + dtype_text(dtype));
    if (t.device() != device) {
      if (!t.is_cuda()) value_error(std::string(name_) + " must be device tensors");
      value_error(std::string(name_) + " is on " + t.device().str() + ", expected " + device.str());
    }
    if (t.numel() != numel)
      value_error(std::string(name_) + ": " + std::to_string(t.numel()) + " elements, expected " +
                  std::to_string(numel));
    if (!t.is_contiguous()) value_error(std::string(name_) + " must be contiguous");
    return t.data_ptr();
  }

 private:
  PyObject* seq_ = nullptr;
  const char* name_;
};

constexpr int64_t kScaleBlock = 256;  // elements that share one scale of an 8-bit moment

// params, grads, exp_avgs, exp_avg_sqs, copies, avg_scales, sq_scales,
// grad_scale, lr, beta1, beta2, eps, weight_decay, step, seed
PyObject* adamw(PyObject* const* a) {
  const Column params(a[0], "params"), grads(a[1], "grads"), avgs(a[2], "exp_avgs"), sqs(a[3], "exp_avg_sqs");
  const Column copies(a[4], "copies"), avg_scales(a[5], "avg_scales"), sq_scales(a[6], "sq_scales");
  const int64_t n = params.size();
  if (n == 0) Py_RETURN_NONE;
  const Tensor first = params.at(0);
  if (!first.is_cuda()) value_error("params must be device tensors");
  for (const Column* c : {&grads, &avgs, &sqs}) {
    if (!c->given() || c->size() != n) value_error("grads, exp_avgs and exp_avg_sqs must hold one tensor per parameter");
  }
  for (const Column* c : {&copies, &avg_scales, &sq_scales}) c->check_size(n);
  const at::ScalarType grad = grads.at(0).scalar_type(), state = avgs.at(0).scalar_type();
  const bool e4m3 = state == at::kFloat8_e4m3fn;
  if (!e4m3 && state != at::kFloat) type_error("moments must be torch.float32 or torch.float8_e4m3fn");
  if (grad != at::kFloat && grad != at::kBFloat16) type_error("grads must be torch.bfloat16 or torch.float32");
  if (e4m3 && (!avg_scales.given() || !sq_scales.given())) value_error("8-bit moments need avg_scales and sq_scales");
  // numbers first: reading one may run Python code, and from here on tensors are held by address
  dpg_adamw_options o{};
  o.lr = number(a[8], "lr");
  o.beta1 = number(a[9], "beta1");
  o.beta2 = number(a[10], "beta2");
  o.eps = number(a[11], "eps");
  o.weight_decay = number(a[12], "weight_decay");
  o.step = integer(a[13], "step");
  o.seed = (uint32_t)integer(a[14], "seed");
  std::vector<dpg_adamw_tensor> table(n);
  std::vector<c10::TensorImpl*> outputs;
  outputs.reserve(6 * n);
  const at::Device device = first.device();
  for (int64_t i = 0; i < n; ++i) {
    const Tensor& p = params.at(i);
    const int64_t numel = p.numel(), blocks = (numel + kScaleBlock - 1) / kScaleBlock;
    dpg_adamw_tensor& t = table[i];
    t.param = (float*)params.pointer(i, at::kFloat, device, numel, &outputs);
    t.grad = grads.pointer(i, grad, device, numel);
    t.exp_avg = avgs.pointer(i, state, device, numel, &outputs);
    t.exp_avg_sq = sqs.pointer(i, state, device, numel, &outputs);
    t.avg_scale = e4m3 ? (float*)avg_scales.pointer(i, at::kFloat, device, blocks, &outputs) : nullptr;
    t.sq_scale = e4m3 ? (float*)sq_scales.pointer(i, at::kFloat, device, blocks, &outputs) : nullptr;
    t.copy = copies.pointer(i, at::kBFloat16, device, numel, &outputs);
    t.numel = numel;
  }
  if (a[7] != Py_None) {
    const Tensor& s = packed(a[7], at::kFloat, "grad_scale");
    if (s.numel() != 1) value_error("grad_scale must hold one value");
    same_device(first, s, "grad_scale");
    o.grad_scale = data<float>(s);
  }
  o.grad_dtype = grad == at::kFloat ? DPG_F32 : DPG_BF16;
  o.state_dtype = e4m3 ? DPG_E4M3 : DPG_F32;
  const c10::DeviceGuard guard(first.device());
  check_status(dpg_adamw(table.data(), n, &o, stream_of(first)), "dpg_adamw");
  for (c10::TensorImpl* t : outputs)
    if (!t->is_inference()) t->bump_version();
  Py_RETURN_NONE;
}

// ------------------------------------- between the projections of a block --
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a truth value");
  }
  return v != 0;
}

// p, seed and step of a dropout
dpg_dropout_options dropout_of(PyObject* const* a, const Tensor& like) {
  dpg_dropout_options o{};
  o.p = number(a[0], "p");
  o.seed = PyLong_AsUnsignedLongLongMask(a[1]);
  if (o.seed == (uint64_t)-1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("seed must be an integer");
  }
  if (a[2] != Py_None) {
    const Tensor& step = packed(a[2], at::kLong, "step");
    if (step.numel() != 1) value_error("step must hold one value");
    same_device(like, step, "step");
    o.step = data<int64_t>(step);
  }
  return o;
}

// FP32 [n], or null for None
float* columns_of(PyObject* o, int64_t n, const Tensor& like, const char* name) {
  if (o == Py_None) return nullptr;
  const Tensor& t = floats(o, {n}, name);
  same_device(like, t, name);
  return data<float>(t);
}

void check_kind(const Tensor& t, at::ScalarType dtype, const char* name) {
  if (t.scalar_type() != dtype) type_error(std::string(name) + " must be " + dtype_text(dtype));
}

// x, p, seed, step, residual, out, out_dtype
PyObject* dropout(PyObject* const* a) {
  const Tensor& x = rows_input(a[0], "x");
  const int64_t T = x.size(0), H = x.size(1);
  const dpg_dropout_options o = dropout_of(a + 1, x);
  at::ScalarType kind = x.scalar_type();
  const void* r = nullptr;
  int64_t ldr = 0;
  if (a[4] != Py_None) {
    const Tensor& residual = rows_input(a[4], "residual");
    check_shape(residual, {T, H}, "residual");
    same_device(x, residual, "residual");
    kind = residual.scalar_type();
    r = residual.data_ptr();
    ldr = row_stride(residual, "residual");
  }
  const c10::DeviceGuard guard(x.device());
  Tensor out = output(a[5], {T, H}, dtype_of(a[6], kind), x);
  if (r) check_kind(out, kind, "out");
  check_status(dpg_dropout(x.data_ptr(), row_stride(x, "x"), code_of(x.scalar_type()), T > 0 && H > 0 ? r : nullptr, ldr,
                           out.data_ptr(), row_stride(out, "out"), code_of(out.scalar_type()), T, H, &o, stream_of(x)),
               "dpg_dropout");
  written(a[5], out);
  return wrap(std::move(out));
}

// x, weight, bias, eps, out, out_dtype
PyObject* layer_norm(PyObject* const* a) {
  const Tensor& x = rows_input(a[0], "x");
  const int64_t T = x.size(0), H = x.size(1);
  const float *w = columns_of(a[1], H, x, "weight"), *b = columns_of(a[2], H, x, "bias");
  const double eps = number(a[3], "eps");
  const c10::DeviceGuard guard(x.device());
  Tensor out = output(a[4], {T, H}, dtype_of(a[5], x.scalar_type()), x);
  Block block(2 * Block::padded(4 * T), x);
  Tensor mean = block.part({T}, at::kFloat), rstd = block.part({T}, at::kFloat);
  check_status(dpg_layer_norm(x.data_ptr(), row_stride(x, "x"), code_of(x.scalar_type()), w, b, out.data_ptr(),
                              row_stride(out, "out"), code_of(out.scalar_type()), data<float>(mean), data<float>(rstd),
                              T, H, eps, stream_of(x)),
               "dpg_layer_norm");
  written(a[4], out);
  return Py_BuildValue("(NNN)", wrap(std::move(out)), wrap(std::move(mean)), wrap(std::move(rstd)));
}

// x, residual, weight, bias, eps, p, seed, step, out, sum, out_dtype
PyObject* add_layer_norm(PyObject* const* a) {
  const Tensor& x = rows_input(a[0], "x");
  const int64_t T = x.size(0), H = x.size(1);
  const Tensor& residual = rows_input(a[1], "residual");
  check_shape(residual, {T, H}, "residual");
  same_device(x, residual, "residual");
  const float *w = columns_of(a[2], H, x, "weight"), *b = columns_of(a[3], H, x, "bias");
  const double eps = number(a[4], "eps");
  const dpg_dropout_options o = dropout_of(a + 5, x);
  const c10::DeviceGuard guard(x.device());
  Tensor out = output(a[8], {T, H}, dtype_of(a[10], x.scalar_type()), x);
  Tensor sum = output(a[9], {T, H}, residual.scalar_type(), x);
  check_kind(sum, residual.scalar_type(), "sum");
  Block block(2 * Block::padded(4 * T), x);
  Tensor mean = block.part({T}, at::kFloat), rstd = block.part({T}, at::kFloat);
  check_status(dpg_add_layer_norm(x.data_ptr(), row_stride(x, "x"), code_of(x.scalar_type()), residual.data_ptr(),
                                  row_stride(residual, "residual"), sum.data_ptr(), row_stride(sum, "sum"),
                                  code_of(sum.scalar_type()), w, b, out.data_ptr(), row_stride(out, "out"),
                                  code_of(out.scalar_type()), data<float>(mean), data<float>(rstd), T, H, eps, &o,
                                  stream_of(x)),
               "dpg_add_layer_norm");
  written(a[8], out);
  written(a[9], sum);
  return Py_BuildValue("(NNNN)", wrap(std::move(out)), wrap(std::move(mean)), wrap(std::move(rstd)),
                       wrap(std::move(sum)));
}

// The gradients of weight and bias, and the workspace that their sums go through.
struct WeightGrads {
  Tensor dweight, dbias, workspace;
  WeightGrads(bool wanted, int64_t T, int64_t H, PyObject* given, const Tensor& like) {
    if (!wanted) return;
    Block block(2 * Block::padded(4 * H), like);
    dweight = block.part({H}, at::kFloat);
    dbias = block.part({H}, at::kFloat);
    const size_t need = dpg_layer_norm_workspace_size(T, H);
    if (need != (size_t)-1) workspace = workspace_of(given, need, like);
  }
  static float* at(const Tensor& t) { return t.defined() ? data<float>(t) : nullptr; }
  static PyObject* object(Tensor& t) {
    if (t.defined()) return wrap(std::move(t));
    Py_RETURN_NONE;
  }
};

// dy, x, mean, rstd, weight, weight_grads, workspace
PyObject* layer_norm_dgrad(PyObject* const* a) {
  const Tensor& dy = rows_input(a[0], "dy");
  const int64_t T = dy.size(0), H = dy.size(1);
  const Tensor& x = rows_input(a[1], "x");
  check_shape(x, {T, H}, "x");
  same_device(dy, x, "x");
  const Tensor &mean = floats(a[2], {T}, "mean"), &rstd = floats(a[3], {T}, "rstd");
  same_device(dy, mean, "mean");
  same_device(dy, rstd, "rstd");
  const float* w = columns_of(a[4], H, dy, "weight");
  const bool wanted = truth(a[5], "weight_grads");
  const c10::DeviceGuard guard(dy.device());
  Tensor dx = fresh({T, H}, x.scalar_type(), dy);
  WeightGrads g(wanted, T, H, a[6], dy);
  check_status(dpg_layer_norm_dgrad(dy.data_ptr(), row_stride(dy, "dy"), code_of(dy.scalar_type()), x.data_ptr(),
                                    row_stride(x, "x"), code_of(x.scalar_type()), data<float>(mean), data<float>(rstd),
                                    w, dx.data_ptr(), row_stride(dx, "dx"), g.at(g.dweight), g.at(g.dbias), T, H,
                                    workspace_data(g.workspace), workspace_bytes(g.workspace), stream_of(dy)),
               "dpg_layer_norm_dgrad");
  return Py_BuildValue("(NNN)", wrap(std::move(dx)), g.object(g.dweight), g.object(g.dbias));
}

// dy, sum, mean, rstd, weight, dsum, p, seed, step, x_dtype, weight_grads, workspace
PyObject* add_layer_norm_dgrad(PyObject* const* a) {
  const Tensor& dy = rows_input(a[0], "dy");
  const int64_t T = dy.size(0), H = dy.size(1);
  const Tensor& sum = rows_input(a[1], "sum");
  check_shape(sum, {T, H}, "sum");
  same_device(dy, sum, "sum");
  const Tensor &mean = floats(a[2], {T}, "mean"), &rstd = floats(a[3], {T}, "rstd");
  same_device(dy, mean, "mean");
  same_device(dy, rstd, "rstd");
  const float* w = columns_of(a[4], H, dy, "weight");
  const void* more = nullptr;
  int64_t ldm = 0;
  if (a[5] != Py_None) {
    const Tensor& dsum = rows_input(a[5], "dsum");
    check_shape(dsum, {T, H}, "dsum");
    check_kind(dsum, sum.scalar_type(), "dsum");
    same_device(dy, dsum, "dsum");
    more = T > 0 && H > 0 ? dsum.data_ptr() : nullptr;
    ldm = row_stride(dsum, "dsum");
  }
  const dpg_dropout_options o = dropout_of(a + 6, dy);
  const at::ScalarType kind = dtype_of(a[9], dy.scalar_type());
  const bool wanted = truth(a[10], "weight_grads");
  const c10::DeviceGuard guard(dy.device());
  code_of(kind);
  Tensor dx = fresh({T, H}, kind, dy), dres = fresh({T, H}, sum.scalar_type(), dy);
  WeightGrads g(wanted, T, H, a[11], dy);
  check_status(dpg_add_layer_norm_dgrad(dy.data_ptr(), row_stride(dy, "dy"), code_of(dy.scalar_type()), sum.data_ptr(),
                                        row_stride(sum, "sum"), code_of(sum.scalar_type()), data<float>(mean),
                                        data<float>(rstd), w, more, ldm, dx.data_ptr(), row_stride(dx, "dx"),
                                        code_of(kind), dres.data_ptr(), row_stride(dres, "dresidual"),
                                        g.at(g.dweight), g.at(g.dbias), T, H, &o, workspace_data(g.workspace),
                                        workspace_bytes(g.workspace), stream_of(dy)),
               "dpg_add_layer_norm_dgrad");
  return Py_BuildValue("(NNNN)", wrap(std::move(dx)), wrap(std::move(dres)), g.object(g.dweight), g.object(g.dbias));
}

// Sequences of a recurrence: x is [B, T, D], or [R, D] with offsets [S + 1].
struct Sequences {
  int64_t S, R, D;
  const int32_t* offsets;
  at::ScalarType kind;
  Sequences(const Tensor& x, PyObject* off) : offsets(nullptr), kind(x.scalar_type()) {
    if (off == Py_None) {
      if (x.dim() != 3) value_error("x must be [B, T, D], or [R, D] with offsets");
      S = x.size(0);
      R = S * x.size(1);
      D = x.size(2);
    } else {
      if (x.dim() != 2) value_error("x must be [R, D] with offsets");
      const Tensor& t = offsets_of(off, -1);
      same_device(x, t, "offsets");
      S = t.size(0) - 1;
      R = x.size(0);
      D = x.size(1);
      offsets = data<int32_t>(t);
    }
  }
};

const Tensor& sequence_input(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    type_error(std::string(name) + " must be torch.bfloat16 or torch.float32");
  if (!t.is_cuda()) value_error(std::string(name) + " must be a device tensor");
  return t;
}
const Tensor& sequence_like(PyObject* o, const Tensor& x, const char* name) {
  const Tensor& t = sequence_input(o, name);
  check_kind(t, x.scalar_type(), name);
  check_shape(t, x.sizes(), name);
  same_device(x, t, name);
  return t;
}

// One stride between all rows, those of one sequence and of the next.
int64_t sequence_stride(const Tensor& t, const char* name) {
  if (t.dim() == 2) return row_stride(t, name);
  const int64_t b = t.size(0), n = t.size(1), d = t.size(2), wide = std::max<int64_t>(8, (d + 7) / 8 * 8);
  if (t.numel() == 0) return wide;
  if (d > 1 && t.stride(2) != 1) value_error(std::string(name) + ": the last dimension must be contiguous");
  if (n == 1) return b > 1 ? t.stride(0) : wide;
  if (b > 1 && t.stride(0) != n * t.stride(1))
    value_error(std::string(name) + ": sequences must follow each other at the stride of their rows");
  return t.stride(1);
}

// x, gate, offsets, state, coupled, carries, out, state_out, workspace
PyObject* recurrence(PyObject* const* a) {
  const Tensor& x = sequence_input(a[0], "x");
  const Sequences q(x, a[2]);
  const Tensor& gate = sequence_like(a[1], x, "gate");
  const float* state = nullptr;
  if (a[3] != Py_None) {
    const Tensor& t = floats(a[3], {q.S, q.D}, "state");
    same_device(x, t, "state");
    state = data<float>(t);
  }
  const bool coupled = truth(a[4], "coupled"), keep = truth(a[5], "carries");
  const c10::DeviceGuard guard(x.device());
  Tensor out = output(a[6], x.sizes(), q.kind, x);
  check_kind(out, q.kind, "out");
  Tensor last;
  if (a[7] == Py_None) {
    last = fresh({q.S, q.D}, at::kFloat, x);
  } else {
    last = floats(a[7], {q.S, q.D}, "state_out");
    same_device(x, last, "state_out");
  }
  const int packed_rows = q.offsets != nullptr;
  const dpg_dtype kind = code_of(q.kind);
  const size_t need = dpg_recurrence_workspace_size(q.S, q.R, q.D, kind, packed_rows);
  const size_t carry = dpg_recurrence_carries_size(q.S, q.R, q.D, kind, packed_rows);
  if (need == (size_t)-1) throw Status{DPG_ERR_UNSUPPORTED, "dpg_recurrence"};
  const Tensor ws = workspace_of(a[8], need, x);
  Tensor carries;
  if (keep) carries = fresh({(int64_t)(carry / 4)}, at::kFloat, x);
  check_status(dpg_recurrence(gate.data_ptr(), sequence_stride(gate, "gate"), x.data_ptr(), sequence_stride(x, "x"),
                              out.data_ptr(), sequence_stride(out, "out"), kind, state, data<float>(last),
                              carries.defined() ? data<float>(carries) : nullptr, q.offsets, q.S, q.R, q.D, coupled,
                              workspace_data(ws), workspace_bytes(ws), stream_of(x)),
               "dpg_recurrence");
  written(a[6], out);
  written(a[7], last);
  return Py_BuildValue("(NNN)", wrap(std::move(out)), wrap(std::move(last)), WeightGrads::object(carries));
}

// dh, gate, x, carries, offsets, state, dstate, coupled, workspace
PyObject* recurrence_dgrad(PyObject* const* a) {
  const Tensor& x = sequence_input(a[2], "x");
  const Sequences q(x, a[4]);
  const Tensor &gate = sequence_like(a[1], x, "gate"), &dh = sequence_like(a[0], x, "dh");
  const int packed_rows = q.offsets != nullptr;
  const dpg_dtype kind = code_of(q.kind);
  const size_t need = dpg_recurrence_workspace_size(q.S, q.R, q.D, kind, packed_rows);
  const size_t carry = dpg_recurrence_carries_size(q.S, q.R, q.D, kind, packed_rows);
  if (need == (size_t)-1) throw Status{DPG_ERR_UNSUPPORTED, "dpg_recurrence_dgrad"};
  const Tensor& carries = floats(a[3], {(int64_t)(carry / 4)}, "carries");
  same_device(x, carries, "carries");
  const float* states[2] = {nullptr, nullptr};
  const char* const names[2] = {"state", "dstate"};
  for (int i = 0; i < 2; ++i) {
    if (a[5 + i] == Py_None) continue;
    const Tensor& t = floats(a[5 + i], {q.S, q.D}, names[i]);
    same_device(x, t, names[i]);
    states[i] = data<float>(t);
  }
  const bool coupled = truth(a[7], "coupled");
  const c10::DeviceGuard guard(x.device());
  const Tensor ws = workspace_of(a[8], need, x);
  Tensor dgate = fresh(x.sizes(), q.kind, x), dx = fresh(x.sizes(), q.kind, x), first;
  if (states[0]) first = fresh({q.S, q.D}, at::kFloat, x);
  check_status(dpg_recurrence_dgrad(dh.data_ptr(), sequence_stride(dh, "dh"), gate.data_ptr(),
                                    sequence_stride(gate, "gate"), x.data_ptr(), sequence_stride(x, "x"),
                                    data<float>(carries), states[0], states[1], dgate.data_ptr(),
                                    sequence_stride(dgate, "dgate"), dx.data_ptr(), sequence_stride(dx, "dx"),
                                    first.defined() ? data<float>(first) : nullptr, kind, q.offsets, q.S, q.R, q.D,
                                    coupled, workspace_data(ws), workspace_bytes(ws), stream_of(x)),
               "dpg_recurrence_dgrad");
  return Py_BuildValue("(NNN)", wrap(std::move(dgate)), wrap(std::move(dx)), WeightGrads::object(first));
}

// Entry with a fixed number of positional arguments; C++ exceptions end here.
template <PyObject* (*FN)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return FN(args);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  } catch (const Status& s) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", s.code, s.where) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s: status %d", s.where, s.code);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))&entry<&name, n>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(grouped_forward, 6),
                           ENTRY(grouped_dgrad, 6),
                           ENTRY(grouped_wgrad, 6),
                           ENTRY(route, 4),
                           ENTRY(route_dgrad, 6),
                           ENTRY(dispatch, 4),
                           ENTRY(combine, 6),
                           ENTRY(combine_dgrad, 5),
                           ENTRY(adamw, 15),
                           ENTRY(dropout, 7),
                           ENTRY(layer_norm, 6),
                           ENTRY(add_layer_norm, 11),
                           ENTRY(layer_norm_dgrad, 7),
                           ENTRY(add_layer_norm_dgrad, 12),
                           ENTRY(recurrence, 9),
                           ENTRY(recurrence_dgrad, 9),
                           {"set_error", &set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) {
  return PyModule_Create(&g_module);
}

// Python entry points of the operators of include/block_ops.h: checks of tensors, output
// allocation and the call of the C ABI, in C++ because a call on a few tokens lasts as long as
// its host side (marshalling in Python took 20-28 us a call, this takes about 6).
//
// Plain CPython functions over positional arguments; the Python modules norm_quant, rope and
// linear hold the signatures and the documentation.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <utility>
#include <vector>

#include "../../../include/block_ops.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // FusedNormError

// Thrown once the Python error is set.
struct Raised {};
template <typename... A>
Raised TypeError(const char* format, A... a) {
  PyErr_Format(PyExc_TypeError, format, a...);
  return Raised();
}
template <typename... A>
Raised ValueError(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  return Raised();
}

void check_status(fn_status s, const char* what) {
  if (s == FN_OK) return;
  std::string detail = block_ops_status_string(s);
  if (s == FN_ERR_CUDA) {
    const int e = block_ops_last_cuda_error();
    detail += " (cudaError " + std::to_string(e) + ")";
    if (e == cudaErrorLaunchTimeout) detail += ": a wait of an earlier linear_gate_residual ran out, its output is incomplete";
  }
  PyObject* e = PyObject_CallFunction(g_error, "iss", (int)s, what, detail.c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// ---- arguments -------------------------------------------------------------------------------

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kHalf: return "float16";
    case at::kFloat: return "float32";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    default: return c10::toString(t);
  }
}
std::string shape_of(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}
int code_of(at::ScalarType t) { return t == at::kBFloat16 ? BO_BF16 : t == at::kHalf ? BO_FP16 : BO_E4M3; }

const Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw TypeError("%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}
void on_device(const Tensor& t, const char* name, const at::Device& device) {
  if (t.device() != device)
    throw ValueError("%s is on %s, expected %s", name, t.device().str().c_str(), device.str().c_str());
}
// dtype, device and contiguous channels
void check_tensor(const Tensor& t, const char* name, const at::Device& device, at::ScalarType dtype) {
  if (t.scalar_type() != dtype) throw TypeError("%s must be %s, got %s", name, name_of(dtype), name_of(t.scalar_type()));
  on_device(t, name, device);
  if (t.dim() >= 1 && t.size(-1) > 1 && t.stride(-1) != 1) throw ValueError("%s needs a contiguous channel dimension", name);
}
void check_shape(const Tensor& t, const char* name, c10::IntArrayRef shape, at::ScalarType dtype, const at::Device& device) {
  if (t.scalar_type() != dtype || t.sizes() != shape || t.device() != device)
    throw ValueError("%s must be a %s tensor of shape %s on %s", name, name_of(dtype), shape_of(shape).c_str(), device.str().c_str());
}
// Of a (B, L, D) tensor. The stride along an extent of 1 means nothing (PyTorch leaves any there).
fn_operand rows_of(const Tensor& t) {
  return fn_operand{t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, 0, t.size(1) > 1 ? t.stride(1) : 0};
}

// A gate, scale or shift for x of (B, L, D); *frames is the frame count the call has so far.
fn_operand operand_of(const Tensor& t, const char* name, int64_t B, int64_t L, int64_t D, at::ScalarType dtype,
                      const at::Device& device, int64_t* frames) {
  check_tensor(t, name, device, dtype);
  const int64_t dim = t.dim();
  if (dim < 1 || dim > 4) throw ValueError("%s has unsupported rank %d", name, (int)dim);
  if (t.size(-1) != D) throw ValueError("%s has %lld channels, expected %lld", name, (long long)t.size(-1), (long long)D);
  fn_operand o{t.data_ptr(), 0, 0, 0};
  const auto s = t.sizes();
  bool ok = true;
  if (dim == 2) {
    ok = s[0] == 1 || s[0] == B;
    if (s[0] > 1) o.stride_b = t.stride(0);
  } else if (dim == 3) {
    ok = (s[0] == 1 || s[0] == B) && (s[1] == 1 || s[1] == L);
    if (s[0] > 1) o.stride_b = t.stride(0);
    if (s[1] > 1) o.stride_l = t.stride(1);
  } else if (dim == 4) {
    const int64_t F = s[1];
    if ((s[0] != 1 && s[0] != B) || s[2] != 1 || F < 1 || L % F != 0)
      throw ValueError("%s of shape %s is not a (B, F, 1, D) frame operand for L=%lld", name, shape_of(s).c_str(), (long long)L);
    if (s[0] > 1) o.stride_b = t.stride(0);
    if (F > 1) o.stride_f = t.stride(1);
    if (*frames && *frames != F)
      throw ValueError("operands disagree on the frame count: %lld and %lld", (long long)*frames, (long long)F);
    *frames = F;
  }
  if (!ok)
    throw ValueError("%s of shape %s does not broadcast against (%lld, %lld, %lld)", name, shape_of(s).c_str(), (long long)B,
                     (long long)L, (long long)D);
  return o;
}

// A contiguous vector of n values, of x's type or fp32.
const void* vector_of(const Tensor& t, const char* name, int64_t n, at::ScalarType dtype, bool fp32_too, const at::Device& device) {
  if (t.scalar_type() != dtype && !(fp32_too && t.scalar_type() == at::kFloat))
    throw TypeError("%s must be %s%s, got %s", name, name_of(dtype), fp32_too ? " or float32" : "", name_of(t.scalar_type()));
  on_device(t, name, device);
  if (t.numel() != n || !t.is_contiguous()) throw ValueError("%s must be a contiguous (%lld,) vector", name, (long long)n);
  return t.data_ptr();
}

// An index into `names` by a Python string.
int choice(PyObject* o, const char* name, std::initializer_list<const char*> names) {
  int i = 0;
  std::string all;
  for (const char* n : names) {
    if (PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, n) == 0) return i;
    all += (i++ ? ", '" : "'") + std::string(n) + "'";
  }
  PyObject* r = PyObject_Repr(o);
  const char* text = r ? PyUnicode_AsUTF8(r) : nullptr;
  const std::string got = text ? text : "?";
  Py_XDECREF(r);
  PyErr_Clear();
  throw ValueError("%s must be one of %s, got %s", name, all.c_str(), got.c_str());
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

Tensor empty(c10::IntArrayRef shape, at::ScalarType dtype, const at::Device& device) {
  return at::detail::empty_cuda(shape, dtype, device, std::nullopt);
}
// The result as Python has it; autograd is told that a tensor of the caller's has changed.
PyObject* wrap(PyObject* given, const Tensor& t) {
  if (given == Py_None) return THPVariable_Wrap(t);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return Py_NewRef(given);
}

// The device and stream of a call: x's device, and the caller's torch.cuda.Stream or the current
// one. Outputs and workspace come from that stream's memory, which no other stream is using.
class Place {
 public:
  Place(PyObject* stream, const at::Device& device) : device_(device) {
    if (stream != Py_None) {
      PyObject* v = PyObject_GetAttrString(stream, "cuda_stream");
      if (!v) throw Raised();
      void* s = PyLong_AsVoidPtr(v);
      Py_DECREF(v);
      if (PyErr_Occurred()) throw Raised();
      stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), device.index()));
    }
    handle_ = reinterpret_cast<fn_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  }
  fn_stream_t stream() const { return handle_; }

 private:
  const c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
  fn_stream_t handle_;
};

// Handles of the configurations used last, the latest first. Configurations are zeroed before they
// are filled, so their bytes compare; the interpreter's lock guards the list. A launch keeps nothing
// of its handle, so one whose configuration has not come for kHandles others is given up (theta and
// eps are part of a configuration: a program may change them with each length).
constexpr size_t kHandles = 64;
template <typename Config, typename Handle>
Handle handle_for(const Config& c, fn_status (*create)(Handle*, const Config*), fn_status (*destroy)(Handle), const char* what) {
  static std::vector<std::pair<Config, Handle>> known;
  for (size_t i = 0; i < known.size(); ++i)
    if (std::memcmp(&known[i].first, &c, sizeof(c)) == 0) {
      std::rotate(known.begin(), known.begin() + i, known.begin() + i + 1);
      return known.front().second;
    }
  Handle h;
  check_status(create(&h, &c), what);
  if (known.size() == kHandles) {
    destroy(known.back().second);
    known.pop_back();
  }
  known.emplace(known.begin(), c, h);
  return h;
}
template <typename T>
T zeroed() {
  T v;
  std::memset(&v, 0, sizeof(v));
  return v;
}

// A function of `n` positional arguments; Python errors come out as they were set.
#define ENTRY(name, n)                                                                 \
  PyObject* name##_impl(PyObject* const* a);                                           \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t count) {                    \
    HANDLE_TH_ERRORS                                                                   \
    try {                                                                              \
      if (count != (n)) throw TypeError(#name " takes %d arguments", (int)(n));        \
      return name##_impl(a);                                                           \
    } catch (const Raised&) {                                                          \
      return nullptr;                                                                  \
    }                                                                                  \
    END_HANDLE_TH_ERRORS                                                               \
  }                                                                                    \
  PyObject* name##_impl(PyObject* const* a)

// ---- norm_quant ------------------------------------------------------------------------------
// residual, x, gate, weight, bias, scale, shift, norm_type, eps, out, row_scale_out,
// residual_out, stream -> (q, row_scale, r), without r where residual is None
ENTRY(norm_quant, 13) {
  const Tensor* residual = tensor(a[0], "residual", true);
  const Tensor& x = *tensor(a[1], "x");
  const Tensor *gate = tensor(a[2], "gate", true), *weight = tensor(a[3], "weight", true), *bias = tensor(a[4], "bias", true);
  const Tensor *scale = tensor(a[5], "scale", true), *shift = tensor(a[6], "shift", true);
  if (x.dim() != 3) throw ValueError("x must be a (B, L, D) tensor");
  if (!x.is_cuda()) throw ValueError("x must be a CUDA tensor");
  const at::Device device = x.device();
  const at::ScalarType bf = at::kBFloat16;
  check_tensor(x, "x", device, bf);
  const int64_t B = x.size(0), L = x.size(1), D = x.size(2);
  if (D % 16 || D < 16 || D > 16384) throw ValueError("D must be a multiple of 16 from 16 to 16384, got %lld", (long long)D);
  if (!scale != !shift) throw ValueError("scale and shift come together");
  const double eps = number(a[8]);
  if (!(eps >= 0) || !std::isfinite(eps)) throw ValueError("eps must be finite and not negative");

  nq_config c = zeroed<nq_config>();
  c.D = (int)D;
  c.is_rms = choice(a[7], "norm_type", {"layer", "rms", "ln", "rmsnorm", "layernorm"}) % 2;
  c.has_residual = residual != nullptr, c.has_gate = gate != nullptr;
  c.has_weight = weight != nullptr, c.has_bias = bias != nullptr;
  c.has_modulation = scale != nullptr;
  c.eps = eps;
  nq_args g = zeroed<nq_args>();
  g.B = B, g.L = L;
  g.x = rows_of(x);
  int64_t frames = 0;
  if (gate) g.gate = operand_of(*gate, "gate", B, L, D, bf, device, &frames);
  if (scale) g.scale = operand_of(*scale, "scale", B, L, D, bf, device, &frames);
  if (shift) g.shift = operand_of(*shift, "shift", B, L, D, bf, device, &frames);
  g.tokens_per_frame = frames ? L / frames : 0;
  if (weight) g.weight = vector_of(*weight, "weight", D, bf, true, device);
  if (bias) g.bias = vector_of(*bias, "bias", D, bf, true, device);
  if (weight && bias && weight->scalar_type() != bias->scalar_type()) throw TypeError("weight and bias must have the same dtype");
  c.affine_fp32 = (weight && weight->scalar_type() == at::kFloat) || (bias && bias->scalar_type() == at::kFloat);

  const Place place(a[12], device);
  Tensor r, q, s;
  if (residual) {
    check_tensor(*residual, "residual", device, bf);
    if (residual->sizes() != x.sizes()) throw ValueError("residual must match x");
    g.residual = rows_of(*residual);
    r = a[11] == Py_None ? empty(x.sizes(), bf, device) : *tensor(a[11], "residual_out");
    check_shape(r, "residual_out", x.sizes(), bf, device);
    check_tensor(r, "residual_out", device, bf);
    const fn_operand to = rows_of(r);
    g.r = r.data_ptr(), g.r_stride_b = to.stride_b, g.r_stride_l = to.stride_l;
  }
  q = a[9] == Py_None ? empty(x.sizes(), at::kFloat8_e4m3fn, device) : *tensor(a[9], "out");
  check_shape(q, "out", x.sizes(), at::kFloat8_e4m3fn, device);
  if (q.stride(2) != 1) throw ValueError("out needs a contiguous channel dimension");
  s = a[10] == Py_None ? empty({B, L}, at::kFloat, device) : *tensor(a[10], "row_scale_out");
  check_shape(s, "row_scale_out", {B, L}, at::kFloat, device);
  if (!s.is_contiguous()) throw ValueError("row_scale_out must be contiguous");
  const fn_operand to = rows_of(q);
  g.q = q.data_ptr(), g.q_stride_b = to.stride_b, g.q_stride_l = to.stride_l;
  g.row_scale = static_cast<float*>(s.data_ptr());
  const norm_quant_t h = handle_for(c, norm_quant_create, norm_quant_destroy, "norm_quant_create");
  check_status(norm_quant_launch(h, &g, place.stream()), "norm_quant_launch");
  PyObject* out = PyTuple_New(residual ? 3 : 2);
  if (!out) throw Raised();
  PyTuple_SET_ITEM(out, 0, wrap(a[9], q));
  PyTuple_SET_ITEM(out, 1, wrap(a[10], s));
  if (residual) PyTuple_SET_ITEM(out, 2, wrap(a[11], r));
  return out;
}

// ---- rope_norm -------------------------------------------------------------------------------

rn_rows heads_of(const Tensor& t, const char* name, const Tensor* like) {
  if (t.dim() != 4) throw ValueError("%s must be a (B, L, H, hd) tensor", name);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
    throw TypeError("%s must be bfloat16 or float16, got %s", name, name_of(t.scalar_type()));
  if (!t.is_cuda()) throw ValueError("%s must be a CUDA tensor", name);
  if (like) check_shape(t, name, like->sizes(), like->scalar_type(), like->device());
  if (t.size(3) > 1 && t.stride(3) != 1) throw ValueError("%s needs contiguous channels", name);
  return rn_rows{t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0, t.size(2) > 1 ? t.stride(2) : 0};
}

struct RopeCall {
  rope_norm_t h;
  const void *positions, *weight;
  int64_t psb, psl;
  int values;  // of the weight
};
// a: positions, sections, weight, theta, pairing, shared_frequencies, norm, eps
RopeCall rope_call(const Tensor& x, PyObject* const* a) {
  const int64_t B = x.size(0), L = x.size(1), H = x.size(2), hd = x.size(3);
  const Tensor &pos = *tensor(a[0], "positions"), *weight = tensor(a[2], "weight", true);
  rn_config c = zeroed<rn_config>();
  c.norm = choice(a[6], "norm", {"none", "head", "all"});
  c.half_pairs = choice(a[4], "pairing", {"interleaved", "half"});
  c.shared_frequencies = truth(a[5]);
  c.theta = number(a[3]), c.eps = number(a[7]);
  if (!std::isfinite(c.theta) || c.theta <= 0) throw ValueError("theta must be finite and positive");
  if (!std::isfinite(c.eps) || c.eps < 0) throw ValueError("eps must be finite and not negative");
  PyObject* seq = PySequence_Fast(a[1], "sections must be a sequence of numbers");
  if (!seq) throw Raised();
  const Py_ssize_t axes = PySequence_Fast_GET_SIZE(seq);
  bool ok = axes >= 1 && axes <= 4;
  int64_t pairs = 0;
  for (Py_ssize_t i = 0; ok && i < axes; ++i) {
    const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
    if (v == -1 && PyErr_Occurred()) {
      Py_DECREF(seq);
      throw Raised();
    }
    ok = v >= 1 && v <= 1 << 20;
    c.section[i] = (int)v;
    pairs += v;
  }
  Py_DECREF(seq);
  if (!ok) throw ValueError("sections must be one to four positive numbers");
  if (H < 1 || hd % 16 || hd < 16 || hd > 512 || H * hd > 16384)
    throw ValueError("heads must be of a multiple of 16 channels up to 512, and 16384 in all, got (%lld, %lld)", (long long)H, (long long)hd);
  if (2 * pairs > hd) throw ValueError("sections turn %lld channels of %lld", (long long)(2 * pairs), (long long)hd);
  if (c.half_pairs && pairs % 8) throw ValueError("pairing 'half' needs sections that add up to a multiple of 8, got %lld", (long long)pairs);
  c.axes = (int)axes;
  c.dtype = code_of(x.scalar_type());
  c.heads = (int)H, c.head_dim = (int)hd;

  RopeCall r{};
  if (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong) throw TypeError("positions must be an int32 or int64 tensor");
  on_device(pos, "positions", x.device());
  const bool batched = pos.dim() == 3;
  if ((pos.dim() != 2 && !batched) || pos.size(-2) != L || pos.size(-1) != axes || (batched && pos.size(0) != 1 && pos.size(0) != B))
    throw ValueError("positions must be (%lld, %d) or (%lld, %lld, %d), got %s", (long long)L, (int)axes, (long long)B, (long long)L,
                     (int)axes, shape_of(pos.sizes()).c_str());
  if (axes > 1 && pos.stride(-1) != 1) throw ValueError("positions needs a contiguous last dimension");
  c.index64 = pos.scalar_type() == at::kLong;
  r.positions = pos.data_ptr();
  r.psb = batched && pos.size(0) > 1 ? pos.stride(0) : 0;
  r.psl = L > 1 ? pos.stride(-2) : 0;
  r.values = (int)(c.norm == BO_NORM_ALL ? H * hd : hd);
  if (weight) {
    if (c.norm == BO_NORM_NONE) throw ValueError("weight needs a norm");
    r.weight = vector_of(*weight, "weight", r.values, x.scalar_type(), true, x.device());
    c.has_weight = 1;
    c.weight_fp32 = weight->scalar_type() == at::kFloat;
  }
  r.h = handle_for(c, rope_norm_create, rope_norm_destroy, "rope_norm_create");
  return r;
}

// x, positions, sections, weight, theta, pairing, shared_frequencies, norm, eps, out, stream -> y
ENTRY(rope_norm, 11) {
  const Tensor& x = *tensor(a[0], "x");
  rn_args g = zeroed<rn_args>();
  g.x = heads_of(x, "x", nullptr);
  const RopeCall call = rope_call(x, a + 1);
  const Place place(a[10], x.device());
  const Tensor y = a[9] == Py_None ? empty(x.sizes(), x.scalar_type(), x.device()) : *tensor(a[9], "out");
  g.B = x.size(0), g.L = x.size(1);
  g.positions = call.positions, g.pos_stride_b = call.psb, g.pos_stride_l = call.psl, g.weight = call.weight;
  g.y = heads_of(y, "out", &x);
  check_status(rope_norm_launch(call.h, &g, place.stream()), "rope_norm_launch");
  return wrap(a[9], y);
}

// grad, x, positions, sections, weight, theta, pairing, shared_frequencies, norm, eps, out,
// stream -> (dx, dweight or None)
ENTRY(rope_norm_backward, 12) {
  const Tensor &grad = *tensor(a[0], "grad"), &x = *tensor(a[1], "x");
  rn_backward_args g = zeroed<rn_backward_args>();
  g.x = heads_of(x, "x", nullptr);
  g.grad = heads_of(grad, "grad", &x);
  const RopeCall call = rope_call(x, a + 2);
  if (choice(a[8], "norm", {"none", "head", "all"}) == BO_NORM_NONE) g.x = rn_rows{nullptr, 0, 0, 0};
  const Place place(a[11], x.device());
  const Tensor dx = a[10] == Py_None ? empty(x.sizes(), x.scalar_type(), x.device()) : *tensor(a[10], "out");
  g.B = x.size(0), g.L = x.size(1);
  g.positions = call.positions, g.pos_stride_b = call.psb, g.pos_stride_l = call.psl, g.weight = call.weight;
  g.dx = heads_of(dx, "out", &x);
  Tensor dw, work;
  if (call.weight) {
    const Tensor& w = THPVariable_Unpack(a[4]);
    dw = empty(w.sizes(), at::kFloat, x.device());
    check_status(rope_norm_backward_workspace(call.h, g.B, g.L, &g.workspace_bytes), "rope_norm_backward_workspace");
    work = empty({(int64_t)g.workspace_bytes}, at::kByte, x.device());
    g.dweight = static_cast<float*>(dw.data_ptr());
    g.workspace = g.workspace_bytes ? work.data_ptr() : nullptr;
  }
  check_status(rope_norm_backward_launch(call.h, &g, place.stream()), "rope_norm_backward_launch");
  PyObject* out = PyTuple_New(2);
  if (!out) throw Raised();
  PyTuple_SET_ITEM(out, 0, wrap(a[10], dx));
  PyTuple_SET_ITEM(out, 1, call.weight ? THPVariable_Wrap(dw) : Py_NewRef(Py_None));
  return out;
}

// ---- linear_gate -----------------------------------------------------------------------------
// x, weight, bias, gate, residual, activation, x_scale, weight_scale, out, stream -> out
ENTRY(linear_gate, 10) {
  const Tensor &x = *tensor(a[0], "x"), &w = *tensor(a[1], "weight");
  const Tensor *bias = tensor(a[2], "bias", true), *gate = tensor(a[3], "gate", true), *residual = tensor(a[4], "residual", true);
  const Tensor *xs = tensor(a[6], "x_scale", true), *ws = tensor(a[7], "weight_scale", true);
  if (x.dim() != 3) throw ValueError("x must be a (B, L, K) tensor");
  const at::ScalarType type = x.scalar_type();
  const bool fp8 = type == at::kFloat8_e4m3fn;
  if (type != at::kBFloat16 && type != at::kHalf && !fp8)
    throw TypeError("x must be bfloat16, float16 or float8_e4m3fn, got %s", name_of(type));
  if (!x.is_cuda()) throw ValueError("x must be a CUDA tensor");
  const at::Device device = x.device();
  const at::ScalarType dtype = fp8 ? at::kBFloat16 : type;
  check_tensor(x, "x", device, type);
  check_tensor(w, "weight", device, type);
  const int64_t B = x.size(0), L = x.size(1), K = x.size(2);
  if (w.dim() != 2 || w.size(1) != K) throw ValueError("weight must be an (N, %lld) matrix, got %s", (long long)K, shape_of(w.sizes()).c_str());
  const int64_t N = w.size(0), unit = fp8 ? 16 : 8;
  if (K < 8 || N < 8 || K % unit || N % 8 || K > 1 << 20 || N > 1 << 20)
    throw ValueError("K must be a multiple of %d and N of 8, up to 2^20, got K=%lld, N=%lld", (int)unit, (long long)K, (long long)N);
  lg_config c = zeroed<lg_config>();
  c.dtype = code_of(type), c.K = K, c.N = N;
  c.act = choice(a[5], "activation", {"none", "silu", "gelu", "gelu_tanh"});
  c.has_bias = bias != nullptr, c.has_gate = gate != nullptr, c.has_residual = residual != nullptr;
  lg_args g = zeroed<lg_args>();
  g.B = B, g.L = L;
  g.x = rows_of(x);
  g.weight = w.data_ptr(), g.weight_stride = w.stride(0);
  if (fp8 != (xs != nullptr) || fp8 != (ws != nullptr))
    throw ValueError("x_scale and weight_scale are given with float8_e4m3fn, and only then");
  if (fp8) {
    check_shape(*xs, "x_scale", {B, L}, at::kFloat, device);
    check_shape(*ws, "weight_scale", {N}, at::kFloat, device);
    if (!xs->is_contiguous() || !ws->is_contiguous()) throw ValueError("x_scale and weight_scale must be contiguous");
    g.x_scale = static_cast<const float*>(xs->data_ptr()), g.weight_scale = static_cast<const float*>(ws->data_ptr());
  }
  if (bias) g.bias = vector_of(*bias, "bias", N, dtype, false, device);
  int64_t frames = 0;
  if (gate) g.gate = operand_of(*gate, "gate", B, L, N, dtype, device, &frames);
  g.tokens_per_frame = frames ? L / frames : 0;
  if (residual) {
    check_shape(*residual, "residual", {B, L, N}, dtype, device);
    check_tensor(*residual, "residual", device, dtype);
    g.residual = rows_of(*residual);
  }
  const Place place(a[9], device);
  const Tensor out = a[8] == Py_None ? empty({B, L, N}, dtype, device) : *tensor(a[8], "out");
  check_shape(out, "out", {B, L, N}, dtype, device);
  check_tensor(out, "out", device, dtype);
  const fn_operand to = rows_of(out);
  g.out = out.data_ptr(), g.out_stride_b = to.stride_b, g.out_stride_l = to.stride_l;
  const linear_gate_t h = handle_for(c, linear_gate_create, linear_gate_destroy, "linear_gate_create");
  check_status(linear_gate_launch(h, &g, place.stream()), "linear_gate_launch");
  return wrap(a[8], out);
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(norm_quant), METHOD(rope_norm), METHOD(rope_norm_backward), METHOD(linear_gate), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* abi = PyImport_ImportModule("rmsnorm_row_b200._abi");
  if (!abi) return nullptr;
  g_error = PyObject_GetAttrString(abi, "FusedNormError");
  Py_DECREF(abi);
  return g_error ? PyModule_Create(&kModule) : nullptr;
}

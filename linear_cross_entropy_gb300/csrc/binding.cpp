// Python module _native: the norms and the clipping on torch tensors, over the
// C ABI of include/cce_ops.h.  It checks arguments, describes strided rows,
// allocates results and workspaces with torch, and calls the library on the
// current stream.
//
// These calls are short (a norm of one token takes the GPU 2 us), so what the
// host does around them is most of their time.  Here instead of in Python, with
// the autograd nodes in C++ as well, the backward pass runs on the autograd
// engine's thread without the interpreter.
#include <ATen/TracerMode.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/cce_ops.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;
using OptType = std::optional<at::ScalarType>;

// A status of the library; Python sees it as CCEError.
struct StatusError : std::runtime_error {
  int status;
  StatusError(int s, const std::string& what) : std::runtime_error(what), status(s) {}
};

// `args`: what CCE_ERR_ARG is left to mean once the tensors have been checked here.
void check_status(cce_status st, const char* call, const char* args) {
  if (st != CCE_OK) throw StatusError(st, st == CCE_ERR_ARG ? std::string(call) + " (" + args + ")" : call);
}
const char* const NORM_ARGS = "eps must be finite and at least 0, weight_offset finite";
const char* const CLIP_ARGS =
    "eps must be finite and at least 0, and no tensor that is written may overlap another or be given twice";

template <typename... Parts>
[[noreturn]] void refuse(const Parts&... parts) {  // ValueError
  std::ostringstream s;
  (s << ... << parts);
  throw std::invalid_argument(s.str());
}

// What the calls cannot do by their nature; Python sees NotImplementedError.
struct Unsupported : std::runtime_error {
  using std::runtime_error::runtime_error;
};

// The kernels are launched beside torch's dispatcher, so what torch records or carries along there would miss them
// without a word: a traced graph would hold an empty tensor, a tangent would be read as 0.
void refuse_tracing() {
  if (at::tracer::impl::is_dispatch_enabled() ||
      c10::impl::TorchDispatchModeTLS::get_mode(c10::impl::TorchDispatchModeKey::PROXY).has_value())
    throw Unsupported("a call of this operator cannot be traced: its kernels would not be in the graph");
}

// Whether a tensor can have a tangent now.
bool tangents_live() { return torch::autograd::ForwardADLevel::try_get_by_idx(0) != nullptr; }

template <typename... Tensors>
void refuse_tangents(bool live, const Tensors&... tensors) {
  if (!live) return;
  const auto has = [](const Tensor& t) { return t.defined() && t._fw_grad(0).defined(); };
  if ((has(tensors) || ...))
    throw Unsupported("this operator has no forward-mode derivative: an argument has a tangent");
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return at::toString(t);
  }
}

// The library's code of an element type, -1 for others.
int type_code(at::ScalarType t) {
  return t == at::kFloat ? CCE_F32 : t == at::kHalf ? CCE_F16 : t == at::kBFloat16 ? CCE_BF16 : -1;
}

int checked_type(const Tensor& t, const char* name) {
  const int code = type_code(t.scalar_type());
  if (code < 0) refuse(name, " must be bfloat16, float16 or float32, got ", type_name(t.scalar_type()));
  return code;
}

// The values themselves in memory: of torch's lazily negated views a copy.
Tensor plain(const Tensor& t) { return t.defined() && t.is_neg() ? t.resolve_neg() : t; }

void* pointer(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

// -------------------------------------------------------------------- rows
// How the rows of a tensor's last dimension lie (cce_ops.h, "Rows").  Rows that
// are not at one pitch, or in runs at one pitch, or whose elements are apart
// are copied.
struct Rows {
  Tensor t;
  int64_t inner = int64_t(1) << 31, row = 0, outer = 0;
};

Rows rows_of(const Tensor& given) {
  const Tensor t = plain(given);
  Rows r;
  r.t = t;
  const int64_t last = t.dim() - 1;
  r.row = t.size(last);
  if (t.is_contiguous()) return r;
  int64_t n[2] = {1, 1}, s[2] = {0, 0};  // the leading dimensions, outermost first, merged where they continue each other
  int runs = 0;
  bool fits = t.size(last) == 1 || t.stride(last) == 1;
  for (int64_t d = 0; d < last && fits; ++d) {
    if (t.size(d) == 1) continue;
    if (runs > 0 && s[runs - 1] == t.size(d) * t.stride(d)) {
      n[runs - 1] *= t.size(d);
      s[runs - 1] = t.stride(d);
    } else if (runs == 2) {
      fits = false;
    } else {
      n[runs] = t.size(d);
      s[runs++] = t.stride(d);
    }
  }
  if (!fits) {
    r.t = t.contiguous();
  } else if (runs == 1) {
    r.row = s[0];
  } else if (runs == 2) {
    r.inner = n[1];
    r.row = s[1];
    r.outer = s[0];
  }
  return r;
}

// -------------------------------------------------------------------- norms
struct Sizes {
  int64_t N, D;
  at::ScalarType p_type;  // of the parameters; x's without any
};

Sizes check_norm(const Tensor& x, const Tensor& weight, const Tensor& bias) {
  refuse_tracing();
  refuse_tangents(tangents_live(), x, weight, bias);
  if (!x.is_cuda()) refuse("x must be a CUDA tensor (no CPU path)");
  checked_type(x, "x");
  if (x.dim() == 0 || x.size(-1) < 1) refuse("x needs a last dimension of at least one element, got shape ", x.sizes());
  const int64_t D = x.size(-1);
  Sizes s{x.numel() / D, D, x.scalar_type()};
  bool any = false;
  for (const auto& [p, name] : {std::pair{&weight, "weight"}, std::pair{&bias, "bias"}}) {
    if (!p->defined()) continue;
    if (p->device() != x.device()) refuse(name, " must be on ", x.device(), ", got ", p->device());
    checked_type(*p, name);
    if (p->dim() != 1 || p->size(0) != D || !p->is_contiguous())
      refuse(name, " must be contiguous [", D, "], got shape ", p->sizes());
    if (any && p->scalar_type() != s.p_type)
      refuse("weight and bias must have one type, got ", type_name(s.p_type), " and ", type_name(p->scalar_type()));
    s.p_type = p->scalar_type();
    any = true;
  }
  return s;
}

at::ScalarType result_type(const Tensor& x, const OptType& out) {
  if (!out || *out == x.scalar_type()) return x.scalar_type();
  if (type_code(*out) < 0 || x.scalar_type() != at::kFloat)
    refuse("out_dtype ", type_name(*out), " is not available from ", type_name(x.scalar_type()),
           ": the type of x, or a 16-bit type from float32");
  return *out;
}

Tensor statistics(const Tensor& x, int64_t N, bool wanted) {
  return wanted ? at::empty({N}, x.options().dtype(at::kFloat)) : Tensor();
}

std::tuple<Tensor, Tensor, Tensor> layer_forward(const Tensor& x, const Tensor& weight, const Tensor& bias, double eps,
                                                 const OptType& out, bool stats) {
  const Sizes s = check_norm(x, weight, bias);
  const at::ScalarType y_type = result_type(x, out);
  const c10::cuda::CUDAGuard guard(x.device());
  const Rows r = rows_of(x);
  const Tensor w = plain(weight), b = plain(bias);
  Tensor y = at::empty(x.sizes(), x.options().dtype(y_type));
  Tensor mean = statistics(x, s.N, stats), rstd = statistics(x, s.N, stats);
  check_status(cce_layer_norm_forward(pointer(r.t), r.inner, r.row, r.outer, type_code(x.scalar_type()),
                                      pointer(w), pointer(b), type_code(s.p_type), s.N, s.D,
                                      static_cast<float>(eps), pointer(y), type_code(y_type),
                                      static_cast<float*>(pointer(mean)), static_cast<float*>(pointer(rstd)),
                                      stream_of(x)),
               "cce_layer_norm_forward", NORM_ARGS);
  return {y, mean, rstd};
}

std::tuple<Tensor, Tensor> rms_forward(const Tensor& x, const Tensor& weight, double eps, double offset,
                                       const OptType& out, bool stats) {
  const Sizes s = check_norm(x, weight, Tensor());
  const at::ScalarType y_type = result_type(x, out);
  const c10::cuda::CUDAGuard guard(x.device());
  const Rows r = rows_of(x);
  const Tensor w = plain(weight);
  Tensor y = at::empty(x.sizes(), x.options().dtype(y_type));
  Tensor rstd = statistics(x, s.N, stats);
  check_status(cce_rms_norm_forward(pointer(r.t), r.inner, r.row, r.outer, type_code(x.scalar_type()), pointer(w),
                                    type_code(s.p_type), static_cast<float>(offset), s.N, s.D,
                                    static_cast<float>(eps), pointer(y), type_code(y_type),
                                    static_cast<float*>(pointer(rstd)), stream_of(x)),
               "cce_rms_norm_forward", NORM_ARGS);
  return {y, rstd};
}

void check_backward(const Tensor& g, const Tensor& x, int64_t N, const Tensor& stat, const char* name) {
  refuse_tangents(tangents_live(), g, stat);
  if (g.device() != x.device()) refuse("grad_y must be on ", x.device(), ", got ", g.device());
  if (g.sizes() != x.sizes()) refuse("grad_y must have the shape of x, ", x.sizes(), ", got ", g.sizes());
  if (g.scalar_type() != x.scalar_type() && (x.scalar_type() != at::kFloat || type_code(g.scalar_type()) < 0))
    refuse("grad_y must be ", type_name(x.scalar_type()), ", or a 16-bit type for float32 x, got ",
           type_name(g.scalar_type()));
  if (stat.device() != x.device() || stat.scalar_type() != at::kFloat || stat.numel() != N || !stat.is_contiguous() ||
      stat.is_neg())
    refuse(name, " must be contiguous float32 with ", N, " values on ", x.device());
}

std::tuple<Tensor, Tensor, Tensor> layer_backward(const Tensor& g, const Tensor& x, const Tensor& weight,
                                                  const Tensor& mean, const Tensor& rstd, bool need_dx, bool need_dw,
                                                  bool need_db, const OptType& param_type) {
  Sizes s = check_norm(x, weight, Tensor());
  if (!weight.defined() && param_type) {
    if (type_code(*param_type) < 0)
      refuse("param_dtype must be bfloat16, float16 or float32, got ", type_name(*param_type));
    s.p_type = *param_type;
  }
  check_backward(g, x, s.N, mean, "mean");
  check_backward(g, x, s.N, rstd, "rstd");
  const c10::cuda::CUDAGuard guard(x.device());
  const Rows xr = rows_of(x), gr = rows_of(g);
  const Tensor w = plain(weight);
  const auto params = x.options().dtype(s.p_type);
  Tensor dx = need_dx ? at::empty(x.sizes(), x.options()) : Tensor();
  Tensor dw = need_dw ? at::empty({s.D}, params) : Tensor(), db = need_db ? at::empty({s.D}, params) : Tensor();
  const size_t need = need_dw || need_db ? cce_norm_backward_workspace_bytes(s.N, s.D) : 0;
  Tensor ws = need ? at::empty({static_cast<int64_t>(need)}, x.options().dtype(at::kByte)) : Tensor();
  check_status(
      cce_layer_norm_backward(pointer(gr.t), gr.inner, gr.row, gr.outer, type_code(g.scalar_type()), pointer(xr.t),
                              xr.inner, xr.row, xr.outer, type_code(x.scalar_type()), pointer(w),
                              type_code(s.p_type), static_cast<const float*>(pointer(mean)),
                              static_cast<const float*>(pointer(rstd)), s.N, s.D, pointer(dx), pointer(dw),
                              pointer(db), pointer(ws), need, stream_of(x)),
      "cce_layer_norm_backward", NORM_ARGS);
  return {dx, dw, db};
}

std::tuple<Tensor, Tensor> rms_backward(const Tensor& g, const Tensor& x, const Tensor& weight, const Tensor& rstd,
                                        double offset, bool need_dx, bool need_dw) {
  const Sizes s = check_norm(x, weight, Tensor());
  check_backward(g, x, s.N, rstd, "rstd");
  const c10::cuda::CUDAGuard guard(x.device());
  const Rows xr = rows_of(x), gr = rows_of(g);
  const Tensor w = plain(weight);
  need_dw = need_dw && weight.defined();
  Tensor dx = need_dx ? at::empty(x.sizes(), x.options()) : Tensor();
  Tensor dw = need_dw ? at::empty({s.D}, x.options().dtype(s.p_type)) : Tensor();
  const size_t need = need_dw ? cce_norm_backward_workspace_bytes(s.N, s.D) : 0;
  Tensor ws = need ? at::empty({static_cast<int64_t>(need)}, x.options().dtype(at::kByte)) : Tensor();
  check_status(
      cce_rms_norm_backward(pointer(gr.t), gr.inner, gr.row, gr.outer, type_code(g.scalar_type()), pointer(xr.t),
                            xr.inner, xr.row, xr.outer, type_code(x.scalar_type()), pointer(w),
                            type_code(s.p_type), static_cast<float>(offset),
                            static_cast<const float*>(pointer(rstd)), s.N, s.D, pointer(dx), pointer(dw), pointer(ws),
                            need, stream_of(x)),
      "cce_rms_norm_backward", NORM_ARGS);
  return {dx, dw};
}

// ----------------------------------------------------------------- autograd
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// The gradients of a backward pass that is itself recorded: their own gradient
// is an error, not zero.
void no_second_derivative(variable_list& grads) {
  if (!at::GradMode::is_enabled()) return;
  for (auto& g : grads) {
    if (!g.defined()) continue;
    auto error = std::make_shared<torch::autograd::DelayedError>(
        "the norm's gradient is not differentiable: its backward pass has no derivative", 1);
    g = g.detach().set_requires_grad(true);
    g = (*error)({g})[0];
  }
}

Tensor given(const OptTensor& t) { return t ? *t : Tensor(); }

struct LayerNorm : torch::autograd::Function<LayerNorm> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const OptTensor& weight, const OptTensor& bias,
                        double eps, OptType out) {
    auto [y, mean, rstd] = layer_forward(x, given(weight), given(bias), eps, out, true);
    ctx->save_for_backward({x, given(weight), mean, rstd});
    if (bias) ctx->saved_data["param_type"] = static_cast<int64_t>(bias->scalar_type());
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list g) {
    const auto saved = ctx->get_saved_variables();
    OptType p_type;
    if (const auto it = ctx->saved_data.find("param_type"); it != ctx->saved_data.end())
      p_type = static_cast<at::ScalarType>(it->second.toInt());
    // the edges of the tensors that there were, in order
    const bool weight = saved[1].defined();
    const bool need_dw = weight && ctx->needs_input_grad(1);
    const bool need_db = p_type && ctx->needs_input_grad(weight ? 2 : 1);
    variable_list grads;
    {
      const at::NoGradGuard no_grad;
      auto [dx, dw, db] = layer_backward(g[0], saved[0], saved[1], saved[2], saved[3], ctx->needs_input_grad(0),
                                         need_dw, need_db, p_type);
      grads = {dx, dw, db, Tensor(), Tensor()};
    }
    no_second_derivative(grads);
    return grads;
  }
};

struct RMSNorm : torch::autograd::Function<RMSNorm> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const OptTensor& weight, double eps, double offset,
                        OptType out) {
    auto [y, rstd] = rms_forward(x, given(weight), eps, offset, out, true);
    ctx->save_for_backward({x, given(weight), rstd});
    ctx->saved_data["offset"] = offset;
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list g) {
    const auto saved = ctx->get_saved_variables();
    variable_list grads;
    {
      const at::NoGradGuard no_grad;
      auto [dx, dw] = rms_backward(g[0], saved[0], saved[1], saved[2], ctx->saved_data["offset"].toDouble(),
                                   ctx->needs_input_grad(0),
                                   saved[1].defined() && ctx->needs_input_grad(1));
      grads = {dx, dw, Tensor(), Tensor(), Tensor()};
    }
    no_second_derivative(grads);
    return grads;
  }
};

bool records(const Tensor& t) { return t.defined() && t.requires_grad(); }

Tensor layer_norm(const Tensor& x, const OptTensor& weight, const OptTensor& bias, double eps, const OptType& out) {
  const Tensor w = given(weight), b = given(bias);
  if (at::GradMode::is_enabled() && (records(x) || records(w) || records(b)))
    return LayerNorm::apply(x, weight, bias, eps, out);
  return std::get<0>(layer_forward(x, w, b, eps, out, false));
}

Tensor rms_norm(const Tensor& x, const OptTensor& weight, double eps, double offset, const OptType& out) {
  const Tensor w = given(weight);
  if (at::GradMode::is_enabled() && (records(x) || records(w))) return RMSNorm::apply(x, weight, eps, offset, out);
  return std::get<0>(rms_forward(x, w, eps, offset, out, false));
}

// ----------------------------------------------------------------- clipping
struct Dim {
  int64_t size, in, out;  // in and out: strides
};

// Dimensions of g and o, outermost first, without those of size one and merged
// where the elements of both tensors continue.
std::vector<Dim> dims_of(const Tensor& g, const Tensor& o) {
  std::vector<Dim> all;
  for (int64_t d = 0; d < g.dim(); ++d) {
    if (g.size(d) != 1) all.push_back({g.size(d), g.stride(d), o.stride(d)});
  }
  std::stable_sort(all.begin(), all.end(),
                   [](const Dim& a, const Dim& b) { return a.out != b.out ? a.out > b.out : a.in > b.in; });
  std::vector<Dim> dims;
  for (const Dim& d : all) {
    if (!dims.empty() && dims.back().in == d.size * d.in && dims.back().out == d.size * d.out) {
      dims.back() = {dims.back().size * d.size, d.in, d.out};
    } else {
      dims.push_back(d);
    }
  }
  return dims;
}

void check_dense(const Tensor& t, const Tensor& first, const char* name) {
  if (t.layout() != at::kStrided) refuse(name, " must be dense tensors");
  if (!t.is_cuda()) refuse(name, " must be CUDA tensors (no CPU path)");
  if (type_code(t.scalar_type()) < 0)
    refuse(name, " must be bfloat16, float16 or float32, got ", type_name(t.scalar_type()));
  if (t.device() != first.device()) refuse(name, " must be on one device, got ", first.device(), " and ", t.device());
}

struct Tables {
  std::vector<int64_t> dense;  // four words a tensor
  std::vector<cce_strided> strided;

  void add_dense(const Tensor& g, const Tensor& o) {
    dense.insert(dense.end(), {reinterpret_cast<int64_t>(g.data_ptr()), reinterpret_cast<int64_t>(o.data_ptr()),
                               g.numel(), type_code(g.scalar_type()) + 256 * type_code(o.scalar_type())});
  }
  void add_strided(const Tensor& g, const Tensor& o, bool written) {
    std::vector<Dim> dims = dims_of(g, o);
    for (const Dim& d : dims) {
      if (written && d.out == 0)
        refuse("an expanded tensor cannot be written: several of its elements share memory");
    }
    if (dims.empty() || (dims.size() == 1 && dims[0].in == 1 && dims[0].out == 1)) return add_dense(g, o);
    if (dims.size() > 4)
      refuse("a tensor of shape ", g.sizes(), " and strides ", g.strides(),
             " has more than 4 dimensions that do not continue each other: make it contiguous");
    cce_strided s{g.data_ptr(), o.data_ptr(), type_code(g.scalar_type()), type_code(o.scalar_type()), {}, {}, {}};
    const size_t pad = 4 - dims.size();
    for (size_t i = 0; i < 4; ++i) {
      const Dim d = i < pad ? Dim{1, 0, 0} : dims[i - pad];
      s.size[i] = d.size;
      s.in_stride[i] = d.in;
      s.out_stride[i] = d.out;
    }
    strided.push_back(s);
  }
};

// The norm of the tensors; with outs, clipped by it into them.
Tensor clip(const std::vector<Tensor>& grads, const std::vector<Tensor>* outs, int norm_type, double max_norm,
            double eps) {
  refuse_tracing();
  const bool live = tangents_live();
  Tables t;
  t.dense.reserve(4 * grads.size());
  for (size_t i = 0; i < grads.size(); ++i) {
    const Tensor& g = grads[i];
    const Tensor& o = outs ? (*outs)[i] : g;
    refuse_tangents(live, g, o);
    check_dense(g, grads[0], "gradients");
    if (!o.is_same(g)) {
      check_dense(o, grads[0], "out");
      if (o.sizes() != g.sizes())
        refuse("out must have the shapes of the gradients: ", o.sizes(), " for ", g.sizes());
      if (o.is_neg() != g.is_neg()) refuse("a gradient or its out is a negated view (resolve_neg), the other is not");
    }
    if (g.is_contiguous() && o.is_contiguous()) {
      t.add_dense(g, o);
    } else if (g.numel() > 0) {
      t.add_strided(g, o, outs != nullptr);
    }
  }
  const c10::cuda::CUDAGuard guard(grads[0].device());
  const int64_t rows = static_cast<int64_t>(t.dense.size() / 4), strided = static_cast<int64_t>(t.strided.size());
  Tensor norm = at::empty({}, grads[0].options().dtype(at::kFloat));
  const size_t need = cce_grad_norm_workspace_bytes(rows, strided);
  Tensor ws = at::empty({static_cast<int64_t>(need)}, grads[0].options().dtype(at::kByte));
  if (!outs) {
    check_status(cce_grad_norm(t.dense.data(), rows, t.strided.data(), strided, norm_type, norm.data_ptr<float>(),
                               ws.data_ptr(), need, stream_of(norm)),
                 "cce_grad_norm", CLIP_ARGS);
    return norm;
  }
  check_status(cce_clip_grads(t.dense.data(), rows, t.strided.data(), strided, norm_type, static_cast<float>(max_norm),
                              static_cast<float>(eps), norm.data_ptr<float>(), ws.data_ptr(), need, stream_of(norm)),
               "cce_clip_grads", CLIP_ARGS);
  for (const Tensor& o : *outs) {  // autograd learns that these were written
    if (!o.is_inference()) o.unsafeGetTensorImpl()->bump_version();
  }
  return norm;
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  py::register_local_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const Unsupported& e) {
      PyErr_SetString(PyExc_NotImplementedError, e.what());
    } catch (const StatusError& e) {
      const py::object type = py::module_::import("linear_cross_entropy_gb300._lib").attr("CCEError");
      PyErr_SetObject(type.ptr(), type(e.status, e.what()).ptr());
    }
  });
  using Free = py::call_guard<py::gil_scoped_release>;
  m.def("layer_norm", &layer_norm, Free());
  m.def("rms_norm", &rms_norm, Free());
  m.def(
      "layer_norm_forward",
      [](const Tensor& x, const OptTensor& weight, const OptTensor& bias, double eps, const OptType& out, bool stats) {
        return layer_forward(x, given(weight), given(bias), eps, out, stats);
      },
      Free());
  m.def(
      "rms_norm_forward",
      [](const Tensor& x, const OptTensor& weight, double eps, double offset, const OptType& out, bool stats) {
        return rms_forward(x, given(weight), eps, offset, out, stats);
      },
      Free());
  m.def(
      "layer_norm_backward",
      [](const Tensor& g, const Tensor& x, const OptTensor& weight, const Tensor& mean, const Tensor& rstd, bool dx,
         bool dw, bool db, const OptType& p_type) {
        return layer_backward(g, x, given(weight), mean, rstd, dx, dw, db, p_type);
      },
      Free());
  m.def(
      "rms_norm_backward",
      [](const Tensor& g, const Tensor& x, const OptTensor& weight, const Tensor& rstd, double offset, bool dx,
         bool dw) { return rms_backward(g, x, given(weight), rstd, offset, dx, dw); },
      Free());
  m.def(
      "grad_norm",
      [](const std::vector<Tensor>& grads, int norm_type) { return clip(grads, nullptr, norm_type, 0.0, 0.0); },
      Free());
  m.def(
      "clip_grads",
      [](const std::vector<Tensor>& grads, const std::optional<std::vector<Tensor>>& outs, int norm_type,
         double max_norm, double eps) { return clip(grads, outs ? &*outs : &grads, norm_type, max_norm, eps); },
      Free());
  m.def("rows", [](const Tensor& t) {
    const Rows r = rows_of(t);
    return py::make_tuple(r.t, r.inner, r.row, r.outer);
  });
  m.def("dims", [](const Tensor& g, const Tensor& o) {
    py::list dims;
    for (const Dim& d : dims_of(g, o)) dims.append(py::make_tuple(d.size, d.in, d.out));
    return dims;
  });
}

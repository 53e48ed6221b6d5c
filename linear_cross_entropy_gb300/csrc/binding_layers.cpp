// The layers in front of the head on torch tensors, over the C ABI of
// include/cce_layers.h and include/cce_layers_ex.h: checks, operands that the tensor cores' copies can read,
// results, workspaces and the autograd nodes.
#include <array>
#include <atomic>

#include "../../include/cce_layers_ex.h"
#include "binding.h"

using namespace binding;

namespace {

const char* const ARGS = "an argument is outside of what the call takes";

std::atomic<uint64_t> used_devices{0};  // by index: those whose error word may be set

void note_device(const Tensor& t) { used_devices |= uint64_t(1) << (t.get_device() & 63); }

int activation_code(const std::string& name) {
  static const std::array<const char*, 5> names = {"none", "relu", "gelu", "gelu_tanh", "silu"};
  for (size_t i = 0; i < names.size(); ++i) {
    if (name == names[i]) return static_cast<int>(i);
  }
  refuse("activation must be one of None, 'relu', 'gelu', 'gelu_tanh', 'silu', got '", name, "'");
}

// Rows at one pitch.
struct Pitched {
  Tensor t;
  int64_t pitch = 0;
};

// The matrices of a call.  Rows that are not as the products take them are copied, all of a call in one launch.
class Matrices {
 public:
  // The matrix of a tensor's last dimension; others than operands of a product may have any one pitch.
  Pitched matrix(const Tensor& given, bool operand = false) {
    if (!given.defined()) return {};
    const Rows r = rows_of(given);
    const int64_t cols = given.size(-1), bytes = given.element_size(), vec = 16 / bytes;
    const bool one_pitch = r.outer == 0 && r.row >= cols && r.row < (int64_t(1) << 30);
    if (one_pitch && (!operand || (reinterpret_cast<uintptr_t>(r.t.data_ptr()) % 16 == 0 && r.row % vec == 0)))
      return {r.t, r.row};
    const int64_t rows = cols ? given.numel() / cols : 0, pitch = (cols + vec - 1) / vec * vec;
    Tensor to = at::empty({rows, pitch}, given.options().requires_grad(false));
    kept_.push_back(r.t);
    copies_.push_back({r.t.data_ptr(), to.data_ptr(), r.inner, r.row, r.outer, pitch, rows, cols, static_cast<int32_t>(bytes)});
    return {to, pitch};
  }
  Pitched operand(const Tensor& given) { return matrix(given, true); }

  void copy(const Tensor& on) {
    if (copies_.empty()) return;
    check_status(cce_copy_rows(copies_.data(), static_cast<int>(copies_.size()), stream_of(on)), "cce_copy_rows", ARGS);
  }

 private:
  std::vector<cce_row_copy> copies_;
  std::vector<Tensor> kept_;
};

// Rows that a kernel reads where they are, in runs at one pitch.
Rows read_rows(const Tensor& given) {
  Rows r = rows_of(given);
  if (r.row >= int64_t(1) << 30 || r.outer >= int64_t(1) << 45) r = rows_of(given.contiguous());
  return r;
}

struct Sizes {
  int64_t M, N, K;
  int type;
};

void check_weight(const Tensor& w, const Tensor& x, const char* name) {
  if (w.device() != x.device()) refuse(name, " must be on ", x.device(), ", got ", w.device());
  if (w.dim() != 2 || w.size(0) < 1 || w.size(1) != x.size(-1))
    refuse(name, " must be [N, ", x.size(-1), "] with N >= 1, got shape ", w.sizes());
  if (w.scalar_type() != x.scalar_type())
    refuse(name, " must be ", type_name(x.scalar_type()), " as x is, got ", type_name(w.scalar_type()));
}

Sizes check_layer(const Tensor& x, const Tensor& w, const char* weight_name) {
  if (!x.is_cuda()) refuse("x must be a CUDA tensor (no CPU path)");
  const int type = type_code(x.scalar_type());
  if (type != CCE_BF16 && type != CCE_F16)
    refuse("x must be bfloat16 or float16 (the tensor cores' types), got ", type_name(x.scalar_type()));
  if (x.dim() == 0 || x.size(-1) < 1) refuse("x needs a last dimension of at least one element, got shape ", x.sizes());
  check_weight(w, x, weight_name);
  return {x.numel() / x.size(-1), w.size(0), x.size(-1), type};
}

std::vector<int64_t> result_shape(const Tensor& x, int64_t N) {
  std::vector<int64_t> s = x.sizes().vec();
  s.back() = N;
  return s;
}

at::ScalarType result_type(const Tensor& x, const OptType& out) {
  if (!out || *out == x.scalar_type()) return x.scalar_type();
  if (*out != at::kFloat)
    refuse("out_dtype ", type_name(*out), " is not available from ", type_name(x.scalar_type()),
           ": the type of x, or float32");
  return at::kFloat;
}

void check_bias(const Tensor& bias, const Tensor& x, int64_t N) {
  if (!bias.defined()) return;
  if (bias.device() != x.device()) refuse("bias must be on ", x.device(), ", got ", bias.device());
  checked_type(bias, "bias");
  if (bias.dim() != 1 || bias.size(0) != N || !bias.is_contiguous())
    refuse("bias must be contiguous [", N, "], got shape ", bias.sizes());
}

// A matrix with a row for each row of x.
void check_rows(const Tensor& t, const Tensor& x, int64_t N, const char* name) {
  if (!t.defined()) return;
  if (t.device() != x.device()) refuse(name, " must be on ", x.device(), ", got ", t.device());
  if (t.sizes() != at::IntArrayRef(result_shape(x, N)))
    refuse(name, " must have the shape ", at::IntArrayRef(result_shape(x, N)), ", got ", t.sizes());
}

Tensor workspace(size_t need, const Tensor& x) {
  if (need == 0) refuse("the layer's sizes are outside of what the library takes");
  if (need <= 16) return Tensor();  // none needed
  return at::empty({static_cast<int64_t>(need)}, x.options().dtype(at::kByte).requires_grad(false));
}

// Pre-activations are kept in 16 bits of the library's own for bf16 (CCE_KEPT16, to torch int16), as they are for fp16.
at::ScalarType kept_type(const Tensor& x) { return x.scalar_type() == at::kBFloat16 ? at::kShort : x.scalar_type(); }

int kept_code(const Tensor& z, const Tensor& x, const char* name) {
  if (z.scalar_type() == x.scalar_type()) return type_code(z.scalar_type());
  if (z.scalar_type() != kept_type(x))
    refuse(name, " must be what the forward pass kept, or ", type_name(x.scalar_type()), " as x is, got ",
           type_name(z.scalar_type()));
  return CCE_KEPT16;
}

// What a relu's backward pass reads of z is its sign, and bf16 has one for all but z's last subnormals.
at::ScalarType kept_type(const Tensor& x, const std::string& activation) {
  return activation == "relu" ? x.scalar_type() : kept_type(x);
}

// z is kept in the type of `keep`, if there is one.
std::tuple<Tensor, Tensor> linear_forward(const Tensor& x, const Tensor& weight, const Tensor& bias,
                                          const Tensor& residual, const std::string& activation, const OptType& out,
                                          const OptType& keep) {
  refuse_tracing();
  refuse_tangents(tangents_live(), x, weight, bias, residual);
  const Sizes s = check_layer(x, weight, "weight");
  const int act = activation_code(activation);
  const at::ScalarType y_type = result_type(x, out);
  check_bias(bias, x, s.N);
  check_rows(residual, x, s.N, "residual");
  if (residual.defined() && residual.scalar_type() != y_type)
    refuse("residual must be ", type_name(y_type), " as the result is, got ", type_name(residual.scalar_type()));
  const at::NoGradGuard no_grad;
  const c10::cuda::CUDAGuard guard(x.device());
  const size_t need = cce_linear_forward_workspace_bytes(s.M, s.N, s.K);
  const Tensor ws = workspace(need, x);
  Matrices m;
  const Pitched xp = m.operand(x), wp = m.operand(weight);
  m.copy(x);
  const Rows r = residual.defined() ? read_rows(residual) : Rows{};
  const Tensor b = plain(bias);
  const auto shape = result_shape(x, s.N);
  Tensor y = at::empty(shape, x.options().dtype(y_type).requires_grad(false));
  Tensor z = keep && act != CCE_ACT_NONE ? at::empty(shape, x.options().dtype(*keep).requires_grad(false)) : Tensor();
  note_device(x);
  check_status(cce_linear_forward(pointer(xp.t), xp.pitch, pointer(wp.t), wp.pitch, s.type, pointer(b),
                                  b.defined() ? type_code(b.scalar_type()) : s.type, pointer(r.t), r.inner, r.row, r.outer, act,
                                  s.M, s.N, s.K, pointer(y), s.N, type_code(y_type), pointer(z), s.N,
                                  z.defined() ? kept_code(z, x, "z") : s.type, pointer(ws), need,
                                  stream_of(x)),
               "cce_linear_forward", ARGS);
  return {y, z};
}

std::tuple<Tensor, Tensor, Tensor> linear_backward(const Tensor& g, const Tensor& x, const Tensor& weight,
                                                   const Tensor& z, const std::string& activation, bool need_dx,
                                                   bool need_dw, bool need_db, const OptType& bias_type) {
  refuse_tracing();
  refuse_tangents(tangents_live(), g, x, weight, z);
  const Sizes s = check_layer(x, weight, "weight");
  const int act = activation_code(activation);
  check_rows(g, x, s.N, "grad_y");
  if (g.scalar_type() != x.scalar_type() && g.scalar_type() != at::kFloat)
    refuse("grad_y must be ", type_name(x.scalar_type()), " or torch.float32, got ", type_name(g.scalar_type()));
  int z_type = s.type;
  if (act != CCE_ACT_NONE) {
    if (!z.defined()) refuse("z, the forward's pre-activation, is needed with an activation");
    check_rows(z, x, s.N, "z");
    z_type = kept_code(z, x, "z");
  }
  const at::ScalarType b_type = bias_type ? *bias_type : x.scalar_type();
  if (type_code(b_type) < 0) refuse("bias_dtype must be bfloat16, float16 or float32, got ", type_name(b_type));
  const at::NoGradGuard no_grad;
  const c10::cuda::CUDAGuard guard(x.device());
  Matrices m;
  const Pitched gp = m.matrix(g), xp = m.operand(x), wp = m.operand(weight);
  const Pitched zp = act != CCE_ACT_NONE ? m.matrix(z) : Pitched{};
  m.copy(x);
  const bool direct = act == CCE_ACT_NONE && g.scalar_type() == x.scalar_type() &&
                      reinterpret_cast<uintptr_t>(pointer(gp.t)) % 16 == 0 && gp.pitch % 8 == 0;
  const int want = (need_dx ? CCE_WANT_DX : 0) | (need_dw ? CCE_WANT_DW : 0) | (need_db ? CCE_WANT_DB : 0);
  const size_t need = cce_linear_backward_workspace_bytes_ex(
      s.M, s.N, s.K, want | (!direct && (need_dx || need_dw) ? CCE_WANT_DZ : 0));
  const Tensor ws = workspace(need, x);
  const auto plainly = x.options().requires_grad(false);
  Tensor dx = need_dx ? at::empty(x.sizes(), plainly) : Tensor();
  Tensor dw = need_dw ? at::empty({s.N, s.K}, plainly) : Tensor();
  Tensor db = need_db ? at::empty({s.N}, plainly.dtype(b_type)) : Tensor();
  note_device(x);
  check_status(cce_linear_backward(pointer(gp.t), gp.pitch, type_code(g.scalar_type()), pointer(xp.t), xp.pitch,
                                   pointer(wp.t), wp.pitch, s.type, pointer(zp.t), zp.pitch, z_type, act, s.M, s.N, s.K,
                                   pointer(dx), pointer(dw), pointer(db), type_code(b_type), pointer(ws), need,
                                   stream_of(x)),
               "cce_linear_backward", ARGS);
  return {dx, dw, db};
}

std::tuple<Tensor, Tensor, Tensor> gated_forward(const Tensor& x, const Tensor& gate_weight, const Tensor& up_weight,
                                                 const std::string& activation, bool save) {
  refuse_tracing();
  refuse_tangents(tangents_live(), x, gate_weight, up_weight);
  const Sizes s = check_layer(x, gate_weight, "gate_weight");
  check_weight(up_weight, x, "up_weight");
  if (up_weight.size(0) != s.N)
    refuse("gate_weight and up_weight must have one shape, got ", gate_weight.sizes(), " and ", up_weight.sizes());
  const int act = activation_code(activation);
  const at::NoGradGuard no_grad;
  const c10::cuda::CUDAGuard guard(x.device());
  const size_t need = cce_gated_linear_forward_workspace_bytes(s.M, s.N, s.K);
  const Tensor ws = workspace(need, x);
  Matrices m;
  const Pitched xp = m.operand(x), gp = m.operand(gate_weight), up = m.operand(up_weight);
  m.copy(x);
  const auto shape = result_shape(x, s.N);
  const auto plainly = x.options().requires_grad(false);
  const auto kept = plainly.dtype(kept_type(x));
  Tensor y = at::empty(shape, plainly), z0 = save ? at::empty(shape, kept) : Tensor(),
         z1 = save ? at::empty(shape, kept) : Tensor();
  note_device(x);
  check_status(cce_gated_linear_forward(pointer(xp.t), xp.pitch, pointer(gp.t), gp.pitch, pointer(up.t), up.pitch,
                                        s.type, act, s.M, s.N, s.K, pointer(y), s.N, pointer(z0), pointer(z1), s.N,
                                        save ? kept_code(z0, x, "gate") : s.type, pointer(ws), need, stream_of(x)),
               "cce_gated_linear_forward", ARGS);
  return {y, z0, z1};
}

std::tuple<Tensor, Tensor, Tensor> gated_backward(const Tensor& g, const Tensor& x, const Tensor& gate_weight,
                                                  const Tensor& up_weight, const Tensor& gate, const Tensor& up,
                                                  const std::string& activation, bool need_dx, bool need_dg,
                                                  bool need_du) {
  refuse_tracing();
  refuse_tangents(tangents_live(), g, x, gate_weight, up_weight, gate, up);
  const Sizes s = check_layer(x, gate_weight, "gate_weight");
  check_weight(up_weight, x, "up_weight");
  if (up_weight.size(0) != s.N)
    refuse("gate_weight and up_weight must have one shape, got ", gate_weight.sizes(), " and ", up_weight.sizes());
  const int act = activation_code(activation);
  for (const auto& [t, name] : {std::pair{&g, "grad_y"}, std::pair{&gate, "gate"}, std::pair{&up, "up"}})
    check_rows(*t, x, s.N, name);
  if (g.scalar_type() != x.scalar_type())
    refuse("grad_y must be ", type_name(x.scalar_type()), " as x is, got ", type_name(g.scalar_type()));
  const int z_type = kept_code(gate, x, "gate");
  if (kept_code(up, x, "up") != z_type) refuse("gate and up must have one type");
  const at::NoGradGuard no_grad;
  const c10::cuda::CUDAGuard guard(x.device());
  const size_t need = cce_gated_linear_backward_workspace_bytes_ex(
      s.M, s.N, s.K, (need_dx ? CCE_WANT_DX : 0) | (need_dg ? CCE_WANT_DW : 0) | (need_du ? CCE_WANT_DW_UP : 0));
  const Tensor ws = workspace(need, x);
  Matrices m;
  const Pitched gy = m.matrix(g), xp = m.operand(x), wg = m.operand(gate_weight), wu = m.operand(up_weight);
  const Pitched z0 = m.matrix(gate), z1 = m.matrix(up);
  m.copy(x);
  const auto plainly = x.options().requires_grad(false);
  Tensor dx = need_dx ? at::empty(x.sizes(), plainly) : Tensor();
  Tensor dg = need_dg ? at::empty({s.N, s.K}, plainly) : Tensor();
  Tensor du = need_du ? at::empty({s.N, s.K}, plainly) : Tensor();
  note_device(x);
  check_status(cce_gated_linear_backward(pointer(gy.t), gy.pitch, pointer(xp.t), xp.pitch, pointer(wg.t), wg.pitch,
                                         pointer(wu.t), wu.pitch, s.type, pointer(z0.t), z0.pitch, pointer(z1.t),
                                         z1.pitch, z_type, act, s.M, s.N, s.K, pointer(dx), pointer(dg), pointer(du),
                                         pointer(ws), need, stream_of(x)),
               "cce_gated_linear_backward", ARGS);
  return {dx, dg, du};
}

// ----------------------------------------------------------------- autograd
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

struct Linear : torch::autograd::Function<Linear> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const OptTensor& bias,
                        const OptTensor& residual, const std::string& activation, OptType out) {
    auto [y, z] = linear_forward(x, weight, given(bias), given(residual), activation, out, kept_type(x, activation));
    ctx->save_for_backward({x, weight, z});
    ctx->saved_data["activation"] = activation;
    if (bias) ctx->saved_data["bias_type"] = static_cast<int64_t>(bias->scalar_type());
    ctx->saved_data["residual"] = residual.has_value();
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list g) {
    const auto saved = ctx->get_saved_variables();
    OptType b_type;
    if (const auto it = ctx->saved_data.find("bias_type"); it != ctx->saved_data.end())
      b_type = static_cast<at::ScalarType>(it->second.toInt());
    // the edges of the tensors that there were, in order
    const bool need_db = b_type && ctx->needs_input_grad(2);
    const bool need_dr = ctx->saved_data["residual"].toBool() && ctx->needs_input_grad(b_type ? 3 : 2);
    variable_list grads;
    if (ctx->needs_input_grad(0) || ctx->needs_input_grad(1) || need_db) {
      const at::NoGradGuard no_grad;
      auto [dx, dw, db] = linear_backward(g[0], saved[0], saved[1], saved[2], ctx->saved_data["activation"].toStringRef(),
                                          ctx->needs_input_grad(0), ctx->needs_input_grad(1), need_db, b_type);
      grads = {dx, dw, db};
    } else {
      grads = {Tensor(), Tensor(), Tensor()};
    }
    no_second_derivative(grads, "linear layer");
    grads.insert(grads.end(), {need_dr ? g[0] : Tensor(), Tensor(), Tensor()});
    return grads;
  }
};

struct GatedLinear : torch::autograd::Function<GatedLinear> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& gate_weight, const Tensor& up_weight,
                        const std::string& activation) {
    auto [y, gate, up] = gated_forward(x, gate_weight, up_weight, activation, true);
    ctx->save_for_backward({x, gate_weight, up_weight, gate, up});
    ctx->saved_data["activation"] = activation;
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list g) {
    const auto s = ctx->get_saved_variables();
    variable_list grads;
    {
      const at::NoGradGuard no_grad;
      auto [dx, dg, du] =
          gated_backward(g[0], s[0], s[1], s[2], s[3], s[4], ctx->saved_data["activation"].toStringRef(),
                         ctx->needs_input_grad(0), ctx->needs_input_grad(1), ctx->needs_input_grad(2));
      grads = {dx, dg, du, Tensor()};
    }
    no_second_derivative(grads, "gated linear layer");
    return grads;
  }
};

bool records(const Tensor& t) { return t.defined() && t.requires_grad(); }

Tensor linear(const Tensor& x, const Tensor& weight, const OptTensor& bias, const OptTensor& residual,
              const std::string& activation, const OptType& out) {
  const Tensor b = given(bias), r = given(residual);
  if (at::GradMode::is_enabled() && (records(x) || records(weight) || records(b) || records(r)))
    return Linear::apply(x, weight, bias, residual, activation, out);
  return std::get<0>(linear_forward(x, weight, b, r, activation, out, {}));
}

Tensor gated_linear(const Tensor& x, const Tensor& gate_weight, const Tensor& up_weight,
                    const std::string& activation) {
  if (at::GradMode::is_enabled() && (records(x) || records(gate_weight) || records(up_weight)))
    return GatedLinear::apply(x, gate_weight, up_weight, activation);
  return std::get<0>(gated_forward(x, gate_weight, up_weight, activation, false));
}

// The error words of all devices that these layers ran on, behind everything issued there.
int32_t take_error() {
  int32_t all = 0;
  for (int d = 0; d < 64; ++d) {
    if (!(used_devices.load() >> d & 1)) continue;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(d));
    c10::cuda::device_synchronize();
    int32_t word = 0;
    check_status(cce_layers_take_error(&word, c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(d)).stream()),
                 "cce_layers_take_error", ARGS);
    all |= word;
  }
  return all;
}

}  // namespace

void binding::bind_layers(py::module_& m) {
  using Free = py::call_guard<py::gil_scoped_release>;
  m.def("linear", &linear, Free());
  m.def("gated_linear", &gated_linear, Free());
  m.def(
      "linear_forward",
      [](const Tensor& x, const Tensor& w, const OptTensor& b, const OptTensor& r, const std::string& activation,
         const OptType& out, bool save) {
        return linear_forward(x, w, given(b), given(r), activation, out, save ? OptType(kept_type(x)) : OptType());
      },
      Free());
  m.def(
      "linear_backward",
      [](const Tensor& g, const Tensor& x, const Tensor& w, const OptTensor& z, const std::string& activation, bool dx,
         bool dw, bool db, const OptType& b_type) {
        return linear_backward(g, x, w, given(z), activation, dx, dw, db, b_type);
      },
      Free());
  m.def("gated_linear_forward", &gated_forward, Free());
  m.def("gated_linear_backward", &gated_backward, Free());
  m.def("layers_take_error", &take_error, Free());
}

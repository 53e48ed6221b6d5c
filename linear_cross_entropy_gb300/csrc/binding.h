// What the parts of the Python module _native share: errors, checks and the
// description of strided rows.
#pragma once

#include <ATen/TracerMode.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/cce_ops.h"

namespace binding {

using at::Tensor;
using OptTensor = std::optional<Tensor>;
using OptType = std::optional<at::ScalarType>;

// A status of the library; Python sees it as CCEError, and from a backward pass, which runs on the autograd engine's
// thread, as a RuntimeError of the same text.
struct StatusError : std::runtime_error {
  int status;
  std::string call;
  StatusError(int s, const std::string& c)
      : std::runtime_error(c + ": " + cce_status_string(static_cast<cce_status>(s))), status(s), call(c) {}
};

// `args`: what CCE_ERR_ARG is left to mean once the tensors have been checked here.
inline void check_status(cce_status st, const char* call, const char* args) {
  if (st != CCE_OK) throw StatusError(st, st == CCE_ERR_ARG ? std::string(call) + " (" + args + ")" : call);
}

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
inline void refuse_tracing() {
  if (at::tracer::impl::is_dispatch_enabled() ||
      c10::impl::TorchDispatchModeTLS::get_mode(c10::impl::TorchDispatchModeKey::PROXY).has_value())
    throw Unsupported("a call of this operator cannot be traced: its kernels would not be in the graph");
}

// Whether a tensor can have a tangent now.
inline bool tangents_live() { return torch::autograd::ForwardADLevel::try_get_by_idx(0) != nullptr; }

template <typename... Tensors>
void refuse_tangents(bool live, const Tensors&... tensors) {
  if (!live) return;
  const auto has = [](const Tensor& t) { return t.defined() && t._fw_grad(0).defined(); };
  if ((has(tensors) || ...))
    throw Unsupported("this operator has no forward-mode derivative: an argument has a tangent");
}

inline const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return at::toString(t);
  }
}

// The library's code of an element type, -1 for others.
inline int type_code(at::ScalarType t) {
  return t == at::kFloat ? CCE_F32 : t == at::kHalf ? CCE_F16 : t == at::kBFloat16 ? CCE_BF16 : -1;
}

inline int checked_type(const Tensor& t, const char* name) {
  const int code = type_code(t.scalar_type());
  if (code < 0) refuse(name, " must be bfloat16, float16 or float32, got ", type_name(t.scalar_type()));
  return code;
}

// The values themselves in memory: of torch's lazily negated views a copy.
inline Tensor plain(const Tensor& t) { return t.defined() && t.is_neg() ? t.resolve_neg() : t; }

inline void* pointer(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

inline void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

// -------------------------------------------------------------------- rows
// How the rows of a tensor's last dimension lie (cce_ops.h, "Rows").  Rows that
// are not at one pitch, or in runs at one pitch, or whose elements are apart
// are copied.
struct Rows {
  Tensor t;
  int64_t inner = int64_t(1) << 31, row = 0, outer = 0;
};

inline Rows rows_of(const Tensor& given) {
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

// ----------------------------------------------------------------- autograd
// The gradients of a backward pass that is itself recorded: their own gradient
// is an error, not zero.
inline void no_second_derivative(torch::autograd::variable_list& grads, const char* of) {
  if (!at::GradMode::is_enabled()) return;
  for (auto& g : grads) {
    if (!g.defined()) continue;
    auto error = std::make_shared<torch::autograd::DelayedError>(
        std::string("the ") + of + "'s gradient is not differentiable: its backward pass has no derivative", 1);
    g = g.detach().set_requires_grad(true);
    g = (*error)({g})[0];
  }
}

inline Tensor given(const OptTensor& t) { return t ? *t : Tensor(); }

// The parts, each in a file of its own.
void bind_layers(pybind11::module_& m);
void bind_optim(pybind11::module_& m);

}  // namespace binding

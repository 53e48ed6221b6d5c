// AdamW on torch tensors, over the C ABI of include/cce_optim.h: checks, the table
// of tensors, version counters.
#include <ATen/ops/copy.h>
#include <ATen/ops/empty_like.h>

#include "../../include/cce_optim.h"
#include "binding.h"

using namespace binding;

namespace {

const char* const ARGS =
    "betas must be in [0, 1), lr, eps and weight_decay finite and at least 0, step at least 1, and no tensor that is "
    "written may overlap another or be given twice";

// Whether two tensors of one shape have their elements in one order.
bool same_order(const Tensor& a, const Tensor& b) {
  for (int64_t d = 0; d < a.dim(); ++d) {
    if (a.size(d) != 1 && a.stride(d) != b.stride(d)) return false;
  }
  return true;
}

void check_tensor(const Tensor& t, const Tensor& first, const char* name) {
  if (t.layout() != at::kStrided) refuse(name, " must be dense tensors");
  if (!t.is_cuda()) refuse(name, " must be CUDA tensors (no CPU path)");
  if (t.device() != first.device()) refuse(name, " must be on one device, got ", first.device(), " and ", t.device());
}

// A tensor that is read and written beside the parameter p.
void check_beside(const Tensor& t, const Tensor& p, at::ScalarType type, const char* name) {
  check_tensor(t, p, name);
  if (t.scalar_type() != type)
    refuse(name, " must be ", type == at::kFloat ? "torch.float32" : "torch.float8_e4m3fn", ", got ",
           type_name(t.scalar_type()));
  if (t.sizes() != p.sizes() || !same_order(t, p))
    refuse(name, " must have the parameter's shape and strides, ", p.sizes(), " and ", p.strides(), ", got ", t.sizes(),
           " and ", t.strides());
  if (t.is_neg()) refuse(name, " must not be a lazily negated view");
}

void check_scale(const Tensor& t, const Tensor& p, const char* name) {
  check_tensor(t, p, name);
  const int64_t blocks = (p.numel() + CCE_ADAMW_BLOCK - 1) / CCE_ADAMW_BLOCK;
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != blocks || !t.is_contiguous() || t.is_neg())
    refuse(name, " must be contiguous float32 [", blocks, "] for a parameter of ", p.numel(), " values, got ",
           type_name(t.scalar_type()), " ", t.sizes());
}

void check_scalar(const OptTensor& t, const Tensor& first, at::ScalarType type, const char* name) {
  if (!t) return;
  check_tensor(*t, first, name);
  if (t->numel() != 1 || t->scalar_type() != type || t->is_neg())
    refuse(name, " must be one ", type == at::kFloat ? "float32" : "int64", " value, got ", type_name(t->scalar_type()),
           " ", t->sizes());
}

using List = std::vector<Tensor>;

void adamw(const List& params, const List& grads, const std::vector<OptTensor>& masters, const List& m, const List& v,
           const List& ms, const List& rs, int bits, int64_t step, const OptTensor& step_at, double lr,
           const OptTensor& lr_at, double beta1, double beta2, double eps, const std::vector<double>& decay,
           const OptTensor& norm, double max_norm, double eps_norm, uint32_t seed) {
  refuse_tracing();
  const bool live = tangents_live();
  const bool eight = bits == 8;
  const Tensor& first = params[0];
  std::vector<cce_adamw_tensor> table;
  table.reserve(params.size());
  List kept;  // gradients that had to be copied
  for (size_t i = 0; i < params.size(); ++i) {
    const Tensor& p = params[i];
    const Tensor& g = grads[i];
    const Tensor master = given(masters[i]);
    refuse_tangents(live, p, g, master);
    check_tensor(p, first, "params");
    check_tensor(g, first, "grads");
    const int p_type = checked_type(p, "params"), g_type = checked_type(g, "grads");
    if (!p.is_non_overlapping_and_dense())
      refuse("params must be dense in memory, got shape ", p.sizes(), " and strides ", p.strides());
    if (p.is_neg()) refuse("params must not be lazily negated views");
    if (g.sizes() != p.sizes()) refuse("grads must have the shapes of the params: ", g.sizes(), " for ", p.sizes());
    if (master.defined()) check_beside(master, p, at::kFloat, "masters");
    check_beside(m[i], p, eight ? at::kFloat8_e4m3fn : at::kFloat, "exp_avgs");
    check_beside(v[i], p, eight ? at::kFloat8_e4m3fn : at::kFloat, eight ? "exp_avg_rms" : "exp_avg_sqs");
    if (eight) {
      check_scale(ms[i], p, "exp_avg_scales");
      check_scale(rs[i], p, "rms_scales");
    }
    Tensor read = g;
    if (g.is_neg() || !same_order(g, p)) {
      const at::NoGradGuard no_grad;
      const c10::cuda::CUDAGuard guard(p.device());
      read = at::empty_like(p, p.options().dtype(g.scalar_type()).requires_grad(false));
      read.copy_(g);
      kept.push_back(read);
    }
    table.push_back({read.data_ptr(), p.data_ptr(), static_cast<float*>(pointer(master)), m[i].data_ptr(),
                     v[i].data_ptr(), eight ? ms[i].data_ptr<float>() : nullptr,
                     eight ? rs[i].data_ptr<float>() : nullptr, p.numel(), g_type, p_type,
                     static_cast<float>(decay[decay.size() == 1 ? 0 : i])});
  }
  check_scalar(step_at, first, at::kLong, "step");
  check_scalar(lr_at, first, at::kFloat, "lr");
  check_scalar(norm, first, at::kFloat, "grad_norm");
  const c10::cuda::CUDAGuard guard(first.device());
  const cce_adamw_options o{lr,
                            beta1,
                            beta2,
                            eps,
                            step,
                            step_at ? step_at->const_data_ptr<int64_t>() : nullptr,
                            lr_at ? lr_at->const_data_ptr<float>() : nullptr,
                            norm ? norm->const_data_ptr<float>() : nullptr,
                            static_cast<float>(max_norm),
                            static_cast<float>(eps_norm),
                            seed};
  check_status(cce_adamw_step(table.data(), static_cast<int64_t>(table.size()), bits, &o, stream_of(first)),
               "cce_adamw_step", ARGS);
  const auto wrote = [](const Tensor& t) {  // autograd learns that these were written
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  };
  for (size_t i = 0; i < params.size(); ++i) {
    wrote(params[i]);
    wrote(given(masters[i]));
    wrote(m[i]);
    wrote(v[i]);
    if (eight) {
      wrote(ms[i]);
      wrote(rs[i]);
    }
  }
}

}  // namespace

void binding::bind_optim(py::module_& m) { m.def("adamw_step", &adamw, py::call_guard<py::gil_scoped_release>()); }

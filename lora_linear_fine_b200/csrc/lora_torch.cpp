// lora_torch.cpp — the torch functions of the attention block without the
// interpreter's share of a call: checks, output tensors, stream and the C entry
// point in one step.  A smallest call is bound by its host work: 13 us through
// the interpreter (three tensors 4, the launch 4), 7 us through this.
//
// Only for the plain case: tensors of the right types and shapes, dense, on the
// current device, on its current stream.  Anything else answers None, and the
// Python function checks, refuses or takes the long way.  A status other than
// LORA_OK is returned as a number.
#include <torch/extension.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>

#include "lora_linear.h"

namespace {

using at::Tensor;
using Shape = std::initializer_list<int64_t>;

bool is(const Tensor& t, at::ScalarType type, Shape shape, int device) {
  return t.is_cuda() && t.scalar_type() == type && t.get_device() == device && t.sizes() == at::IntArrayRef(shape) &&
         t.is_contiguous();
}
bool is(const std::optional<Tensor>& t, at::ScalarType type, Shape shape, int device) {
  return !t.has_value() || is(*t, type, shape, device);
}

// The device of x if it is the current one, else -1.
int current(const Tensor& x) {
  if (!x.is_cuda() || x.dim() != 2) return -1;
  const int device = static_cast<int>(x.get_device());
  return device == c10::cuda::current_device() ? device : -1;
}

void* stream_of(int device) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}
void* ptr(const std::optional<Tensor>& t) { return t.has_value() ? t->data_ptr() : nullptr; }
float* f32(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;

py::object layer_norm(const Tensor& X, const Tensor& g, const std::optional<Tensor>& b, double eps) {
  const int dev = current(X);
  if (dev < 0) return py::none();
  const int64_t M = X.size(0), d = X.size(1);
  if (!is(X, kBf16, {M, d}, dev) || !is(g, kBf16, {d}, dev) || !is(b, kBf16, {d}, dev)) return py::none();
  Tensor Y = at::empty({M, d}, X.options());
  Tensor mean = at::empty({M}, X.options().dtype(kF32)), rstd = at::empty({M}, X.options().dtype(kF32));
  const auto st = lora_linear_layernorm_fwd(X.data_ptr(), g.data_ptr(), ptr(b), M, d, static_cast<float>(eps),
                                            Y.data_ptr(), f32(mean), f32(rstd), stream_of(dev));
  if (st != LORA_OK) return py::int_(static_cast<int>(st));
  return py::make_tuple(Y, mean, rstd);
}

py::object layer_norm_backward(const Tensor& dY, const Tensor& X, const Tensor& g, const Tensor& mean,
                               const Tensor& rstd, bool bias, const Tensor& ws) {
  const int dev = current(X);
  if (dev < 0) return py::none();
  const int64_t M = X.size(0), d = X.size(1);
  const bool wide = dY.scalar_type() == kF32;
  const size_t need = lora_linear_layernorm_workspace_size(M, d);
  if (!is(X, kBf16, {M, d}, dev) || !is(dY, wide ? kF32 : kBf16, {M, d}, dev) || !is(g, kBf16, {d}, dev) ||
      !is(mean, kF32, {M}, dev) || !is(rstd, kF32, {M}, dev) || ws.get_device() != dev ||
      static_cast<size_t>(ws.numel()) < need)
    return py::none();
  Tensor dX = at::empty({M, d}, X.options()), dg = at::empty({d}, X.options().dtype(kF32));
  std::optional<Tensor> db;
  if (bias) db = at::empty({d}, X.options().dtype(kF32));
  const auto st = lora_linear_layernorm_bwd(dY.data_ptr(), wide, X.data_ptr(), g.data_ptr(), f32(mean), f32(rstd), M,
                                            d, dX.data_ptr(), f32(dg), static_cast<float*>(ptr(db)), ws.data_ptr(),
                                            static_cast<size_t>(ws.numel()), stream_of(dev));
  if (st != LORA_OK) return py::int_(static_cast<int>(st));
  return py::make_tuple(dX, dg, db);
}

py::object rotary_tables(int64_t n_pos, int rot, double base, int scaling, double factor, double low, double high,
                         double original, double amplitude) {
  const int dev = c10::cuda::current_device();
  const lora_rotary_table_desc desc{n_pos, rot, scaling, base, factor, low, high, original, amplitude};
  const auto opt = at::TensorOptions().dtype(kF32).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev));
  Tensor cos = at::empty({n_pos, rot / 2}, opt), sin = at::empty({n_pos, rot / 2}, opt);
  const auto st = lora_linear_rotary_tables(&desc, f32(cos), f32(sin), stream_of(dev));
  if (st != LORA_OK) return py::int_(static_cast<int>(st));
  return py::make_tuple(cos, sin);
}

py::object rotary(const Tensor& Q, const std::optional<Tensor>& K, const Tensor& pos, const Tensor& cos,
                  const Tensor& sin, int64_t head_dim, int interleaved, bool inverse, const Tensor& ws) {
  const int dev = current(Q);
  if (dev < 0 || cos.dim() != 2 || (K.has_value() && K->dim() != 2) || head_dim <= 0) return py::none();
  const int64_t M = Q.size(0), q = Q.size(1), k = K.has_value() ? K->size(1) : 0, n = cos.size(0), half = cos.size(1);
  if (q % head_dim != 0 || k % head_dim != 0 || !is(Q, kBf16, {M, q}, dev) || !is(K, kBf16, {M, k}, dev) ||
      !is(pos, at::kInt, {M}, dev) || !is(cos, kF32, {n, half}, dev) || !is(sin, kF32, {n, half}, dev) ||
      ws.get_device() != dev)
    return py::none();
  Tensor Yq = at::empty({M, q}, Q.options());
  std::optional<Tensor> Yk;
  if (K.has_value()) Yk = at::empty({M, k}, Q.options());
  const lora_rotary_desc desc{M, static_cast<int32_t>(q / head_dim), static_cast<int32_t>(k / head_dim),
                              static_cast<int32_t>(head_dim), static_cast<int32_t>(2 * half), interleaved, inverse};
  const lora_rope_desc rope{static_cast<const int32_t*>(pos.data_ptr()), f32(cos), f32(sin), n,
                            static_cast<int32_t>(head_dim)};
  const auto st = lora_linear_rotary(&desc, &rope, Q.data_ptr(), ptr(K), Yq.data_ptr(), ptr(Yk), ws.data_ptr(),
                                     static_cast<size_t>(ws.numel()), stream_of(dev));
  if (st != LORA_OK) return py::int_(static_cast<int>(st));
  return py::make_tuple(Yq, Yk);
}

// Whether a call's operands fit each other and the plan; fills the descriptor.
bool attention_fits(int dev, const Tensor& Q, const Tensor& K, const Tensor& V, const Tensor& plan, int64_t rows,
                    int64_t docs, bool causal, int64_t heads, int64_t kv_heads, std::optional<double> scale,
                    double softcap, const std::optional<Tensor>& slopes, lora_attn_desc* desc) {
  if (dev < 0 || heads <= 0 || kv_heads <= 0 || Q.size(1) % heads != 0) return false;
  const int64_t M = Q.size(0), D = Q.size(1) / heads;
  if (M != rows || !is(Q, kBf16, {M, heads * D}, dev) || !is(K, kBf16, {M, kv_heads * D}, dev) ||
      !is(V, kBf16, {M, kv_heads * D}, dev) || !is(slopes, kF32, {heads}, dev) || plan.get_device() != dev)
    return false;
  *desc = {M, docs, static_cast<int32_t>(heads), static_cast<int32_t>(kv_heads), static_cast<int32_t>(D), causal,
           static_cast<float>(scale.has_value() ? *scale : 1.0 / std::sqrt(static_cast<double>(D))),
           static_cast<float>(softcap)};
  return true;
}

py::object attention(const Tensor& Q, const Tensor& K, const Tensor& V, const Tensor& plan, int64_t rows, int64_t docs,
                     bool causal, int64_t heads, int64_t kv_heads, std::optional<double> scale, double softcap,
                     const std::optional<Tensor>& slopes) {
  const int dev = current(Q);
  lora_attn_desc desc;
  if (!attention_fits(dev, Q, K, V, plan, rows, docs, causal, heads, kv_heads, scale, softcap, slopes, &desc))
    return py::none();
  Tensor O = at::empty({rows, Q.size(1)}, Q.options()), lse = at::empty({rows, heads}, Q.options().dtype(kF32));
  const auto st = lora_linear_attn_fwd(&desc, plan.data_ptr(), static_cast<size_t>(plan.numel()), Q.data_ptr(),
                                       K.data_ptr(), V.data_ptr(), static_cast<float*>(ptr(slopes)), O.data_ptr(),
                                       f32(lse), stream_of(dev));
  if (st != LORA_OK) return py::int_(static_cast<int>(st));
  return py::make_tuple(O, lse);
}

py::object attention_backward(const Tensor& dO, const Tensor& Q, const Tensor& K, const Tensor& V, const Tensor& O,
                              const Tensor& lse, const Tensor& plan, int64_t rows, int64_t docs, bool causal,
                              int64_t heads, int64_t kv_heads, std::optional<double> scale, double softcap,
                              const std::optional<Tensor>& slopes, const Tensor& ws) {
  const int dev = current(Q);
  lora_attn_desc desc;
  if (!attention_fits(dev, Q, K, V, plan, rows, docs, causal, heads, kv_heads, scale, softcap, slopes, &desc) ||
      !is(dO, kBf16, {rows, Q.size(1)}, dev) || !is(O, kBf16, {rows, Q.size(1)}, dev) ||
      !is(lse, kF32, {rows, heads}, dev) || ws.get_device() != dev ||
      static_cast<size_t>(ws.numel()) < lora_linear_attn_workspace_size(&desc))
    return py::none();
  Tensor dQ = at::empty({rows, Q.size(1)}, Q.options()), dK = at::empty({rows, K.size(1)}, Q.options()),
         dV = at::empty({rows, K.size(1)}, Q.options());
  const auto st = lora_linear_attn_bwd(&desc, plan.data_ptr(), static_cast<size_t>(plan.numel()), dO.data_ptr(),
                                       Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), f32(lse),
                                       static_cast<float*>(ptr(slopes)), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
                                       ws.data_ptr(), static_cast<size_t>(ws.numel()), stream_of(dev));
  if (st != LORA_OK) return py::int_(static_cast<int>(st));
  return py::make_tuple(dQ, dK, dV);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("layer_norm", &layer_norm);
  m.def("layer_norm_backward", &layer_norm_backward);
  m.def("rotary_tables", &rotary_tables);
  m.def("rotary", &rotary);
  m.def("attention", &attention);
  m.def("attention_backward", &attention_backward);
}

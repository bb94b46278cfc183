// fa_torch.cpp — torch side of differential attention and of the rotary
// positions: checks tensors, allocates outputs and workspaces from torch's
// allocator, fills the parameter structs of include/fa.h and calls the library
// on the current stream; and the autograd nodes of both. Their kernels take a
// few microseconds on single tokens and short sequences, which the same steps in
// Python outlast several times over. No arithmetic happens here. The library's
// entry points come as addresses (bind), so that the module follows whichever
// build of the library fa.py has loaded.
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <optional>
#include <tuple>
#include <vector>

#include "fa.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

struct Api {
  decltype(&fa_diff_fwd) fwd = nullptr;
  decltype(&fa_diff_bwd) bwd = nullptr;
  decltype(&fa_rotary) rotary = nullptr;
  decltype(&fa_diff_fwd_workspace_size) fwd_ws = nullptr;
  decltype(&fa_diff_bwd_workspace_size) bwd_ws = nullptr;
  decltype(&fa_strerror) text = nullptr;
} api;

void bind(size_t fwd, size_t bwd, size_t rotary, size_t fwd_ws, size_t bwd_ws, size_t text) {
  api.fwd = reinterpret_cast<decltype(api.fwd)>(fwd);
  api.bwd = reinterpret_cast<decltype(api.bwd)>(bwd);
  api.rotary = reinterpret_cast<decltype(api.rotary)>(rotary);
  api.fwd_ws = reinterpret_cast<decltype(api.fwd_ws)>(fwd_ws);
  api.bwd_ws = reinterpret_cast<decltype(api.bwd_ws)>(bwd_ws);
  api.text = reinterpret_cast<decltype(api.text)>(text);
}

void ok(int status, const char* what) {
  TORCH_CHECK(status == FA_OK, what, ": status ", status, " (", api.text(status), ")");
}

fa_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

int as_int(int64_t n) {
  TORCH_CHECK_VALUE(n <= INT_MAX, "a size of ", n, " is too large");
  return static_cast<int>(n);
}

// Every buffer must have the shape, dtype and device that q and k imply: the
// library gets addresses and those sizes only.
void expect(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  TORCH_CHECK_VALUE(t.sizes() == shape, name, ": expected shape ", shape, ", got ", t.sizes());
  TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, ": expected ", dtype, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.device() == like.device(), name, " is on ", t.device(), ", q on ", like.device());
}

int dtype_code(const Tensor& t) {
  TORCH_CHECK_TYPE(t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16, "fp16/bf16 tensors only, got ",
                   t.scalar_type());
  return t.scalar_type() == at::kHalf ? FA_FP16 : FA_BF16;
}

void need_cuda(const Tensor& t) {
  TORCH_CHECK_VALUE(t.is_cuda(), "tensors must live on a CUDA device (the library has no CPU path)");
}

void last_axis(const char* name, const Tensor& t) {
  TORCH_CHECK_VALUE(t.stride(-1) == 1 || t.size(-1) == 1, name, ": the last axis must be contiguous");
}

// [B, S, H, D] view.
fa_tensor flat(const char* name, const Tensor& t) {
  last_axis(name, t);
  return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

// The two maps' views of a [B, S, H, 2, D] tensor of 16-bit values.
void pair(const char* name, const Tensor& t, fa_tensor (&out)[2]) {
  last_axis(name, t);
  for (int c = 0; c < 2; ++c)
    out[c] = {static_cast<char*>(t.data_ptr()) + 2 * c * t.stride(3), t.stride(0), t.stride(1), t.stride(2)};
}

struct Sizes {
  int B, Sq, H, D, Sk, Hk, Dv, dtype;
};

Sizes sizes_of(const Tensor& q, const Tensor& k, const Tensor& v) {
  TORCH_CHECK_VALUE(q.dim() == 5 && k.dim() == 5 && v.dim() == 4 && q.size(3) == 2 && k.size(3) == 2,
                    "expected q [B, Sq, H, 2, D], k [B, Sk, Hk, 2, D] and v [B, Sk, Hk, Dv]");
  Sizes s;
  s.dtype = dtype_code(q);
  s.B = as_int(q.size(0)), s.Sq = as_int(q.size(1)), s.H = as_int(q.size(2)), s.D = as_int(q.size(4));
  s.Sk = as_int(v.size(1)), s.Hk = as_int(v.size(2)), s.Dv = as_int(v.size(3));
  expect("k", k, {s.B, s.Sk, s.Hk, 2, s.D}, q.scalar_type(), q);
  expect("v", v, {s.B, s.Sk, s.Hk, s.Dv}, q.scalar_type(), q);
  TORCH_CHECK_VALUE(s.Hk >= 1 && s.H % s.Hk == 0, s.H, " query heads cannot share ", s.Hk, " key heads evenly");
  need_cuda(q);
  return s;
}

// A tensor that the caller gives as an output: no gradient can flow through the
// write, so it is refused where autograd would record one...
void writable(const char* name, const OptTensor& t) {
  TORCH_CHECK_VALUE(!t || !t->requires_grad() || !at::GradMode::is_enabled(), name,
                    ": an output that requires a gradient (use the functions of autograd.py, or torch.no_grad)");
}
// ...and its version goes up, so that a backward pass that has saved it finds out.
void written(std::initializer_list<const OptTensor*> outputs) {
  for (const OptTensor* t : outputs)
    if (*t && !(*t)->is_inference()) (*t)->unsafeGetTensorImpl()->bump_version();
}

fa_diff_lambda lambda_of(const Tensor& lam, const Sizes& s, const Tensor& q) {
  TORCH_CHECK_VALUE(lam.dim() <= 3, "lam must be a tensor that broadcasts to [B, Sq, H]");
  const int full[3] = {s.B, s.Sq, s.H};
  int64_t ext[3] = {1, 1, 1}, st[3] = {0, 0, 0};
  const int none = 3 - static_cast<int>(lam.dim());
  for (int i = none; i < 3; ++i) {
    ext[i] = lam.size(i - none);
    st[i] = lam.stride(i - none);
    TORCH_CHECK_VALUE(ext[i] == 1 || ext[i] == full[i], "lam: ", lam.sizes(), " does not broadcast to [", s.B, ", ",
                      s.Sq, ", ", s.H, "]");
  }
  const bool wide = lam.scalar_type() == at::kFloat;
  TORCH_CHECK_TYPE(wide || lam.scalar_type() == q.scalar_type(), "lam: expected float32 or ", q.scalar_type(), ", got ",
                   lam.scalar_type());
  TORCH_CHECK_VALUE(lam.device() == q.device(), "lam is on ", lam.device(), ", q on ", q.device());
  return {lam.data_ptr(), st[0], st[1], st[2], static_cast<int>(ext[0]), static_cast<int>(ext[1]),
          static_cast<int>(ext[2]), wide ? FA_LAMBDA_FP32 : s.dtype};
}

void check_lse(const Tensor& lse, const Sizes& s, const Tensor& q) {
  expect("lse", lse, {2, s.B, s.H, s.Sq}, at::kFloat, q);
  TORCH_CHECK_VALUE(lse.is_contiguous(), "lse must be a contiguous fp32 [2, B, H, Sq] tensor");
}

// A given workspace, or a new one of `bytes`.
template <typename Params>
void set_workspace(Params& p, Tensor& hold, const OptTensor& given, size_t bytes, const Tensor& q) {
  if (given) {
    TORCH_CHECK_VALUE(given->device() == q.device() && given->is_contiguous(),
                      "workspace must be a contiguous buffer on ", q.device());
    hold = *given;
  } else if (bytes > 0) {
    hold = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
  } else {
    return;
  }
  p.workspace = hold.data_ptr();
  p.workspace_bytes = hold.nbytes();
}

std::tuple<int, Tensor, Tensor, OptTensor> diff_forward(const Tensor& q, const Tensor& k, const Tensor& v,
                                                        const Tensor& lam, bool causal, std::optional<double> scale,
                                                        const OptTensor& k_lens, bool need_o2, const OptTensor& out_,
                                                        const OptTensor& out2_, const OptTensor& lse_,
                                                        const OptTensor& workspace) {
  writable("out", out_);
  writable("out2", out2_);
  writable("lse", lse_);
  const Sizes s = sizes_of(q, k, v);
  fa_diff_fwd_params p{};
  p.lambda = lambda_of(lam, s, q);
  if (k_lens) {
    expect("k_lens", *k_lens, {s.B}, at::kInt, q);
    TORCH_CHECK_VALUE(k_lens->is_contiguous(), "k_lens must be contiguous");
    p.k_lens = static_cast<const int*>(k_lens->data_ptr());
  }
  const int64_t shape[4] = {s.B, s.Sq, s.H, s.Dv};
  if (out_) expect("out", *out_, shape, q.scalar_type(), q);
  if (out2_) expect("out2", *out2_, shape, q.scalar_type(), q);
  if (lse_) check_lse(*lse_, s, q);
  Tensor out = out_ ? *out_ : at::empty(shape, q.options());
  OptTensor out2 = out2_;
  if (!out2 && need_o2) out2 = at::empty(shape, q.options());
  Tensor lse = lse_ ? *lse_ : at::empty({2, s.B, s.H, s.Sq}, q.options().dtype(at::kFloat));
  pair("q", q, p.q);
  pair("k", k, p.k);
  p.v = flat("v", v);
  p.o = flat("out", out);
  if (out2) p.o2 = flat("out2", *out2);
  p.lse = static_cast<float*>(lse.data_ptr());
  p.B = s.B, p.H = s.H, p.Hk = s.Hk, p.Sq = s.Sq, p.Sk = s.Sk, p.D = s.D, p.Dv = s.Dv;
  p.scale = static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(s.D)));
  p.causal = causal;
  p.dtype = s.dtype;
  Tensor hold;
  const size_t bytes = workspace ? 0 : api.fwd_ws(s.B, s.H, s.Hk, s.Sq, s.Sk, s.D, s.Dv, causal);
  set_workspace(p, hold, workspace, bytes, q);
  const int status = api.fwd(&p, stream_of(q));
  if (status == FA_OK) written({&out_, &out2_, &lse_});
  return {status, out, lse, out2};
}

std::tuple<int, Tensor, Tensor, Tensor, Tensor> diff_backward(
    const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& lam, const Tensor& o, const Tensor& o2,
    const Tensor& lse, const Tensor& dO, bool causal, std::optional<double> scale, const OptTensor& dq_,
    const OptTensor& dk_, const OptTensor& dv_, const OptTensor& dlam_, const OptTensor& workspace, bool deterministic) {
  writable("dq", dq_);
  writable("dk", dk_);
  writable("dv", dv_);
  writable("dlam", dlam_);
  const Sizes s = sizes_of(q, k, v);
  fa_diff_bwd_params p{};
  p.lambda = lambda_of(lam, s, q);
  const int64_t shape[4] = {s.B, s.Sq, s.H, s.Dv};
  expect("o", o, shape, q.scalar_type(), q);
  expect("o2", o2, shape, q.scalar_type(), q);
  expect("do", dO, shape, q.scalar_type(), q);
  check_lse(lse, s, q);
  auto grad = [&](const char* name, const OptTensor& given, const Tensor& like) {
    if (!given) return at::empty(like.sizes(), like.options());
    expect(name, *given, like.sizes(), like.scalar_type(), q);
    return *given;
  };
  Tensor dq = grad("dq", dq_, q), dk = grad("dk", dk_, k), dv = grad("dv", dv_, v), dlam = grad("dlam", dlam_, lam);
  TORCH_CHECK_VALUE(dlam.is_contiguous(), "dlam must be contiguous");
  pair("q", q, p.q);
  pair("k", k, p.k);
  p.v = flat("v", v);
  p.o = flat("o", o);
  p.o2 = flat("o2", o2);
  p.dO = flat("do", dO);
  pair("dq", dq, p.dq);
  pair("dk", dk, p.dk);
  p.dv = flat("dv", dv);
  p.lse = static_cast<const float*>(lse.data_ptr());
  p.dlambda = dlam.data_ptr();
  p.B = s.B, p.H = s.H, p.Hk = s.Hk, p.Sq = s.Sq, p.Sk = s.Sk, p.D = s.D, p.Dv = s.Dv;
  p.scale = static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(s.D)));
  p.causal = causal;
  p.dtype = s.dtype;
  p.deterministic = deterministic;
  Tensor hold;
  const size_t bytes = workspace ? 0 : api.bwd_ws(s.B, s.H, s.Hk, s.Sq, s.Sk, s.D, s.Dv, causal, deterministic);
  set_workspace(p, hold, workspace, bytes, q);
  const int status = api.bwd(&p, stream_of(q));
  if (status == FA_OK) written({&dq_, &dk_, &dv_, &dlam_});
  return {status, dq, dk, dv, dlam};
}

// What one launch turns: a [B, S, heads, D] view and where it goes.
struct Turn {
  Tensor in, out;
};

void check_heads(const char* name, const Tensor& t) {
  TORCH_CHECK_VALUE(t.dim() == 4 || t.dim() == 5, name, " must be [B, S, heads, D] or [B, S, H, 2, D]");
}

// Whether the head and map axes of a [B, S, H, 2, D] tensor are one run of heads.
bool one_run(const Tensor& t) {
  return t.dim() == 4 || t.size(2) <= 1 || t.stride(2) == t.size(3) * t.stride(3);
}

Tensor joined(const Tensor& t) {
  if (t.dim() == 4) return t;
  return t.as_strided({t.size(0), t.size(1), t.size(2) * t.size(3), t.size(4)},
                      {t.stride(0), t.stride(1), t.stride(3), t.stride(4)});
}

// [B, S, heads, D] in one piece, [B, S, H, 2, D] with its maps as neighbouring
// heads, or map by map where the strides of either side do not allow that.
std::vector<Turn> turns_of(const char* name, const Tensor& in, const Tensor& out) {
  if (one_run(in) && one_run(out)) return {{joined(in), joined(out)}};
  // (What the library finds wrong with one map's views it finds with the first's.)
  TORCH_CHECK_VALUE(in.stride(3) % 8 == 0 && out.stride(3) % 8 == 0, name,
                    ": the strides must be multiples of 8 elements");
  std::vector<Turn> turns;
  for (int64_t c = 0; c < in.size(3); ++c) turns.push_back({in.select(3, c), out.select(3, c)});
  return turns;
}

std::tuple<int, Tensor, OptTensor> rotary(const Tensor& q, const OptTensor& k, const Tensor& positions,
                                          const Tensor& inv_freq, const std::optional<std::vector<int64_t>>& sections,
                                          bool interleaved, bool inverse, const OptTensor& out_q_,
                                          const OptTensor& out_k_) {
  writable("out_q", out_q_);
  writable("out_k", out_k_);
  fa_rotary_params p{};
  p.dtype = dtype_code(q);
  need_cuda(q);
  check_heads("q", q);
  const int64_t B = q.size(0), S = q.size(1), D = q.size(-1);
  if (k) {
    check_heads("k", *k);
    std::vector<int64_t> shape = k->sizes().vec();
    shape[0] = B, shape[1] = S, shape.back() = D;
    expect("k", *k, shape, q.scalar_type(), q);
  }
  TORCH_CHECK_VALUE(positions.dim() == 2 || positions.dim() == 3, "positions: expected [axes, B, S] or [B, S]");
  const Tensor pos = positions.dim() == 2 ? positions.unsqueeze(0) : positions;
  TORCH_CHECK_VALUE(pos.size(1) == B && pos.size(2) == S, "positions: expected [axes, ", B, ", ", S, "], got ",
                    positions.sizes());
  TORCH_CHECK_TYPE(pos.scalar_type() == at::kInt || pos.scalar_type() == at::kLong,
                   "positions: expected int32 or int64, got ", pos.scalar_type());
  TORCH_CHECK_TYPE(inv_freq.scalar_type() == at::kFloat || inv_freq.scalar_type() == at::kDouble,
                   "inv_freq: expected float32 or float64, got ", inv_freq.scalar_type());
  TORCH_CHECK_VALUE(inv_freq.dim() == 1 && inv_freq.is_contiguous(), "inv_freq must be a contiguous [pairs] tensor");
  TORCH_CHECK_VALUE(pos.device() == q.device(), "positions is on ", pos.device(), ", q on ", q.device());
  TORCH_CHECK_VALUE(inv_freq.device() == q.device(), "inv_freq is on ", inv_freq.device(), ", q on ", q.device());
  const int64_t axes = pos.size(0), pairs = inv_freq.size(0);
  const std::vector<int64_t> parts = sections ? *sections : std::vector<int64_t>{pairs};
  TORCH_CHECK_VALUE(static_cast<int64_t>(parts.size()) == axes && axes >= 1 && axes <= FA_ROTARY_MAX_AXES,
                    "sections: expected one entry for each of 1 to ", FA_ROTARY_MAX_AXES, " axes, got ", parts.size(),
                    " for ", axes);
  int64_t sum = 0;
  for (size_t i = 0; i < parts.size(); ++i) {
    TORCH_CHECK_VALUE(parts[i] >= 0 && parts[i] <= pairs, "sections ", parts, " do not add up to inv_freq's ", pairs,
                      " pairs");
    sum += parts[i];
    p.sections[i] = static_cast<int>(parts[i]);
  }
  TORCH_CHECK_VALUE(sum == pairs, "sections ", parts, " do not add up to inv_freq's ", pairs, " pairs");
  TORCH_CHECK_VALUE(2 * pairs <= D, pairs, " pairs do not fit into ", D, " columns");
  if (out_q_) expect("out_q", *out_q_, q.sizes(), q.scalar_type(), q);
  TORCH_CHECK_VALUE(k || !out_k_, "out_k without k");
  if (out_k_) expect("out_k", *out_k_, k->sizes(), q.scalar_type(), q);
  Tensor out_q = out_q_ ? *out_q_ : at::empty(q.sizes(), q.options());
  OptTensor out_k = out_k_;
  if (k && !out_k) out_k = at::empty(k->sizes(), q.options());
  const std::vector<Turn> qs = turns_of("q", q, out_q);
  const std::vector<Turn> ks = k ? turns_of("k", *k, *out_k) : std::vector<Turn>();
  p.positions = pos.data_ptr();
  p.pos_stride_axis = pos.stride(0), p.pos_stride_b = pos.stride(1), p.pos_stride_s = pos.stride(2);
  p.pos_int64 = pos.scalar_type() == at::kLong;
  p.inv_freq = inv_freq.data_ptr();
  p.inv_freq_fp64 = inv_freq.scalar_type() == at::kDouble;
  p.axes = as_int(axes);
  p.B = as_int(B), p.S = as_int(S), p.D = as_int(D);
  p.interleaved = interleaved;
  p.inverse = inverse;
  // One launch, unless maps lie apart. The first one checks every view but for
  // the further maps' places, so that a refused call writes nothing.
  int status = FA_OK;
  for (size_t i = 0; i < std::max(qs.size(), ks.size()) && status == FA_OK; ++i) {
    const Turn& t = i < qs.size() ? qs[i] : ks[i];
    p.q = flat("q", t.in);
    p.q_out = flat("out_q", t.out);
    p.H = as_int(t.in.size(2));
    p.Hk = 0;
    if (i < qs.size() && i < ks.size()) {
      p.k = flat("k", ks[i].in);
      p.k_out = flat("out_k", ks[i].out);
      p.Hk = as_int(ks[i].in.size(2));
    }
    status = api.rotary(&p, stream_of(q));
  }
  if (status == FA_OK) written({&out_q_, &out_k_});
  return {status, out_q, out_k};
}

// ------------------------------------------------------------------ autograd
// `t`, or a dense copy if its strides, alignment or an expanded axis keep the
// kernels from reading it.
Tensor ready(const Tensor& t) {
  bool fine = reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && t.dim() > 0 &&
              (t.stride(-1) == 1 || t.size(-1) == 1);
  for (int64_t i = 0; fine && i + 1 < t.dim(); ++i)
    fine = t.size(i) == 1 || (t.stride(i) > 0 && t.stride(i) % 8 == 0);
  return fine ? t : t.clone(at::MemoryFormat::Contiguous);
}

// Gradients of a backward pass that is itself recorded: they may be used, but a
// further derivative through them raises.
torch::autograd::variable_list once(torch::autograd::variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  auto node = std::make_shared<torch::autograd::DelayedError>(
      "trying to differentiate twice a function that is differentiable once", static_cast<int64_t>(grads.size()));
  return (*node)(std::move(grads));
}

struct DiffAttention : torch::autograd::Function<DiffAttention> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& q_, const Tensor& k_, const Tensor& v_,
                        const Tensor& lam, bool causal, double scale, bool deterministic, bool need) {
    const c10::DeviceGuard guard(q_.device());
    const Tensor q = ready(q_), k = ready(k_), v = ready(v_);
    auto [status, o, lse, o2] =
        diff_forward(q, k, v, lam, causal, scale, std::nullopt, need, std::nullopt, std::nullopt, std::nullopt,
                     std::nullopt);
    ok(status, "fa_diff_fwd");
    if (need) {
      ctx->save_for_backward({q, k, v, lam, o, *o2, lse});
      ctx->saved_data["causal"] = causal;
      ctx->saved_data["scale"] = scale;
      ctx->saved_data["deterministic"] = deterministic;
    }
    return o;
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto t = ctx->get_saved_variables();
    const c10::DeviceGuard guard(t[0].device());
    torch::autograd::variable_list out;
    {
      const at::AutoGradMode off(false);
      auto [status, dq, dk, dv, dlam] =
          diff_backward(t[0], t[1], t[2], t[3], t[4], t[5], t[6], ready(grads[0]), ctx->saved_data["causal"].toBool(),
                        ctx->saved_data["scale"].toDouble(), std::nullopt, std::nullopt, std::nullopt, std::nullopt,
                        std::nullopt, ctx->saved_data["deterministic"].toBool());
      ok(status, "fa_diff_bwd");
      out = {dq, dk, dv, dlam};
    }
    out = once(std::move(out));
    out.resize(8);
    return out;
  }
};

bool recorded(std::initializer_list<const Tensor*> inputs) {
  if (!at::GradMode::is_enabled()) return false;
  for (const Tensor* t : inputs)
    if (t->defined() && t->requires_grad()) return true;
  return false;
}

Tensor diff_attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& lam, bool causal, double scale,
                      bool deterministic) {
  return DiffAttention::apply(q, k, v, lam, causal, scale, deterministic, recorded({&q, &k, &v, &lam}));
}

struct Rotary : torch::autograd::Function<Rotary> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& q,
                                                const OptTensor& k, const Tensor& positions, const Tensor& inv_freq,
                                                const std::optional<std::vector<int64_t>>& sections, bool interleaved) {
    const c10::DeviceGuard guard(q.device());
    auto [status, oq, ok_] = rotary(ready(q), k ? OptTensor(ready(*k)) : OptTensor(), positions, inv_freq, sections,
                                    interleaved, false, std::nullopt, std::nullopt);
    ok(status, "fa_rotary");
    ctx->save_for_backward({positions, inv_freq});
    if (sections) ctx->saved_data["sections"] = *sections;
    ctx->saved_data["interleaved"] = interleaved;
    if (ok_) return {oq, *ok_};
    return {oq};
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto t = ctx->get_saved_variables();
    const c10::DeviceGuard guard(t[0].device());
    std::optional<std::vector<int64_t>> sections;
    if (ctx->saved_data.count("sections")) sections = ctx->saved_data["sections"].toIntVector();
    torch::autograd::variable_list out;
    {
      const at::AutoGradMode off(false);
      auto [status, gq, gk] = rotary(ready(grads[0]), grads.size() > 1 ? OptTensor(ready(grads[1])) : OptTensor(), t[0],
                                     t[1], sections, ctx->saved_data["interleaved"].toBool(), true, std::nullopt,
                                     std::nullopt);
      ok(status, "fa_rotary");
      out = {gq};
      if (gk) out.push_back(*gk);
    }
    out = once(std::move(out));
    out.resize(6);
    return out;
  }
};

std::tuple<Tensor, OptTensor> rotary_attached(const Tensor& q, const OptTensor& k, const Tensor& positions,
                                              const Tensor& inv_freq,
                                              const std::optional<std::vector<int64_t>>& sections, bool interleaved) {
  TORCH_CHECK_VALUE(!recorded({&inv_freq}), "inv_freq requires a gradient: there is none in the frequencies");
  auto out = Rotary::apply(q, k, positions, inv_freq, sections, interleaved);
  return {out[0], out.size() > 1 ? OptTensor(out[1]) : OptTensor()};
}

}  // namespace

PYBIND11_MODULE(_fa_torch, m) {
  m.def("bind", &bind);
  m.def("diff_forward", &diff_forward);
  m.def("diff_backward", &diff_backward);
  m.def("rotary", &rotary);
  m.def("diff_attention", &diff_attention, pybind11::call_guard<pybind11::gil_scoped_release>());
  m.def("rotary_attached", &rotary_attached, pybind11::call_guard<pybind11::gil_scoped_release>());
}

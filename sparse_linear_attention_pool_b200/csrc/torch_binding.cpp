// PyTorch binding of the operators beside the attention (modules rotary and
// prompt): argument checks, output tensors and autograd around the C ABI of
// include/sla.h. Compiled, because a decoding step calls these for every layer:
// the same marshalling in Python took 11 to 20 us a call, several times the
// kernels' own time on single tokens.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <cstring>
#include <limits>
#include <string>
#include <vector>

#include "../../include/sla.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;
using OptInt = std::optional<int64_t>;

struct StatusError : std::exception {
  int status;
  std::string text;
  StatusError(int s, const char* call) : status(s), text(call) {}
  const char* what() const noexcept override { return text.c_str(); }
};
void check_status(sla_status st, const char* call) {
  if (st != SLA_OK) throw StatusError(st, call);
}

void* stream_of(const Tensor& x) { return c10::cuda::getCurrentCUDAStream(x.device().index()).stream(); }

// A plan and a table keep memory between calls, allocated on the stream that was current when they
// were made (`home`). A call on another stream tells the allocator: dropped right after the call,
// the memory is not handed out again before that stream is done with it.
cudaStream_t home_of(const Tensor& kept) {
  return kept.is_cuda() ? c10::cuda::getCurrentCUDAStream(kept.device().index()).stream() : nullptr;
}
void record_use(const Tensor& kept, cudaStream_t home) {
  const auto now = c10::cuda::getCurrentCUDAStream(kept.device().index());
  if (now.stream() != home) kept.record_stream(now);
}

// A caller's scratch: the library sees its address and its bytes alone.
void check_workspace(const OptTensor& w, const at::Device& device) {
  TORCH_CHECK_VALUE(!w || (w->is_cuda() && w->device() == device && w->is_contiguous()),
                    "workspace: a contiguous tensor on the inputs' device");
}

// The autograd functions here have no forward-mode derivative. A dual tensor need not require grad,
// so it is looked for by its tangent.
template <typename... Ts>
void refuse_tangents(const char* call, const Ts&... xs) {
  const bool dual = ((xs.defined() && xs._fw_grad(/*level=*/0).defined()) || ...);
  TORCH_CHECK_NOT_IMPLEMENTED(!dual, call, " has no forward-mode derivative");
}

// A kernel wrote to a caller's tensor: autograd is told, as by torch's own operations in place, so that
// a backward which saved the old values is refused.
void written(const Tensor& out) {
  if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
}
// What the call writes there would not be what autograd holds it for.
void check_out(const Tensor& out) {
  TORCH_CHECK_VALUE(!(at::GradMode::is_enabled() && out.requires_grad()), "out: a tensor that requires grad");
}

// ---------------------------------------------------------------------------
// rotary positions
// ---------------------------------------------------------------------------

struct RopeTable {
  Tensor turns;
  OptTensor axis;
  float gain;
  int rot_dim, layout, n_axes;
  cudaStream_t home;
};
using TablePtr = std::shared_ptr<RopeTable>;

int dtype_code(const Tensor& x, const char* what) {
  switch (x.scalar_type()) {
    case at::kBFloat16: return SLA_BF16;
    case at::kHalf: return SLA_FP16;
    case at::kFloat: return SLA_FP32;
    default: TORCH_CHECK_VALUE(false, what, ": bfloat16, float16 or float32, not ", x.scalar_type());
  }
}

void check_heads(const Tensor& x, const char* what) {
  TORCH_CHECK_VALUE(x.dim() == 3 || x.dim() == 4, what, ": [B, H, N, d] or [T, H, d], not ", x.sizes());
  TORCH_CHECK_VALUE(x.is_cuda(), what, ": a CUDA tensor");
}
void check_like(const Tensor& x, const Tensor& like, const char* what) {
  check_heads(x, what);
  TORCH_CHECK_VALUE(x.dim() == like.dim() && x.scalar_type() == like.scalar_type() && x.device() == like.device() &&
                        x.size(-1) == like.size(-1),
                    what, ": dtype, device, head size or rank differ");
}

Tensor with_rows(const Tensor& x) { return x.stride(-1) == 1 || x.size(-1) == 1 ? x : x.contiguous(); }
int64_t batch(const Tensor& x) { return x.dim() == 4 ? x.size(0) : 1; }
int64_t tokens(const Tensor& x) { return x.dim() == 4 ? x.size(2) : x.size(0); }

sla_heads heads_of(const Tensor& x) {
  if (x.dim() == 4) return {x.data_ptr(), int(x.size(1)), x.stride(0), x.stride(1), x.stride(2)};
  return {x.data_ptr(), int(x.size(1)), 0, x.stride(1), x.stride(0)};
}

// The tokens that a call takes; sizes that the library's int parameters would cut are refused.
int64_t count_of(const Tensor& x, const OptInt& N, const char* call) {
  const int64_t n = tokens(x);
  TORCH_CHECK_VALUE(!N || (*N >= 0 && *N <= n), "N must be 0 .. ", n);
  const int64_t taken = N ? *N : n;
  for (int64_t size : {batch(x), taken, x.size(1), x.size(-1)})
    if (size > std::numeric_limits<int>::max()) throw StatusError(SLA_ERR_UNSUPPORTED, call);
  return taken;
}

// The rotation of a call, positions checked against B and N; `pos` may be undefined.
sla_rope_spec spec_of(const RopeTable& t, const Tensor& pos, int64_t B, int64_t N, const at::Device& device) {
  TORCH_CHECK_VALUE(t.turns.device() == device, "the table is on another device");
  record_use(t.turns, t.home);
  if (t.axis) record_use(*t.axis, t.home);
  sla_rope_spec s{};
  s.turns = static_cast<const unsigned long long*>(t.turns.data_ptr());
  s.axis = t.axis ? static_cast<const unsigned char*>(t.axis->data_ptr()) : nullptr;
  s.gain = t.gain;
  s.pos_bits = 32;
  s.rot_dim = t.rot_dim;
  s.layout = t.layout;
  s.n_axes = t.n_axes;
  if (!pos.defined()) return s;
  TORCH_CHECK_VALUE((pos.scalar_type() == at::kInt || pos.scalar_type() == at::kLong) && pos.device() == device,
                    "positions: int32 or int64 on the tensors' device");
  int64_t at = 0;
  if (t.n_axes > 1) {
    TORCH_CHECK_VALUE(pos.dim() >= 2 && pos.size(0) == t.n_axes, "positions: [", t.n_axes, ", (B,) N] for ", t.n_axes,
                      " axes");
    s.pos_axis = pos.stride(0);
    at = 1;
  }
  const int64_t left = pos.dim() - at;
  const bool fits = (left == 1 || (left == 2 && (pos.size(at) == 1 || pos.size(at) == B))) && pos.size(-1) >= N;
  TORCH_CHECK_VALUE(fits, "positions: one for each of ", B, " x ", N, " tokens, not ", pos.sizes());
  if (left == 2 && pos.size(at) > 1) s.pos_b = pos.stride(at);
  s.pos_n = pos.stride(-1);
  s.pos = pos.data_ptr();
  s.pos_bits = pos.scalar_type() == at::kInt ? 32 : 64;
  return s;
}

Tensor out_for(const Tensor& x, const OptTensor& out, const OptInt& rows, int64_t N) {
  if (!out) {
    if (!rows) return at::empty(x.sizes(), x.options());
    TORCH_CHECK_VALUE(x.dim() == 4, "rows is for [B, H, N, d] tensors");
    TORCH_CHECK_VALUE(*rows >= N, "rows must be at least N");
    return at::empty({x.size(0), x.size(1), *rows, x.size(3)}, x.options());
  }
  check_like(*out, x, "out");
  TORCH_CHECK_VALUE(out->size(1) == x.size(1) && batch(*out) == batch(x) && tokens(*out) >= N, "out: shape ",
                    out->sizes(), " does not take the result");
  TORCH_CHECK_VALUE(out->stride(-1) == 1 || out->size(-1) == 1, "out: rows must be contiguous");
  return *out;
}

// Rows behind N of a gradient are zero.
void zero_tail(const Tensor& t, int64_t N) {
  if (tokens(t) > N) t.narrow(t.dim() == 4 ? 2 : 0, N, tokens(t) - N).zero_();
}

Tensor run_rope(const Tensor& x, const RopeTable& table, const Tensor& pos, int64_t N, Tensor out, bool inverse) {
  const int64_t B = batch(x);
  const sla_rope_spec s = spec_of(table, pos, B, N, x.device());
  const int code = dtype_code(x, "x");
  if (N > 0 && x.numel() > 0) {
    const Tensor in = with_rows(x);
    const sla_heads hx = heads_of(in), hy = heads_of(out);
    check_status(sla_rope(&hx, &hy, B, N, x.size(-1), code, &s, inverse, stream_of(x)), "sla_rope");
  }
  return out;
}

struct RopeMeta : torch::CustomClassHolder {
  TablePtr table;
  Tensor pos;  // or undefined; also saved, so that a change in place before the backward is noticed
  int64_t N = 0;
  OptInt rows;
  bool inverse = false;
  bool zero_behind = false;  // rows behind N of the result are zero: it is a gradient
  float eps = 0.0f;
  std::vector<int64_t> sizes;
};
using RopeMetaPtr = c10::intrusive_ptr<RopeMeta>;
RopeMetaPtr rope_meta(AutogradContext* ctx) {
  return c10::static_intrusive_pointer_cast<RopeMeta>(ctx->saved_data["meta"].toCapsule());
}

struct RopeFunction : torch::autograd::Function<RopeFunction> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, RopeMetaPtr meta) {
    ctx->saved_data["meta"] = c10::IValue::make_capsule(meta);
    if (meta->pos.defined()) ctx->save_for_backward({meta->pos});
    const Tensor y = run_rope(x, *meta->table, meta->pos, meta->N, out_for(x, {}, meta->rows, meta->N), meta->inverse);
    if (meta->zero_behind) zero_tail(y, meta->N);
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const auto meta = rope_meta(ctx);
    const Tensor pos = meta->pos.defined() ? ctx->get_saved_variables()[0] : Tensor(), dy = grads[0];
    if (at::GradMode::is_enabled() && dy.requires_grad()) {  // linear: its gradient is the same rotation
      auto back = c10::make_intrusive<RopeMeta>();
      back->table = meta->table;
      back->pos = pos;
      back->N = meta->N;
      back->inverse = !meta->inverse;
      back->zero_behind = true;
      back->sizes = meta->sizes;
      TORCH_CHECK(!meta->rows, "rope with rows is not differentiable twice");
      return {apply(dy, back), Tensor()};
    }
    const Tensor dx = at::empty(meta->sizes, dy.options());
    run_rope(dy, *meta->table, pos, meta->N, dx, !meta->inverse);
    zero_tail(dx, meta->N);
    return {dx, Tensor()};
  }
};

Tensor rope(const Tensor& x, const TablePtr& table, const OptTensor& positions, const OptInt& N, const OptInt& rows,
            const OptTensor& out, bool inverse) {
  check_heads(x, "x");
  dtype_code(x, "x");
  refuse_tangents("rope", x, out ? *out : Tensor());
  c10::cuda::CUDAGuard guard(x.device());
  const int64_t n = count_of(x, N, "sla_rope");
  const Tensor pos = positions ? *positions : Tensor();
  if (at::GradMode::is_enabled() && x.requires_grad()) {
    TORCH_CHECK_VALUE(!out, "out cannot be given for a tensor that requires grad");
    auto meta = c10::make_intrusive<RopeMeta>();
    meta->table = table;
    meta->N = n;
    meta->rows = rows;
    meta->inverse = inverse;
    meta->sizes = x.sizes().vec();
    meta->pos = pos;
    return RopeFunction::apply(x, meta);
  }
  if (out) check_out(*out);
  const Tensor y = run_rope(x, *table, pos, n, out_for(x, out, rows, n), inverse);
  if (out) written(y);
  return y;
}

// ---------------------------------------------------------------------------
// norms of queries and keys with the rotation
// ---------------------------------------------------------------------------

void check_pair(const Tensor& q, const Tensor& k, const Tensor& wq, const Tensor& wk) {
  check_heads(q, "q");
  dtype_code(q, "q");
  check_like(k, q, "k");
  TORCH_CHECK_VALUE(batch(q) == batch(k) && tokens(q) == tokens(k), "q and k hold different tokens");
  for (const Tensor* w : {&wq, &wk})
    TORCH_CHECK_VALUE(w->dim() == 1 && w->size(0) == q.size(-1) && w->device() == q.device(),
                      "wq and wk: [d] on the tensors' device");
  TORCH_CHECK_VALUE(wq.scalar_type() == wk.scalar_type() &&
                        (wq.scalar_type() == q.scalar_type() || wq.scalar_type() == at::kFloat),
                    "wq and wk: the tensors' dtype, or float32");
}

const sla_rope_spec* spec_or_null(const TablePtr& table, const Tensor& pos, int64_t B, int64_t N, const at::Device& dev,
                                  sla_rope_spec* s) {
  if (!table) {
    TORCH_CHECK_VALUE(!pos.defined(), "positions without a table");
    return nullptr;
  }
  *s = spec_of(*table, pos, B, N, dev);
  return s;
}

void run_norm(const Tensor& q, const Tensor& k, const Tensor& wq, const Tensor& wk, const TablePtr& table,
              const Tensor& pos, float eps, int64_t N, const Tensor& yq, const Tensor& yk) {
  const int64_t B = batch(q);
  sla_rope_spec s{};
  const sla_rope_spec* spec = spec_or_null(table, pos, B, N, q.device(), &s);
  if (B == 0 || N == 0) return;
  const Tensor a = with_rows(q), b = with_rows(k), u = wq.contiguous(), v = wk.contiguous();
  const sla_heads hq = heads_of(a), hk = heads_of(b), oq = heads_of(yq), ok = heads_of(yk);
  check_status(sla_qk_norm_rope(&hq, &hk, u.data_ptr(), v.data_ptr(), u.scalar_type() == at::kFloat, eps, &oq, &ok, B,
                                N, q.size(-1), dtype_code(q, "q"), spec, stream_of(q)),
               "sla_qk_norm_rope");
}

std::tuple<Tensor, Tensor, Tensor, Tensor> run_norm_backward(const Tensor& q, const Tensor& k, const Tensor& wq,
                                                             const Tensor& wk, const Tensor& dyq, const Tensor& dyk,
                                                             const TablePtr& table, const Tensor& pos, float eps,
                                                             int64_t N, bool need_w, const OptTensor& workspace) {
  const int64_t B = batch(q), d = q.size(-1);
  const Tensor dq = at::empty(q.sizes(), q.options()), dk = at::empty(k.sizes(), k.options());
  Tensor dwq, dwk;
  if (need_w) {
    dwq = at::empty(wq.sizes(), wq.options());
    dwk = at::empty(wk.sizes(), wk.options());
  }
  sla_rope_spec s{};
  const sla_rope_spec* spec = spec_or_null(table, pos, B, N, q.device(), &s);
  if (B > 0 && N > 0) {
    const size_t need = sla_qk_norm_rope_backward_workspace_size(B, N, q.size(1), k.size(1), d);
    const Tensor ws = workspace ? *workspace : at::empty({int64_t(need)}, q.options().dtype(at::kByte));
    const Tensor a = with_rows(q), b = with_rows(k), g = with_rows(dyq), h = with_rows(dyk), u = wq.contiguous(),
                 v = wk.contiguous();
    const sla_heads hq = heads_of(a), hk = heads_of(b), gq = heads_of(g), gk = heads_of(h), oq = heads_of(dq),
                    ok = heads_of(dk);
    check_status(sla_qk_norm_rope_backward(&hq, &hk, u.data_ptr(), v.data_ptr(), u.scalar_type() == at::kFloat, eps,
                                           &gq, &gk, &oq, &ok, need_w ? dwq.data_ptr() : nullptr,
                                           need_w ? dwk.data_ptr() : nullptr, B, N, d, dtype_code(q, "q"), spec,
                                           ws.data_ptr(), ws.nbytes(), stream_of(q)),
                 "sla_qk_norm_rope_backward");
  } else if (need_w) {
    dwq.zero_();
    dwk.zero_();
  }
  zero_tail(dq, N);
  zero_tail(dk, N);
  return {dq, dk, dwq, dwk};
}

struct NormFunction : torch::autograd::Function<NormFunction> {
  static variable_list forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& wq,
                               const Tensor& wk, RopeMetaPtr meta) {
    ctx->saved_data["meta"] = c10::IValue::make_capsule(meta);
    if (meta->pos.defined())
      ctx->save_for_backward({q, k, wq, wk, meta->pos});
    else
      ctx->save_for_backward({q, k, wq, wk});
    const Tensor yq = out_for(q, {}, meta->rows, meta->N), yk = out_for(k, {}, meta->rows, meta->N);
    run_norm(q, k, wq, wk, meta->table, meta->pos, meta->eps, meta->N, yq, yk);
    return {yq, yk};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    TORCH_CHECK(!at::GradMode::is_enabled(), "qk_norm_rope is not differentiable twice");
    const auto meta = rope_meta(ctx);
    const auto saved = ctx->get_saved_variables();
    const bool need_w = ctx->needs_input_grad(2) || ctx->needs_input_grad(3);
    // (torch hands over zeros for an output that nothing used)
    auto [dq, dk, dwq, dwk] =
        run_norm_backward(saved[0], saved[1], saved[2], saved[3], grads[0], grads[1], meta->table,
                          meta->pos.defined() ? saved[4] : Tensor(), meta->eps, meta->N, need_w, {});
    return {dq, dk, dwq, dwk, Tensor()};
  }
};

std::tuple<Tensor, Tensor> qk_norm_rope(const Tensor& q, const Tensor& k, const Tensor& wq, const Tensor& wk,
                                        const TablePtr& table, const OptTensor& positions, double eps, const OptInt& N,
                                        const OptInt& rows, const std::optional<std::tuple<Tensor, Tensor>>& out) {
  check_pair(q, k, wq, wk);
  refuse_tangents("qk_norm_rope", q, k, wq, wk, out ? std::get<0>(*out) : Tensor(), out ? std::get<1>(*out) : Tensor());
  c10::cuda::CUDAGuard guard(q.device());
  const int64_t n = count_of(q, N, "sla_qk_norm_rope");
  count_of(k, N, "sla_qk_norm_rope");
  const Tensor pos = positions ? *positions : Tensor();
  if (at::GradMode::is_enabled() &&
      (q.requires_grad() || k.requires_grad() || wq.requires_grad() || wk.requires_grad())) {
    TORCH_CHECK_VALUE(!out, "out cannot be given for tensors that require grad");
    auto meta = c10::make_intrusive<RopeMeta>();
    meta->table = table;
    meta->N = n;
    meta->rows = rows;
    meta->eps = float(eps);
    meta->pos = pos;
    const auto y = NormFunction::apply(q, k, wq, wk, meta);
    return {y[0], y[1]};
  }
  if (out) check_out(std::get<0>(*out)), check_out(std::get<1>(*out));
  const Tensor yq = out_for(q, out ? OptTensor(std::get<0>(*out)) : OptTensor(), rows, n);
  const Tensor yk = out_for(k, out ? OptTensor(std::get<1>(*out)) : OptTensor(), rows, n);
  run_norm(q, k, wq, wk, table, pos, float(eps), n, yq, yk);
  if (out) written(yq), written(yk);
  return {yq, yk};
}

std::tuple<Tensor, Tensor, OptTensor, OptTensor> qk_norm_rope_backward(
    const Tensor& q, const Tensor& k, const Tensor& wq, const Tensor& wk, const Tensor& dyq, const Tensor& dyk,
    const TablePtr& table, const OptTensor& positions, double eps, const OptInt& N, bool want_w,
    const OptTensor& workspace) {
  at::NoGradGuard no_grad;
  check_workspace(workspace, q.device());
  check_pair(q, k, wq, wk);
  c10::cuda::CUDAGuard guard(q.device());
  const int64_t n = count_of(q, N, "sla_qk_norm_rope_backward");
  count_of(k, N, "sla_qk_norm_rope_backward");
  const Tensor* pairs[2][2] = {{&dyq, &q}, {&dyk, &k}};
  for (auto& p : pairs) {
    check_like(*p[0], *p[1], "dyq and dyk");
    TORCH_CHECK_VALUE(p[0]->size(1) == p[1]->size(1) && batch(*p[0]) == batch(*p[1]) && tokens(*p[0]) >= n,
                      "dyq and dyk: shape ", p[0]->sizes());
  }
  auto [dq, dk, dwq, dwk] = run_norm_backward(q, k, wq, wk, dyq, dyk, table, positions ? *positions : Tensor(),
                                              float(eps), n, want_w, workspace);
  return {dq, dk, want_w ? OptTensor(dwq) : OptTensor(), want_w ? OptTensor(dwk) : OptTensor()};
}

// ---------------------------------------------------------------------------
// packed prompt attention
// ---------------------------------------------------------------------------

struct PromptPlan {
  std::vector<unsigned long long> host;  // 8-byte aligned
  size_t bytes;
  Tensor device;
  cudaStream_t home;
  int64_t Tq, Tk, Hq, Hkv, d;
  bool grad;
  int64_t forward_workspace, backward_workspace;
};
using PlanPtr = std::shared_ptr<PromptPlan>;

// x's rows as the kernels take them: whole 16-byte pieces at 16-byte steps (copied where x's are not).
sla_rows rows_of(Tensor& x, int64_t T, int64_t H, const PromptPlan& p, const char* what) {
  TORCH_CHECK_VALUE(x.scalar_type() == at::kBFloat16 && x.is_cuda(), what, ": a bfloat16 CUDA tensor");
  TORCH_CHECK_VALUE(x.dim() == 3 && x.size(0) >= T && x.size(1) == H && x.size(2) == p.d, what, ": [>= ", T, ", ", H,
                    ", ", p.d, "] for this plan, not ", x.sizes());
  TORCH_CHECK_VALUE(x.device() == p.device.device(), what, ": on another device than the plan");
  const int64_t row = x.stride(0), head = x.stride(1);
  if (x.stride(2) != 1 || (T > 1 && (row <= 0 || row % 8 != 0)) || (H > 1 && (head <= 0 || head % 8 != 0)) ||
      reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 != 0)
    x = x.clone(at::MemoryFormat::Contiguous);
  return {x.data_ptr(), x.stride(0), x.stride(1)};
}

sla_rows out_rows(Tensor& out, const Tensor& x, int64_t T, int64_t H, const PromptPlan& p, const char* what) {
  if (!out.defined()) {
    out = at::empty(x.sizes(), x.options());
  } else {
    TORCH_CHECK_VALUE(out.scalar_type() == x.scalar_type() && out.device() == x.device() && out.dim() == 3 &&
                          out.size(0) >= T && out.size(1) == H && out.size(2) == p.d && out.stride(2) == 1,
                      what, ": a [>= ", T, ", ", H, ", ", p.d, "] bfloat16 tensor with contiguous rows");
  }
  return {out.data_ptr(), out.stride(0), out.stride(1)};
}

std::tuple<Tensor, Tensor, Tensor> run_forward(Tensor q, Tensor k, Tensor v, const PromptPlan& p, Tensor out,
                                               bool want_lse, bool want_rest, const OptTensor& workspace) {
  const sla_rows rq = rows_of(q, p.Tq, p.Hq, p, "q"), rk = rows_of(k, p.Tk, p.Hkv, p, "k"),
                 rv = rows_of(v, p.Tk, p.Hkv, p, "v");
  const sla_rows ro = out_rows(out, q, p.Tq, p.Hq, p, "out");
  record_use(p.device, p.home);
  Tensor lse, rest, ws;
  if (want_rest) rest = at::empty({p.Tq, p.Hq, p.d}, q.options());
  if (want_lse) lse = at::empty({p.Tq, p.Hq}, q.options().dtype(at::kFloat));
  if (workspace)
    ws = *workspace;
  else if (p.forward_workspace > 0)
    ws = at::empty({p.forward_workspace}, q.options().dtype(at::kByte));
  check_status(sla_prompt_forward(&rq, &rk, &rv, &ro, want_lse ? lse.data_ptr<float>() : nullptr,
                                  want_rest ? rest.data_ptr() : nullptr, p.host.data(), p.bytes,
                                  p.device.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr,
                                  ws.defined() ? ws.nbytes() : 0, stream_of(q)),
               "sla_prompt_forward");
  return {out, lse, rest};
}

void check_grad(const PromptPlan& p) {
  TORCH_CHECK_VALUE(p.grad, "the plan was made without the backward pass (grad=True)");
}

std::tuple<Tensor, Tensor, Tensor> run_backward(Tensor q, Tensor k, Tensor v, Tensor o, const Tensor& lse,
                                                const Tensor& rest, Tensor dO, const PromptPlan& p, Tensor dq, Tensor dk, Tensor dv,
                                                const OptTensor& workspace) {
  const sla_rows rq = rows_of(q, p.Tq, p.Hq, p, "q"), rk = rows_of(k, p.Tk, p.Hkv, p, "k"),
                 rv = rows_of(v, p.Tk, p.Hkv, p, "v"), ro = rows_of(o, p.Tq, p.Hq, p, "o"),
                 rg = rows_of(dO, p.Tq, p.Hq, p, "do");
  TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.dim() == 2 && lse.size(0) == p.Tq && lse.size(1) == p.Hq &&
                        lse.is_contiguous() && lse.device() == p.device.device(),
                    "lse: prompt_forward's [", p.Tq, ", ", p.Hq, "] float32");
  if (rest.defined())
    TORCH_CHECK_VALUE(rest.scalar_type() == at::kBFloat16 && rest.is_contiguous() && rest.dim() == 3 &&
                          rest.size(0) == p.Tq && rest.size(1) == p.Hq && rest.size(2) == p.d &&
                          rest.device() == p.device.device(),
                      "rest: prompt_forward's [", p.Tq, ", ", p.Hq, ", ", p.d, "] bfloat16");
  record_use(p.device, p.home);
  const bool fresh = !dq.defined();
  const sla_rows oq = out_rows(dq, q, p.Tq, p.Hq, p, "dq"), ok = out_rows(dk, k, p.Tk, p.Hkv, p, "dk"),
                 ov = out_rows(dv, v, p.Tk, p.Hkv, p, "dv");
  const Tensor ws = workspace ? *workspace : at::empty({p.backward_workspace}, q.options().dtype(at::kByte));
  check_status(sla_prompt_backward(&rq, &rk, &rv, &ro, lse.data_ptr<float>(),
                                   rest.defined() ? rest.data_ptr() : nullptr, &rg, &oq, &ok, &ov, p.host.data(),
                                   p.bytes, p.device.data_ptr(), ws.data_ptr(), ws.nbytes(), stream_of(q)),
               "sla_prompt_backward");
  if (fresh) {
    zero_tail(dq, p.Tq);
    zero_tail(dk, p.Tk);
    zero_tail(dv, p.Tk);
  }
  return {dq, dk, dv};
}

struct PlanMeta : torch::CustomClassHolder {
  PlanPtr plan;
  explicit PlanMeta(PlanPtr p) : plan(std::move(p)) {}
};

struct PromptFunction : torch::autograd::Function<PromptFunction> {
  static Tensor forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v,
                        c10::intrusive_ptr<PlanMeta> meta) {
    auto [o, lse, rest] = run_forward(q, k, v, *meta->plan, Tensor(), true, true, {});
    ctx->saved_data["plan"] = c10::IValue::make_capsule(meta);
    ctx->save_for_backward({q, k, v, o, lse, rest});
    return o;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    TORCH_CHECK(!at::GradMode::is_enabled(), "prompt_attention is not differentiable twice");
    const auto meta = c10::static_intrusive_pointer_cast<PlanMeta>(ctx->saved_data["plan"].toCapsule());
    const auto s = ctx->get_saved_variables();
    auto [dq, dk, dv] = run_backward(s[0], s[1], s[2], s[3], s[4], s[5], grads[0], *meta->plan, Tensor(), Tensor(),
                                     Tensor(), {});
    return {dq, dk, dv, Tensor()};
  }
};

std::tuple<Tensor, OptTensor, OptTensor> prompt_forward(const Tensor& q, const Tensor& k, const Tensor& v,
                                                        const PlanPtr& plan, const OptTensor& out, bool want_lse,
                                                        bool want_rest, const OptTensor& workspace) {
  if (out) check_out(*out);
  check_workspace(workspace, plan->device.device());
  at::NoGradGuard no_grad;
  c10::OptionalDeviceGuard guard(plan->device.device());
  auto [o, lse, rest] = run_forward(q, k, v, *plan, out ? *out : Tensor(), want_lse, want_rest, workspace);
  if (out) written(o);
  return {o, want_lse ? OptTensor(lse) : OptTensor(), want_rest ? OptTensor(rest) : OptTensor()};
}

std::tuple<Tensor, Tensor, Tensor> prompt_backward(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o,
                                                   const Tensor& lse, const OptTensor& rest, const Tensor& dO,
                                                   const PlanPtr& plan,
                                                   const std::optional<std::tuple<Tensor, Tensor, Tensor>>& out,
                                                   const OptTensor& workspace) {
  Tensor dq, dk, dv;
  if (out) {
    std::tie(dq, dk, dv) = *out;
    for (const Tensor* t : {&dq, &dk, &dv}) check_out(*t);
  }
  check_workspace(workspace, plan->device.device());
  at::NoGradGuard no_grad;
  check_grad(*plan);
  c10::OptionalDeviceGuard guard(plan->device.device());
  const auto made = run_backward(q, k, v, o, lse, rest ? *rest : Tensor(), dO, *plan, dq, dk, dv, workspace);
  if (out) written(dq), written(dk), written(dv);
  return made;
}

Tensor prompt_attention(const Tensor& q, const Tensor& k, const Tensor& v, const PlanPtr& plan) {
  refuse_tangents("prompt_attention", q, k, v);
  c10::OptionalDeviceGuard guard(plan->device.device());
  if (at::GradMode::is_enabled() && (q.requires_grad() || k.requires_grad() || v.requires_grad())) {
    check_grad(*plan);
    return PromptFunction::apply(q, k, v, c10::make_intrusive<PlanMeta>(plan));
  }
  return std::get<0>(run_forward(q, k, v, *plan, Tensor(), false, false, {}));
}

}  // namespace

PYBIND11_MODULE(_sla_torch, m) {
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const StatusError& e) {
      const py::object cls = py::module_::import("sparse_linear_attention_pool_b200").attr("SLAError");
      PyErr_SetObject(cls.ptr(), cls(e.status, e.text).ptr());
    }
  });
  py::class_<RopeTable, TablePtr>(m, "RopeTable")
      .def(py::init([](Tensor turns, OptTensor axis, double gain, int rot_dim, int layout, int n_axes) {
        return std::make_shared<RopeTable>(RopeTable{turns, axis, float(gain), rot_dim, layout, n_axes, home_of(turns)});
      }));
  py::class_<PromptPlan, PlanPtr>(m, "PromptPlan")
      .def(py::init([](py::bytes host, Tensor device, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t d,
                       bool grad) {
        const std::string raw = host;
        auto p = std::make_shared<PromptPlan>();
        p->host.resize((raw.size() + 7) / 8);
        std::memcpy(p->host.data(), raw.data(), raw.size());
        p->bytes = raw.size();
        p->device = device;
        p->home = home_of(device);
        p->Tq = Tq;
        p->Tk = Tk;
        p->Hq = Hq;
        p->Hkv = Hkv;
        p->d = d;
        p->grad = grad;
        p->forward_workspace = int64_t(sla_prompt_workspace_size(p->host.data()));
        p->backward_workspace = int64_t(sla_prompt_backward_workspace_size(p->host.data()));
        return p;
      }))
      .def_readonly("forward_workspace", &PromptPlan::forward_workspace)
      .def_readonly("backward_workspace", &PromptPlan::backward_workspace);
  m.def("rope", &rope);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_backward", &qk_norm_rope_backward);
  m.def("prompt_forward", &prompt_forward);
  m.def("prompt_backward", &prompt_backward);
  m.def("prompt_attention", &prompt_attention);
}

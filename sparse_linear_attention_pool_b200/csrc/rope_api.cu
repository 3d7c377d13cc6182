// C ABI of the rotary-position operators (declared in include/sla.h): argument
// validation and the arguments of the kernels in rope_kernels.cu.
#include <math.h>

#include "rope.cuh"

using namespace sla;

namespace {

int dtype_size(int dtype) { return dtype == SLA_FP32 ? 4 : 2; }

sla_status check_sizes(int B, int N, int d, int dtype) {
  if (B < 1 || N < 1 || d < 2) return SLA_ERR_INVALID_ARG;
  if (dtype != SLA_BF16 && dtype != SLA_FP16 && dtype != SLA_FP32) return SLA_ERR_INVALID_ARG;
  if (d > 256 || d % 2 != 0) return SLA_ERR_UNSUPPORTED;
  if ((long long)B * N >= (1LL << 31) - 256) return SLA_ERR_UNSUPPORTED;
  return SLA_OK;
}

// Rows of an output are distinct when every axis of more than one entry steps past the axes
// inside it: sorted by stride, each stride is at least the reach of the smaller ones.
bool distinct_rows(const sla_heads& t, int B, int N, int d) {
  long long stride[3] = {t.sb, t.sh, t.sn}, size[3] = {B, t.H, N};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(size[i], size[j]);
      }
  long long reach = d;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (stride[i] < reach) return false;
    reach = stride[i] * (size[i] - 1) + reach;
  }
  return true;
}

sla_status check_heads(const sla_heads* t, int H, int B, int N, int d, int dtype, bool output) {
  if (t == nullptr || t->base == nullptr || t->H < 1) return SLA_ERR_INVALID_ARG;
  if (H > 0 && t->H != H) return SLA_ERR_INVALID_ARG;
  if (t->sb < 0 || t->sh < 0 || t->sn < 0) return SLA_ERR_INVALID_ARG;
  if (t->H > 65535) return SLA_ERR_UNSUPPORTED;  // a grid axis
  if (reinterpret_cast<uintptr_t>(t->base) % dtype_size(dtype) != 0) return SLA_ERR_ALIGNMENT;
  if (output && !distinct_rows(*t, B, N, d)) return SLA_ERR_INVALID_ARG;
  return SLA_OK;
}

sla_status check_rope(const sla_rope_spec* r, int d) {
  if (r == nullptr) return SLA_OK;
  if (r->rot_dim < 0 || r->rot_dim > d || r->rot_dim % 2 != 0) return SLA_ERR_INVALID_ARG;
  if (r->layout != SLA_ROPE_INTERLEAVED && r->layout != SLA_ROPE_HALF) return SLA_ERR_INVALID_ARG;
  if (r->rot_dim > 0 && r->turns == nullptr) return SLA_ERR_INVALID_ARG;
  if (r->n_axes < 1 || r->n_axes > 255) return SLA_ERR_INVALID_ARG;
  if (!isfinite(r->gain)) return SLA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(r->turns) % 8 != 0) return SLA_ERR_ALIGNMENT;
  if (r->pos != nullptr) {
    if (r->pos_bits != 32 && r->pos_bits != 64) return SLA_ERR_INVALID_ARG;
    if (r->pos_axis < 0 || r->pos_b < 0 || r->pos_n < 0) return SLA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(r->pos) % (r->pos_bits / 8) != 0) return SLA_ERR_ALIGNMENT;
  }
  return SLA_OK;
}

void set_rope(RopeArgs& a, const sla_rope_spec* r, int B, int N, int d, int dtype) {
  a.B = B;
  a.N = N;
  a.d = d;
  a.dtype = dtype;
  a.inv_d = 1.0f / float(d);
  a.gain = 1.0f;
  a.half = 1;
  if (r == nullptr) return;
  a.rot = r->rot_dim;
  a.half = r->layout == SLA_ROPE_HALF;
  a.turns = r->turns;
  a.axis = r->axis;
  a.pos = r->pos;
  a.pos64 = r->pos_bits == 64;
  a.pos_axis = r->pos_axis;
  a.pos_b = r->pos_b;
  a.pos_n = r->pos_n;
  a.gain = r->gain;
  a.n_axes = r->n_axes;
}

void set_in(RopeTensor& t, const sla_heads& x) {
  t.x = x.base;
  t.H = x.H;
  t.xb = x.sb;
  t.xh = x.sh;
  t.xn = x.sn;
}
void set_out(RopeTensor& t, const sla_heads& y) {
  t.y = y.base;
  t.yb = y.sb;
  t.yh = y.sh;
  t.yn = y.sn;
}
void set_grad(RopeTensor& t, const sla_heads& g) {
  t.dy = g.base;
  t.gb = g.sb;
  t.gh = g.sh;
  t.gn = g.sn;
}

sla_status check_weights(const void* wq, const void* wk, int w_f32, float eps, int dtype) {
  if (wq == nullptr || wk == nullptr) return SLA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || isinf(eps)) return SLA_ERR_INVALID_ARG;
  const size_t size = (w_f32 || dtype == SLA_FP32) ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(wq) % size != 0 || reinterpret_cast<uintptr_t>(wk) % size != 0)
    return SLA_ERR_ALIGNMENT;
  return SLA_OK;
}

sla_status done(cudaError_t e) { return e == cudaSuccess ? SLA_OK : SLA_ERR_CUDA; }

}  // namespace

extern "C" {

sla_status sla_rope(const sla_heads* x, const sla_heads* y, int B, int N, int d, int dtype,
                    const sla_rope_spec* rope, int inverse, void* stream) {
  sla_status st = check_sizes(B, N, d, dtype);
  if (st == SLA_OK && rope == nullptr) st = SLA_ERR_INVALID_ARG;
  if (st == SLA_OK) st = check_heads(x, 0, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(y, x->H, B, N, d, dtype, true);
  if (st == SLA_OK) st = check_rope(rope, d);
  if (st != SLA_OK) return st;
  RopeArgs a{};
  set_rope(a, rope, B, N, d, dtype);
  a.inverse = inverse != 0;
  set_in(a.t[0], *x);
  set_out(a.t[0], *y);
  return done(launch_rope(a, 1, false, static_cast<cudaStream_t>(stream)));
}

sla_status sla_qk_norm_rope(const sla_heads* q, const sla_heads* k, const void* wq, const void* wk, int w_f32,
                            float eps, const sla_heads* yq, const sla_heads* yk, int B, int N, int d, int dtype,
                            const sla_rope_spec* rope, void* stream) {
  sla_status st = check_sizes(B, N, d, dtype);
  if (st == SLA_OK) st = check_heads(q, 0, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(k, 0, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(yq, q->H, B, N, d, dtype, true);
  if (st == SLA_OK) st = check_heads(yk, k->H, B, N, d, dtype, true);
  if (st == SLA_OK) st = check_rope(rope, d);
  if (st == SLA_OK) st = check_weights(wq, wk, w_f32, eps, dtype);
  if (st != SLA_OK) return st;
  RopeArgs a{};
  set_rope(a, rope, B, N, d, dtype);
  a.eps = eps;
  a.w_f32 = w_f32 != 0 || dtype == SLA_FP32;
  set_in(a.t[0], *q);
  set_in(a.t[1], *k);
  set_out(a.t[0], *yq);
  set_out(a.t[1], *yk);
  a.t[0].w = wq;
  a.t[1].w = wk;
  return done(launch_rope(a, 2, false, static_cast<cudaStream_t>(stream)));
}

size_t sla_qk_norm_rope_backward_workspace_size(int B, int N, int Hq, int Hk, int d) {
  if (check_sizes(B, N, d, SLA_BF16) != SLA_OK || Hq < 1 || Hk < 1 || Hq > 65535 || Hk > 65535) return 0;
  return size_t(rope_bwd_blocks((long long)B * N)) * d * sizeof(float);
}

sla_status sla_qk_norm_rope_backward(const sla_heads* q, const sla_heads* k, const void* wq, const void* wk,
                                     int w_f32, float eps, const sla_heads* dyq, const sla_heads* dyk,
                                     const sla_heads* dq, const sla_heads* dk, void* dwq, void* dwk, int B, int N,
                                     int d, int dtype, const sla_rope_spec* rope, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  sla_status st = check_sizes(B, N, d, dtype);
  if (st == SLA_OK) st = check_heads(q, 0, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(k, 0, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(dyq, q->H, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(dyk, k->H, B, N, d, dtype, false);
  if (st == SLA_OK) st = check_heads(dq, q->H, B, N, d, dtype, true);
  if (st == SLA_OK) st = check_heads(dk, k->H, B, N, d, dtype, true);
  if (st == SLA_OK) st = check_rope(rope, d);
  if (st == SLA_OK) st = check_weights(wq, wk, w_f32, eps, dtype);
  if (st != SLA_OK) return st;
  if ((dwq == nullptr) != (dwk == nullptr)) return SLA_ERR_INVALID_ARG;
  const size_t size = (w_f32 || dtype == SLA_FP32) ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(dwq) % size != 0 || reinterpret_cast<uintptr_t>(dwk) % size != 0)
    return SLA_ERR_ALIGNMENT;
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
      workspace_bytes < sla_qk_norm_rope_backward_workspace_size(B, N, q->H, k->H, d))
    return SLA_ERR_WORKSPACE;
  RopeArgs a{};
  set_rope(a, rope, B, N, d, dtype);
  a.inverse = 1;
  a.eps = eps;
  a.w_f32 = w_f32 != 0 || dtype == SLA_FP32;
  const sla_heads *in[2] = {q, k}, *grad[2] = {dyq, dyk}, *out[2] = {dq, dk};
  const void* w[2] = {wq, wk};
  void* dw[2] = {dwq, dwk};
  for (int i = 0; i < 2; ++i) {
    set_in(a.t[i], *in[i]);
    set_grad(a.t[i], *grad[i]);
    set_out(a.t[i], *out[i]);
    a.t[i].w = w[i];
    a.t[i].dw = dw[i];
  }
  a.partial = static_cast<float*>(workspace);
  return done(launch_rope(a, 2, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

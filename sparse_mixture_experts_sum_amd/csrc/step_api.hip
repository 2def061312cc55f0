// Host side of the layer norms' and the update step's entry points (include/moe.h): argument
// checks and launches on the caller's stream. No allocation, no synchronisation.
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "moe.h"
#include "step_kernels.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31, kMaxWidth = 1 << 20;
constexpr int64_t kMaxNormWidth = 16384;
constexpr int64_t kMaxSide = 1 << 18, kMaxShortSide = 16384;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
template <typename... P>
bool all_aligned16(const P*... p) {
  return (aligned(p, 16) && ...);
}
bool bad_dtype(int32_t t) { return t != MOE_FP32 && t != MOE_BF16; }
moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

moe_status check_norm(const moe_layer_norm_shape* s) {
  if (!s) return MOE_ERR_NULL_ARG;
  if (bad_dtype(s->dtype)) return MOE_ERR_BAD_SHAPE;
  if (s->T < 0 || s->T >= kMaxRows || s->d < 1 || s->d > kMaxWidth) return MOE_ERR_BAD_SHAPE;
  if (!(s->eps > 0.f) || !isfinite(s->eps) || !isfinite(s->residual_scale)) return MOE_ERR_BAD_SHAPE;
  return s->d % 8 || s->d > kMaxNormWidth ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_orth(const moe_orthogonalize_shape* s) {
  if (!s) return MOE_ERR_NULL_ARG;
  if (bad_dtype(s->dtype) || s->m < 1 || s->n < 1 || s->E < 1 || s->steps < 1) return MOE_ERR_BAD_SHAPE;
  if (!isfinite(s->a) || !isfinite(s->b) || !isfinite(s->c) || !(s->eps >= 0.f) || !isfinite(s->eps))
    return MOE_ERR_BAD_SHAPE;
  if (s->m > kMaxSide || s->n > kMaxSide || (s->m > kMaxShortSide && s->n > kMaxShortSide) || s->E > 64 ||
      s->steps > 64)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

OrthArgs orth_args(const moe_orthogonalize_shape& s) {
  OrthArgs o{};
  o.m = s.m;
  o.n = s.n;
  o.E = s.E;
  o.bf16 = s.dtype == MOE_BF16;
  o.steps = s.steps;
  o.a = s.a;
  o.b = s.b;
  o.c = s.c;
  o.eps = s.eps;
  return o;
}

// What both entry points do once their own arguments are checked.
moe_status orthogonalize(OrthArgs& o, int32_t dtype, const void* g, void* out, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
  const uintptr_t size = dtype == MOE_BF16 ? 2 : 4;
  if (!g || !out || !ws) return MOE_ERR_NULL_ARG;
  if (!aligned(g, size) || !aligned(out, size) || !aligned(ws, 256)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < orthogonalize_workspace(o)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  o.g = g;
  o.out = out;
  o.ws = static_cast<char*>(ws);
  return launched(launch_orthogonalize(o, stream));
}

}  // namespace

extern "C" {

moe_status moe_layer_norm(const moe_layer_norm_shape* shape, const void* x, const float* y,
                          const float* gamma, const float* beta, void* out, void* u, float* mean,
                          float* rstd, hipStream_t stream) {
  const moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  const moe_layer_norm_shape& s = *shape;
  // (with rows: a tensor without elements may have no address)
  if (s.T > 0 && !y && out) return MOE_ERR_BAD_SHAPE;
  if (!all_aligned16(x, y, gamma, beta, out, u)) return MOE_ERR_MISALIGNED;
  if (s.T == 0) return MOE_OK;
  if (!x || !gamma || !u || (y && !out)) return MOE_ERR_NULL_ARG;
  LayerNormArgs m{};
  m.x = x;
  m.y = y;
  m.gamma = gamma;
  m.beta = beta;
  m.out = out;
  m.u = u;
  m.mean = mean;
  m.rstd = rstd;
  m.T = s.T;
  m.d = (int)s.d;
  m.bf16 = s.dtype == MOE_BF16;
  m.eps = s.eps;
  m.scale = s.residual_scale;
  return launched(launch_layer_norm(m, stream));
}

moe_status moe_layer_norm_backward_workspace_size(const moe_layer_norm_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL_ARG;
  const moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  *bytes = layer_norm_grad_workspace(shape->T, (int)shape->d) * sizeof(float);
  return MOE_OK;
}

moe_status moe_layer_norm_backward(const moe_layer_norm_shape* shape, const void* out,
                                   const void* d_u, const void* d_out, const float* mean,
                                   const float* rstd, const float* gamma, void* dx, void* dy,
                                   float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  size_t need = 0;
  const moe_status st = moe_layer_norm_backward_workspace_size(shape, &need);
  if (st != MOE_OK) return st;
  const moe_layer_norm_shape& s = *shape;
  if (!all_aligned16(out, d_u, d_out, gamma, dx, dy, ws)) return MOE_ERR_MISALIGNED;
  if (s.T > 0 && (!out || !d_u || !mean || !rstd || !gamma)) return MOE_ERR_NULL_ARG;
  if (need && !ws) return MOE_ERR_NULL_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  LayerNormGradArgs m{};
  m.out = out;
  m.d_u = d_u;
  m.d_out = d_out;
  m.mean = mean;
  m.rstd = rstd;
  m.gamma = gamma;
  m.dx = dx;
  m.dy = dy;
  m.dgamma = dgamma;
  m.dbeta = dbeta;
  m.partial = static_cast<float*>(ws);
  m.T = s.T;
  m.d = (int)s.d;
  m.bf16 = s.dtype == MOE_BF16;
  m.scale = s.residual_scale;
  return launched(launch_layer_norm_grad(m, stream));
}

moe_status moe_orthogonalize_workspace_size(const moe_orthogonalize_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL_ARG;
  const moe_status st = check_orth(shape);
  if (st != MOE_OK) return st;
  *bytes = orthogonalize_workspace(orth_args(*shape));
  return MOE_OK;
}

moe_status moe_orthogonalize(const moe_orthogonalize_shape* shape, const void* g, void* out,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_orth(shape);
  if (st != MOE_OK) return st;
  OrthArgs o = orth_args(*shape);
  return orthogonalize(o, shape->dtype, g, out, ws, ws_bytes, stream);
}

moe_status moe_muon_update(const moe_orthogonalize_shape* shape, const moe_muon_params* params,
                           void* w, const void* g, float* m, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  const moe_status st = check_orth(shape);
  if (st != MOE_OK) return st;
  if (!params || !m) return MOE_ERR_NULL_ARG;
  const moe_muon_params& p = *params;
  if (!isfinite(p.lr) || !isfinite(p.momentum) || !isfinite(p.weight_decay) || !isfinite(p.scale) ||
      (p.nesterov != 0 && p.nesterov != 1))
    return MOE_ERR_BAD_SHAPE;
  if (!aligned(m, 4)) return MOE_ERR_MISALIGNED;
  OrthArgs o = orth_args(*shape);
  o.momentum = m;
  o.nesterov = p.nesterov;
  o.mu = p.momentum;
  o.keep = (float)(1.0 - (double)p.lr * (double)p.weight_decay);
  o.rate = (float)((double)p.lr * (double)p.scale);
  return orthogonalize(o, shape->dtype, g, w, ws, ws_bytes, stream);
}

}  // extern "C"

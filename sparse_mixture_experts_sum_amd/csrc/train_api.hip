// Host side of the training entry points (include/moe.h, "Training"): argument checks and
// launches on the caller's stream. No allocation, no synchronisation.
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "moe.h"
#include "train_kernels.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31, kMaxWidth = 1 << 20;
constexpr int64_t kMaxNormWidth = 16384;
// The grouped products count rows past a group's end, by up to a tile or a ring turn, in int32.
constexpr int64_t kMaxMatmulRows = kMaxRows - (1 << 16);

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P>
bool all_aligned16(const P*... p) {
  return (aligned16(p) && ...);
}
bool bad_dtype(int32_t t) { return t != MOE_FP32 && t != MOE_BF16; }
bool bad_flag(int32_t v) { return v != 0 && v != 1; }
moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Rows are read in 16-byte pieces.
moe_status check_width(int64_t n, int32_t dtype) {
  if (n < 1 || n > kMaxWidth) return MOE_ERR_BAD_SHAPE;
  return n % (dtype == MOE_BF16 ? 8 : 4) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_matmul(const moe_matmul_shape* s) {
  if (!s) return MOE_ERR_NULL_ARG;
  if (s->form != MOE_MATMUL_NN && s->form != MOE_MATMUL_NT && s->form != MOE_MATMUL_TN)
    return MOE_ERR_BAD_SHAPE;
  if (bad_dtype(s->dtype) || bad_dtype(s->out_dtype) || bad_flag(s->accumulate))
    return MOE_ERR_BAD_SHAPE;
  if (s->R < 0 || s->R > kMaxMatmulRows || s->rows_a < 0 || s->rows_a >= kMaxRows || s->E < 1)
    return MOE_ERR_BAD_SHAPE;
  if (s->form == MOE_MATMUL_TN && (s->rows_b < 0 || s->rows_b >= kMaxRows))
    return MOE_ERR_BAD_SHAPE;
  moe_status st = check_width(s->K, s->dtype);
  if (st == MOE_OK) st = check_width(s->N, s->dtype);
  if (st != MOE_OK) return st;
  if (s->E > 64) return MOE_ERR_UNSUPPORTED;
  if (s->out_dtype == MOE_BF16 && (s->dtype != MOE_BF16 || s->accumulate))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

MatmulArgs matmul_args(const moe_matmul_shape& s) {
  MatmulArgs m{};
  m.R = s.R;
  m.rows_a = s.rows_a;
  m.rows_b = s.rows_b;
  m.K = s.K;
  m.N = s.N;
  m.E = s.E;
  m.form = s.form;
  m.bf16_in = s.dtype == MOE_BF16;
  m.bf16_out = s.out_dtype == MOE_BF16;
  m.accumulate = s.accumulate;
  return m;
}

moe_status check_route(const moe_shape* s) {
  if (!s) return MOE_ERR_NULL_ARG;
  if (bad_dtype(s->dtype)) return MOE_ERR_BAD_SHAPE;
  if (s->mode == MOE_EXPERT_CHOICE) return MOE_ERR_UNSUPPORTED;
  if (s->mode != MOE_TOKEN_CHOICE && s->mode != MOE_TOKEN_CHOICE_CAPACITY) return MOE_ERR_BAD_SHAPE;
  if (s->T < 0 || s->T >= kMaxRows || s->d_model < 1 || s->d_model > kMaxWidth || s->E < 1)
    return MOE_ERR_BAD_SHAPE;
  if (s->d_model % 64 || s->E > 64) return MOE_ERR_UNSUPPORTED;
  if (s->k < 1 || s->k > s->E || bad_flag(s->renormalize)) return MOE_ERR_BAD_SHAPE;
  if (s->k > 8) return MOE_ERR_UNSUPPORTED;
  if (s->T * (int64_t)s->k >= kMaxRows) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

moe_status check_norm(const moe_norm_shape* s) {
  if (!s) return MOE_ERR_NULL_ARG;
  if (bad_dtype(s->dtype) || s->gate < MOE_GATE_NONE || s->gate > MOE_GATE_TOKEN)
    return MOE_ERR_BAD_SHAPE;
  if (s->T < 0 || s->T >= kMaxRows || s->d < 1 || s->d > kMaxWidth) return MOE_ERR_BAD_SHAPE;
  if (!(s->eps > 0.f) || !isfinite(s->eps) || !isfinite(s->residual_scale)) return MOE_ERR_BAD_SHAPE;
  if (s->d % 8 || s->d > kMaxNormWidth) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_grouped_matmul_workspace_size(const moe_matmul_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL_ARG;
  const moe_status st = check_matmul(shape);
  if (st != MOE_OK) return st;
  *bytes = shape->R > 0 ? grouped_matmul_workspace(matmul_args(*shape)) : 0;
  return MOE_OK;
}

moe_status moe_grouped_matmul(const moe_matmul_shape* shape, const void* a, const void* b,
                              const int32_t* offsets, const int32_t* gather_a,
                              const int32_t* gather_b, void* out, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  moe_status st = check_matmul(shape);
  if (st != MOE_OK) return st;
  const moe_matmul_shape& s = *shape;
  const bool tn = s.form == MOE_MATMUL_TN;
  if (gather_b && !tn) return MOE_ERR_UNSUPPORTED;
  if (!gather_a && s.rows_a != s.R) return MOE_ERR_BAD_SHAPE;
  if (tn && !gather_b && s.rows_b != s.R) return MOE_ERR_BAD_SHAPE;
  // a gathered row has to exist
  if (s.R > 0 && (s.rows_a < 1 || (tn && s.rows_b < 1))) return MOE_ERR_BAD_SHAPE;
  if (!all_aligned16(a, b, out, ws)) return MOE_ERR_MISALIGNED;
  if (s.R > 0 && (!a || !b || !offsets || !out)) return MOE_ERR_NULL_ARG;
  if (s.R == 0) {
    if (!tn || s.accumulate) return MOE_OK;
    if (!out) return MOE_ERR_NULL_ARG;
    return launched(launch_fill_zero(out, (size_t)s.E * s.K * s.N * (s.out_dtype == MOE_BF16 ? 2 : 4),
                                     stream));
  }
  MatmulArgs m = matmul_args(s);
  const size_t need = grouped_matmul_workspace(m);
  if (need && !ws) return MOE_ERR_NULL_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  m.a = a;
  m.b = b;
  m.offsets = offsets;
  m.gather_a = gather_a;
  m.gather_b = gather_b;
  m.out = out;
  return launched(launch_grouped_matmul(m, static_cast<float*>(ws), stream));
}

moe_status moe_swiglu_backward(const moe_swiglu_shape* shape, const void* g, const void* u,
                               const void* dh, const float* w, const int32_t* src,
                               const int32_t* pos, const int32_t* offsets, void* dg, void* du,
                               void* hw, float* dw, hipStream_t stream) {
  if (!shape) return MOE_ERR_NULL_ARG;
  const moe_swiglu_shape& s = *shape;
  if (bad_dtype(s.dtype) || s.R < 0 || s.R >= kMaxRows) return MOE_ERR_BAD_SHAPE;
  const moe_status st = check_width(s.f, s.dtype);
  if (st != MOE_OK) return st;
  if (offsets) {
    if (s.E < 1) return MOE_ERR_BAD_SHAPE;
    if (s.E > 64) return MOE_ERR_UNSUPPORTED;
  }
  if (pos) {
    if (s.T < 0 || s.T >= kMaxRows || s.k < 1 || (s.R > 0 && s.T < 1)) return MOE_ERR_BAD_SHAPE;
    if (s.k > 8) return MOE_ERR_UNSUPPORTED;
    if (s.R > 0 && (!w || !src)) return MOE_ERR_NULL_ARG;
  }
  if (!all_aligned16(g, u, dh, dg, du, hw)) return MOE_ERR_MISALIGNED;
  if (s.R == 0) return MOE_OK;
  if (!g || !u || !dh) return MOE_ERR_NULL_ARG;
  SwigluGradArgs m{};
  m.g = g;
  m.u = u;
  m.dh = dh;
  m.w = w;
  m.src = src;
  m.pos = pos;
  m.offsets = offsets;
  m.dg = dg;
  m.du = du;
  m.hw = hw;
  m.dw = dw;
  m.R = s.R;
  m.f = s.f;
  m.T = s.T;
  m.k = s.k;
  m.E = s.E;
  m.bf16 = s.dtype == MOE_BF16;
  return launched(launch_swiglu_grad(m, stream));
}

moe_status moe_route_backward_workspace_size(const moe_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL_ARG;
  const moe_status st = check_route(shape);
  if (st != MOE_OK) return st;
  *bytes = route_grad_workspace(shape->T, shape->d_model, shape->E);
  return MOE_OK;
}

moe_status moe_route_backward(const moe_shape* shape, const void* x, const void* W_g,
                              const float* b_g, const float* probs, const int32_t* idx,
                              const float* w, const moe_route_upstream* up, void* dx, void* dW_g,
                              float* db_g, float* dlogits, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  size_t need = 0;
  moe_status st = moe_route_backward_workspace_size(shape, &need);
  if (st != MOE_OK) return st;
  if (!up) return MOE_ERR_NULL_ARG;
  const moe_shape& s = *shape;
  const moe_route_upstream& g = *up;
  if (bad_flag(g.dw_by_row) || !isfinite(g.loss_grad) || !isfinite(g.z_loss_grad) || g.R < 0 ||
      g.R >= kMaxRows)
    return MOE_ERR_BAD_SHAPE;
  if (s.T > 0) {
    if (!x || !W_g || !probs || !idx || !w || !dlogits || (need && !ws)) return MOE_ERR_NULL_ARG;
    if (g.loss_grad != 0.f && !g.f) return MOE_ERR_NULL_ARG;
    if ((g.rows || (g.dw && g.dw_by_row)) && !g.pos) return MOE_ERR_NULL_ARG;
  }
  if (!all_aligned16(x, W_g, g.rows, dx, dW_g, ws)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  RouteGradArgs m{};
  m.x = x;
  m.Wg = W_g;
  m.bias = b_g;
  m.probs = probs;
  m.idx = idx;
  m.w = w;
  m.dw = g.dw;
  m.f = g.f;
  m.rows = g.rows;
  m.pos = g.pos;
  m.T = s.T;
  m.R = g.R;
  m.d = (int)s.d_model;
  m.E = s.E;
  m.k = s.k;
  m.renorm = s.renormalize;
  m.dw_by_row = g.dw_by_row;
  m.bf16 = s.dtype == MOE_BF16;
  m.loss_grad = g.loss_grad;
  m.z_loss_grad = g.z_loss_grad;
  m.dx = dx;
  m.dWg = dW_g;
  m.db = db_g;
  m.dlogits = dlogits;
  m.ws = static_cast<char*>(ws);
  return launched(launch_route_grad(m, stream));
}

moe_status moe_block_norm(const moe_norm_shape* shape, const void* x, const float* y,
                          const float* gamma_post, const float* gate, const float* gamma,
                          void* out, void* u, float* rstd_post, float* rstd, hipStream_t stream) {
  const moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  const moe_norm_shape& s = *shape;
  // what belongs to a part that does not run is not given: a forgotten y or gamma shows (with
  // rows: a tensor without elements may have no address)
  if (s.T > 0 && !y && (gamma_post || gate || out || rstd_post || s.gate != MOE_GATE_NONE))
    return MOE_ERR_BAD_SHAPE;
  if (!gamma && (u || rstd)) return MOE_ERR_BAD_SHAPE;
  if (s.T > 0 && (s.gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_BAD_SHAPE;
  if (!all_aligned16(x, y, gamma_post, gamma, out, u) ||
      (s.gate == MOE_GATE_CHANNEL && !aligned16(gate)))
    return MOE_ERR_MISALIGNED;
  if (s.T == 0) return MOE_OK;
  if (!x || (!y && !gamma) || (y && (!gamma_post || !out)) || (gamma && !u)) return MOE_ERR_NULL_ARG;
  NormArgs m{};
  m.x = x;
  m.y = y;
  m.gamma_post = gamma_post;
  m.gate = gate;
  m.gamma = gamma;
  m.out = out;
  m.u = u;
  m.rstd_post = rstd_post;
  m.rstd = rstd;
  m.T = s.T;
  m.d = (int)s.d;
  m.gate_kind = s.gate;
  m.bf16 = s.dtype == MOE_BF16;
  m.eps = s.eps;
  m.scale = s.residual_scale;
  return launched(launch_block_norm(m, stream));
}

moe_status moe_block_norm_backward_workspace_size(const moe_norm_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL_ARG;
  const moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  *bytes = norm_grad_workspace(shape->T, (int)shape->d) * sizeof(float);
  return MOE_OK;
}

moe_status moe_block_norm_backward(const moe_norm_shape* shape, const void* d_out,
                                   const void* d_u, const void* out, const float* rstd,
                                   const float* gamma, const float* y, const float* rstd_post,
                                   const float* gamma_post, const float* gate, void* dx, void* dy,
                                   float* dgamma, float* dgamma_post, float* dgate, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
  size_t need = 0;
  const moe_status st = moe_block_norm_backward_workspace_size(shape, &need);
  if (st != MOE_OK) return st;
  const moe_norm_shape& s = *shape;
  if (s.T > 0 && !y && (gamma_post || gate || rstd_post || dy || dgamma_post || dgate || s.gate != MOE_GATE_NONE))
    return MOE_ERR_BAD_SHAPE;
  if (s.T > 0 && ((s.gate != MOE_GATE_NONE) != (gate != nullptr) || (dgate && !gate) || (dgamma && !d_u)))
    return MOE_ERR_BAD_SHAPE;
  if (!all_aligned16(d_out, d_u, out, gamma, y, gamma_post, dx, dy, ws) ||
      (s.gate == MOE_GATE_CHANNEL && !aligned16(gate)))
    return MOE_ERR_MISALIGNED;
  if (s.T > 0) {
    if ((!d_out && !d_u) || (d_u && (!out || !rstd || !gamma)) || (y && (!rstd_post || !gamma_post)))
      return MOE_ERR_NULL_ARG;
  }
  if (need && !ws) return MOE_ERR_NULL_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  NormGradArgs m{};
  m.d_out = d_out;
  m.d_u = d_u;
  m.out = out;
  m.rstd = rstd;
  m.gamma = gamma;
  m.y = y;
  m.rstd_post = rstd_post;
  m.gamma_post = gamma_post;
  m.gate = gate;
  m.dx = dx;
  m.dy = dy;
  m.dgamma = dgamma;
  m.dgamma_post = dgamma_post;
  m.dgate = dgate;
  m.partial = static_cast<float*>(ws);
  m.T = s.T;
  m.d = (int)s.d;
  m.gate_kind = s.gate;
  m.bf16 = s.dtype == MOE_BF16;
  m.scale = s.residual_scale;
  return launched(launch_block_norm_grad(m, stream));
}

}  // extern "C"

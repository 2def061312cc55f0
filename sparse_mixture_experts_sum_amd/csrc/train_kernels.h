// Launch wrappers of the training operators' kernels (internal; the public ABI is
// include/moe.h, "Training").
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

// Grouped products, forms as moe_matmul_form.
struct MatmulArgs {
  const void* a;
  const void* b;
  const int32_t* offsets;   // [E + 1]
  const int32_t* gather_a;  // [R] or nullptr
  const int32_t* gather_b;  // [R] or nullptr (TN)
  void* out;
  int64_t R, rows_a, rows_b, K, N;
  int E, form, bf16_in, bf16_out, accumulate;
  // set by the launch
  int splits;               // NN, NT: parts of the summed axis, split_stride values apart in out
  int64_t split_stride;     // values of a part's sum
  int64_t part_rows;        // TN: groups of more rows have their sum in parts, 0: none has
  int64_t part_sums;        // TN: the most part sums there can be
  float* parts;             // TN: the part sums
};
// Bytes of workspace: the parts' sums, where few tiles share a long sum; else 0.
size_t grouped_matmul_workspace(const MatmulArgs& a);
hipError_t launch_grouped_matmul(const MatmulArgs& a, float* ws, hipStream_t s);

struct SwigluGradArgs {
  const void *g, *u, *dh;   // [R, f]
  const float* w;           // [R], [T, k] with pos, or nullptr
  const int32_t* src;       // [R] with pos
  const int32_t* pos;       // [T, k] or nullptr
  const int32_t* offsets;   // [E + 1] or nullptr
  void *dg, *du, *hw;       // [R, f] or nullptr
  float* dw;                // [R] or nullptr
  int64_t R, f, T;
  int k, E, bf16;
};
hipError_t launch_swiglu_grad(const SwigluGradArgs& a, hipStream_t s);

struct RouteGradArgs {
  const void *x, *Wg;
  const float *bias, *probs;
  const int32_t* idx;
  const float *w, *dw, *f;
  const void* rows;
  const int32_t* pos;
  int64_t T, R;
  int d, E, k, renorm, dw_by_row, bf16;
  float loss_grad, z_loss_grad;
  void *dx, *dWg;
  float *db, *dlogits;
  char* ws;                 // workspace: route_grad_workspace bytes
  void* wt;                 // pieces of it (set by the launch)
  float *ds, *partial;
};
// Bytes of workspace.
size_t route_grad_workspace(int64_t T, int64_t d, int E);
hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s);

struct NormArgs {
  const void* x;
  const float *y, *gamma_post, *gate, *gamma;
  void *out, *u;
  float *rstd_post, *rstd;
  int64_t T;
  int d, gate_kind, bf16;
  float eps, scale;
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void *d_out, *d_u, *out;
  const float *rstd, *gamma, *y, *rstd_post, *gamma_post, *gate;
  void *dx, *dy;
  float *dgamma, *dgamma_post, *dgate;
  float* partial;           // workspace: norm_grad_workspace floats
  int64_t T;
  int d, gate_kind, bf16;
  float scale;
};
// Floats of workspace: per-workgroup partial column sums.
size_t norm_grad_workspace(int64_t T, int d);
hipError_t launch_block_norm_grad(const NormGradArgs& a, hipStream_t s);

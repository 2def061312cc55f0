// Launch wrappers of the layer norms' and the update step's kernels (internal; the public ABI
// is include/moe.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

struct LayerNormArgs {
  const void* x;
  const float *y, *gamma, *beta;
  void *out, *u;
  float *mean, *rstd;
  int64_t T;
  int d, bf16;
  float eps, scale;
};
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s);

struct LayerNormGradArgs {
  const void *out, *d_u, *d_out;
  const float *mean, *rstd, *gamma;
  void *dx, *dy;
  float *dgamma, *dbeta;
  float* partial;           // workspace: layer_norm_grad_workspace floats
  int64_t T;
  int d, bf16;
  float scale;
};
// Floats of workspace: per-workgroup partial column sums.
size_t layer_norm_grad_workspace(int64_t T, int d);
hipError_t launch_layer_norm_grad(const LayerNormGradArgs& a, hipStream_t s);

struct OrthArgs {
  const void* g;            // [E, m, n]
  void* out;                // [E, m, n]: the result, or the weights that the update is applied to
  float* momentum;          // [E, m, n], nullptr: g itself is orthogonalised
  int64_t m, n;
  int E, bf16, steps, nesterov;
  float a, b, c, eps;
  float mu, keep, rate;     // with momentum: out <- keep out - rate O
  char* ws;                 // workspace: orthogonalize_workspace bytes
};
// Bytes of workspace.
size_t orthogonalize_workspace(const OrthArgs& a);
hipError_t launch_orthogonalize(const OrthArgs& a, hipStream_t s);

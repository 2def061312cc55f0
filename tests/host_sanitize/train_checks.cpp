// csrc/train_api.hip under the sanitizers: its checks and workspace arithmetic over extreme
// shapes, with host-only stand-ins of the kernel launchers that count the calls that pass.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <vector>

#include "kernels.h"
#include "moe.h"
#include "train_kernels.h"

static long g_launched = 0, g_failures = 0;
#define CHECK(c)                                                     \
  do {                                                               \
    if (!(c)) {                                                      \
      ++g_failures;                                                  \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #c);            \
    }                                                                \
  } while (0)

// stand-ins: every argument a kernel would rely on is in range
size_t grouped_matmul_workspace(const MatmulArgs& a) {
  CHECK(a.R > 0 && a.K > 0 && a.N > 0 && a.E >= 1 && a.E <= 64);
  return a.R > 1000000 && a.N < 4096 ? 4096 : 0;
}
hipError_t launch_grouped_matmul(const MatmulArgs& a, float* ws, hipStream_t) {
  ++g_launched;
  CHECK(a.a && a.b && a.offsets && a.out && a.R > 0 && a.rows_a > 0);
  CHECK(a.K % 4 == 0 && a.N % 4 == 0 && (!a.bf16_in || (a.K % 8 == 0 && a.N % 8 == 0)));
  CHECK(!a.bf16_out || (a.bf16_in && !a.accumulate));
  CHECK(a.form == MOE_MATMUL_TN ? a.rows_b > 0 : !a.gather_b);
  CHECK(a.gather_a || a.rows_a == a.R);
  CHECK(!grouped_matmul_workspace(a) || ws);
  return hipSuccess;
}
hipError_t launch_swiglu_grad(const SwigluGradArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.g && a.u && a.dh && a.R > 0 && a.f > 0 && a.f % 4 == 0);
  CHECK(!a.pos || (a.w && a.src && a.T > 0 && a.k >= 1 && a.k <= 8));
  CHECK(!a.offsets || (a.E >= 1 && a.E <= 64));
  return hipSuccess;
}
size_t route_grad_workspace(int64_t T, int64_t d, int E) {
  CHECK(T >= 0 && d > 0 && d % 64 == 0 && E >= 1 && E <= 64);
  return (size_t)T * 256;
}
hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.T == 0 || (a.x && a.Wg && a.probs && a.idx && a.w && a.dlogits && a.ws));
  CHECK(a.loss_grad == 0.f || a.f || a.T == 0);
  CHECK(a.T == 0 || !(a.rows || (a.dw && a.dw_by_row)) || a.pos);
  CHECK(a.k >= 1 && a.k <= 8 && a.k <= a.E && a.R >= 0);
  return hipSuccess;
}
hipError_t launch_block_norm(const NormArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.x && a.T > 0 && a.d > 0 && a.d % 8 == 0 && a.d <= 16384);
  CHECK((a.y || a.gamma) && (!a.y || (a.gamma_post && a.out)) && (!a.gamma || a.u));
  CHECK((a.gate_kind != MOE_GATE_NONE) == (a.gate != nullptr));
  return hipSuccess;
}
size_t norm_grad_workspace(int64_t T, int d) {
  CHECK(T >= 0 && d > 0 && d <= 16384);
  return (size_t)d * 3;
}
hipError_t launch_block_norm_grad(const NormGradArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.partial && (a.T == 0 || a.d_out || a.d_u));
  CHECK(a.T == 0 || !a.d_u || (a.out && a.rstd && a.gamma));
  CHECK(a.T == 0 || !a.y || (a.rstd_post && a.gamma_post));
  return hipSuccess;
}
hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t) {
  ++g_launched;
  CHECK(p && bytes);
  return hipSuccess;
}

int main() {
  alignas(64) static char buf[64];
  void* p = buf;
  float* f = reinterpret_cast<float*>(buf);
  int32_t* n = reinterpret_cast<int32_t*>(buf);
  const std::initializer_list<int64_t> sizes = {INT64_MIN, -1, 0, 1, 4, 8, 60, 64, 72, 16384, 16392,
                                                (1 << 20), (1 << 20) + 8, 0x7fffffff, 0x80000000LL, INT64_MAX};
  const std::initializer_list<int32_t> small = {INT32_MIN, -1, 0, 1, 2, 3, 8, 9, 64, 65, INT32_MAX};
  size_t bytes = 0;
  for (int64_t R : sizes)
    for (int64_t K : sizes)
      for (int64_t N : sizes)
        for (int32_t E : small)
          for (int32_t form = -1; form <= 3; ++form)
            for (int t = 0; t < 6; ++t) {
              moe_matmul_shape s{R, R, R, K, N, E, form, t & 1, t >> 1, R % 3 == 0};
              for (int32_t* g : {(int32_t*)nullptr, n}) {
                moe_grouped_matmul(&s, p, p, n, g, form == MOE_MATMUL_TN ? g : nullptr, p, p, 4096, nullptr);
                moe_grouped_matmul(&s, p, p, n, g, g, p, nullptr, 0, nullptr);
              }
              moe_grouped_matmul_workspace_size(&s, &bytes);
              s.rows_a = 7;
              moe_grouped_matmul(&s, p, p, n, n, nullptr, p, p, 4096, nullptr);
            }
  for (int64_t R : sizes)
    for (int64_t w : sizes)
      for (int64_t T : sizes)
        for (int32_t k : small)
          for (int32_t E : small)
            for (int t = 0; t < 3; ++t) {
              moe_swiglu_shape s{R, w, T, k, E, t};
              moe_swiglu_backward(&s, p, p, p, f, n, n, n, p, p, p, f, nullptr);
              moe_swiglu_backward(&s, p, p, p, nullptr, nullptr, nullptr, nullptr, p, nullptr, p, nullptr, nullptr);
              moe_swiglu_backward(&s, p, p, p, nullptr, nullptr, n, nullptr, p, p, p, f, nullptr);
              moe_norm_shape q{R, w, t, k, E == 8 ? 0.f : 1e-6f, T == 1 ? 1e38f * 10 : 1.f};
              for (float* y : {(float*)nullptr, f})
                for (float* g : {(float*)nullptr, f}) {
                  moe_block_norm(&q, p, y, y, k ? f : nullptr, g, y ? p : nullptr, g ? p : nullptr, nullptr, nullptr,
                                 nullptr);
                  moe_block_norm_backward(&q, p, g, p, g, g, y, y, y, k ? f : nullptr, p, y ? p : nullptr, g, y,
                                          k ? f : nullptr, p, 1 << 20, nullptr);
                }
              moe_block_norm_backward_workspace_size(&q, &bytes);
            }
  for (int64_t T : sizes)
    for (int64_t d : sizes)
      for (int32_t E : small)
        for (int32_t k : small)
          for (int mode = -1; mode < 4; ++mode) {
            moe_shape s{T, d, 64, E, k, mode, k & 1, E & 1, 1.0};
            moe_route_upstream u{f, E & 1, 1.f, 1.f, f, p, n, d};
            if (moe_route_backward_workspace_size(&s, &bytes) == MOE_OK) {
              moe_route_backward(&s, p, p, f, f, n, f, &u, p, p, f, f, p, bytes, nullptr);
              u.pos = nullptr;
              moe_route_backward(&s, p, p, f, f, n, f, &u, p, p, f, f, p, bytes, nullptr);
              u.rows = nullptr;
              u.f = nullptr;
              moe_route_backward(&s, p, p, f, f, n, f, &u, nullptr, nullptr, nullptr, f, p, bytes, nullptr);
              moe_route_backward(&s, p, p, f, f, n, f, nullptr, p, p, f, f, p, bytes, nullptr);
            }
          }
  std::printf("launched %ld; passed: %ld failure(s)\n", g_launched, g_failures);
  return g_launched > 1000 && g_failures == 0 ? 0 : 1;
}

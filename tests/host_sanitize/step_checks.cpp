// csrc/step_api.hip under the sanitizers: its checks over extreme shapes, with host-only
// stand-ins of the kernel launchers that count the calls that pass.
#include <cmath>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "moe.h"
#include "step_kernels.h"

static long g_launched = 0, g_failures = 0;
#define CHECK(c)                                                     \
  do {                                                               \
    if (!(c)) {                                                      \
      ++g_failures;                                                  \
      std::printf("%s:%d: %s\n", __FILE__, __LINE__, #c);            \
    }                                                                \
  } while (0)

// stand-ins: every argument a kernel would rely on is in range
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.x && a.gamma && a.u && a.T > 0 && a.T < (int64_t(1) << 31) && a.d > 0 && a.d % 8 == 0 && a.d <= 16384);
  CHECK((a.y != nullptr) == (a.out != nullptr) && a.eps > 0.f);
  return hipSuccess;
}
size_t layer_norm_grad_workspace(int64_t T, int d) {
  CHECK(T >= 0 && d > 0 && d <= 16384 && d % 8 == 0);
  return (size_t)d * 2;
}
hipError_t launch_layer_norm_grad(const LayerNormGradArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.partial && a.d > 0 && a.d % 8 == 0 && a.d <= 16384);
  CHECK(a.T == 0 || (a.out && a.d_u && a.mean && a.rstd && a.gamma));
  return hipSuccess;
}
size_t orthogonalize_workspace(const OrthArgs& a) {
  CHECK(a.m >= 1 && a.n >= 1 && a.m <= 1 << 18 && a.n <= 1 << 18 && (a.m <= 16384 || a.n <= 16384));
  CHECK(a.E >= 1 && a.E <= 64 && a.steps >= 1 && a.steps <= 64);
  return (size_t)a.E * (size_t)a.m * (size_t)a.n;
}
hipError_t launch_orthogonalize(const OrthArgs& a, hipStream_t) {
  ++g_launched;
  CHECK(a.g && a.out && a.ws && reinterpret_cast<uintptr_t>(a.ws) % 256 == 0);
  CHECK(std::isfinite(a.a) && std::isfinite(a.b) && std::isfinite(a.c) && a.eps >= 0.f);
  CHECK(!a.momentum || (std::isfinite(a.mu) && (a.nesterov == 0 || a.nesterov == 1)));
  return hipSuccess;
}

int main() {
  alignas(256) static char buf[512];
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 64, 4096, 16384, 16385, 1 << 18, (1 << 18) + 1, 1 << 20,
                           (1 << 20) + 8, (int64_t(1) << 31) - 1, int64_t(1) << 31, INT64_MAX};
  const float values[] = {0.f, -1.f, 1e-5f, std::numeric_limits<float>::quiet_NaN(),
                          std::numeric_limits<float>::infinity(), 3e38f};
  void *p = buf, *odd = buf + 2;
  float* f = reinterpret_cast<float*>(buf);
  long calls = 0;
  for (int64_t T : sizes)
    for (int64_t d : sizes)
      for (int dtype : {-1, 0, 1, 2})
        for (float eps : values)
          for (int miss = 0; miss < 8; ++miss) {
            const moe_layer_norm_shape s{T, d, dtype, eps, miss == 7 ? values[3] : 1.f};
            size_t n = 0;
            moe_layer_norm(&s, miss == 1 ? nullptr : p, miss == 2 ? f : nullptr, miss == 3 ? nullptr : f, f,
                           miss == 4 ? p : nullptr, miss == 5 ? odd : p, f, f, nullptr);
            moe_layer_norm(&s, p, f, f, nullptr, p, p, nullptr, nullptr, nullptr);
            moe_layer_norm_backward_workspace_size(&s, &n);
            moe_layer_norm_backward(&s, p, miss == 1 ? nullptr : p, miss == 2 ? odd : p, f, miss == 3 ? nullptr : f, f, p,
                                    nullptr, f, f, miss == 4 ? nullptr : p, miss == 5 ? n - 1 : n, nullptr);
            calls += 3;
          }
  for (int64_t m : sizes)
    for (int64_t n : sizes)
      for (int E : {INT32_MIN, 0, 1, 64, 65, INT32_MAX})
        for (int steps : {-1, 0, 1, 5, 64, 65})
          for (int miss = 0; miss < 6; ++miss) {
            moe_orthogonalize_shape s{m, n, E, miss % 3, steps, 3.f, -4.f, 2.f, 0.f};
            if (miss == 4) s.b = values[3];
            if (miss == 5) s.eps = values[1];
            size_t bytes = 0;
            const moe_status st = moe_orthogonalize_workspace_size(&s, &bytes);
            CHECK(st == MOE_OK || bytes == 0);
            moe_orthogonalize(&s, miss == 1 ? nullptr : p, p, miss == 2 ? odd : p, bytes, nullptr);
            for (float lr : values) {
              const moe_muon_params q{lr, values[miss], lr, 1.f, miss - 1};
              moe_muon_update(&s, &q, p, p, miss == 3 ? nullptr : f, p, bytes, nullptr);
              ++calls;
            }
          }
  CHECK(moe_layer_norm(nullptr, p, f, f, f, p, p, f, f, nullptr) == MOE_ERR_NULL_ARG);
  CHECK(moe_orthogonalize(nullptr, p, p, p, 0, nullptr) == MOE_ERR_NULL_ARG);
  CHECK(g_launched > 1000);
  std::printf("%ld calls, %ld launched, passed: %ld failure(s)\n", calls, g_launched, g_failures);
  return g_failures != 0;
}

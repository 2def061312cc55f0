// Gradient of the experts' activation, h = silu(g) * u, and of each row's gate weight.
//
// With s = 1 / (1 + e^-g) the row's four results are
//   dg = w dh u s (1 + g (1 - s)),  du = w dh g s,  hw = w g s u,  dw = sum_f dh g s u,
// one pass over three inputs and three outputs: bound by HBM (6 f elements per row). bf16,
// 8192 x 4096: 78 us, 5.1 TB/s (a copy's rate); fp32 155 us, 5.2; 37 x 1408 fp32: 4.3 us, one row's latency.
// A row is read in 16-byte chunks, by one wave where it has at most 256 chunks (the row sum
// is then a shuffle tree, and the workgroup's four rows need no barrier) and by the whole
// workgroup beyond, so that a long row's loads are spread over four waves.
#include "train_common.h"
#include "train_kernels.h"

namespace {

// s = 1 / (1 + e^-g), for both types by expf and IEEE division: dw is fp32 for bf16 rows too, and
// the hardware's base-2 exponential of a rounded -g log2(e) is off by |g| 2^-24 of itself (bf16,
// 8192 x 4096: 78.1 against 78.5 us; 2048 x 4096, in the last-level cache, 16.3 against 17.5).
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// (no __restrict__: dg, du and hw may be g, u and dh)
template <typename TI, bool WAVE_ROW>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(SwigluGradArgs a) {
  constexpr int N = Chunk<TI>::N;
  typedef typename Chunk<TI>::vec vec;
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t first = 0, last = a.R;
  if (a.offsets) {
    int start, end;
    last = group_bounds(a.offsets, a.E, (int)a.R, start, end);
    first = __builtin_amdgcn_readlane(start, 0);
  }
  const int nch = (int)(a.f / N), step = WAVE_ROW ? 64 : 256;
  const int64_t rows = WAVE_ROW ? 4 : 1;
  for (int64_t r = first + blockIdx.x * rows + (WAVE_ROW ? wave : 0); r < last; r += gridDim.x * rows) {
    float w = 1.f;
    if (a.w) {
      if (!a.pos) {
        w = a.w[r];
      } else {
        w = 0.f;
        const int64_t t = min(max((int64_t)a.src[r], (int64_t)0), a.T - 1);
        for (int j = 0; j < a.k; ++j)
          if (a.pos[t * a.k + j] == r) w = a.w[t * a.k + j];
      }
    }
    const size_t base = (size_t)r * a.f;
    float sum = 0.f;
    for (int c = WAVE_ROW ? lane : threadIdx.x; c < nch; c += step) {
      const size_t at = base + (size_t)c * N;
      const vec g = *reinterpret_cast<const vec*>(static_cast<const TI*>(a.g) + at);
      const vec u = *reinterpret_cast<const vec*>(static_cast<const TI*>(a.u) + at);
      const vec dh = *reinterpret_cast<const vec*>(static_cast<const TI*>(a.dh) + at);
      vec og, ou, oh;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float gf = (float)g[i], uf = (float)u[i], df = (float)dh[i];
        const float s = sigmoid(gf), act = gf * s, wd = w * df;
        sum += df * act * uf;
        og[i] = (TI)(wd * uf * s * (1.0f + gf * (1.0f - s)));
        ou[i] = (TI)(wd * act);
        oh[i] = (TI)(w * act * uf);
      }
      if (a.dg) *reinterpret_cast<vec*>(static_cast<TI*>(a.dg) + at) = og;
      if (a.du) *reinterpret_cast<vec*>(static_cast<TI*>(a.du) + at) = ou;
      if (a.hw) *reinterpret_cast<vec*>(static_cast<TI*>(a.hw) + at) = oh;
    }
    if (!a.dw) continue;
    sum = wave_sum(sum);
    if constexpr (WAVE_ROW) {
      if (lane == 0) a.dw[r] = sum;
    } else {
      if (lane == 0) part[wave] = sum;
      __syncthreads();
      if (threadIdx.x == 0) a.dw[r] = ((part[0] + part[1]) + part[2]) + part[3];
      __syncthreads();  // part is written again for the next row
    }
  }
}

template <typename TI>
hipError_t launch(const SwigluGradArgs& a, hipStream_t s) {
  if (a.f / Chunk<TI>::N <= 256)
    swiglu_grad_kernel<TI, true><<<capped_grid((a.R + 3) / 4), 256, 0, s>>>(a);
  else
    swiglu_grad_kernel<TI, false><<<capped_grid(a.R), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu_grad(const SwigluGradArgs& a, hipStream_t s) {
  return a.bf16 ? launch<bf16>(a, s) : launch<float>(a, s);
}

// RMS norms after a block and before the next one, with the block's gate and the residual
// scale, and their gradient.
//
// Forward: out = rs x + gate (y q gamma_post), q = 1 / sqrt(mean y^2 + eps), and
// u = out r gamma, r = 1 / sqrt(mean out^2 + eps), with `out` rounded to its type first.
// A row is held in registers between the two norms, so every tensor is read or written
// once: bound by HBM. bf16, 16384 x 4096, both norms: 132 us, 5.1 TB/s (a copy's rate); 8 rows
// of 4096, the norm before alone: 3.6 us, one row's latency.
// Gradient: D = d_out + r (dz - z mean(dz z)), dx = rs D, dy = q (dn - n mean(dn n)); a row
// is held in registers between its sums and its results. The column sums (dgamma,
// dgamma_post, the per-channel dgate) stay in registers while a workgroup walks its rows and
// go out once per workgroup as partial sums, which a second kernel adds in workgroup order:
// no atomics, one fixed order. 8191 x 2048, both norms, a gate per token: 41 us and 5.5 for
// the partial sums (a copy of those bytes takes 46).
// All values and sums are fp32; outputs are rounded once.
#include "train_common.h"
#include "train_kernels.h"

#include "moe.h"

namespace {

// 8 elements as fp32.
template <typename TI>
__device__ __forceinline__ void load8(const TI* p, float (&v)[8]) {
  if constexpr (sizeof(TI) == 2) {
    const bf16x8 t = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)t[i];
  } else {
    const f32x4 t0 = *reinterpret_cast<const f32x4*>(p), t1 = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = t0[i];
      v[4 + i] = t1[i];
    }
  }
}
template <typename TI>
__device__ __forceinline__ void store8(TI* p, const float (&v)[8]) {
  if constexpr (sizeof(TI) == 2) {
    bf16x8 t;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (bf16)v[i];
    *reinterpret_cast<bf16x8*>(p) = t;
  } else {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// Sum over the TPR threads of a row. TPR = 64: the row is the wave's own. Otherwise the
// whole workgroup's, through `sh` (TPR / 64 floats; two barriers, so that it can be used
// again at once).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) sh[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += sh[i];
    __syncthreads();
  }
  return v;
}

// TPR threads per row, up to CH chunks of 8 elements per thread (chunk c of thread i is
// i + c TPR). Rows in strides of the grid.
template <typename TI, int TPR, int CH>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_kernel(NormArgs a) {
  constexpr int ROWS = TPR > 256 ? 1 : 256 / TPR;  // rows per workgroup
  __shared__ float sh[TPR / 64];
  static_assert(TPR == 64 || ROWS == 1, "a row is one wave's or the workgroup's");
  const int tid = threadIdx.x % TPR, nch = a.d / 8;
  const float inv_d = 1.0f / (float)a.d;
  for (int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR; t < a.T;
       t += (int64_t)gridDim.x * ROWS) {
    float o[CH][8];
    const size_t row = (size_t)t * a.d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i < nch) load8(static_cast<const TI*>(a.x) + row + i * 8, o[c]);
    }
    if (a.y) {
      float v[CH][8];
      float sq = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i >= nch) continue;
        load8(a.y + row + i * 8, v[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += v[c][e] * v[c][e];
      }
      const float q = 1.0f / sqrtf(row_sum<TPR>(sq, sh) * inv_d + a.eps);
      if (tid == 0 && a.rstd_post) a.rstd_post[t] = q;
      const float gt = a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i >= nch) continue;
        float gp[8], gc[8];
        load8(a.gamma_post + i * 8, gp);
        if (a.gate_kind == MOE_GATE_CHANNEL) load8(a.gate + i * 8, gc);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gate = a.gate_kind == MOE_GATE_CHANNEL ? gc[e] : gt;
          o[c][e] = (float)(TI)(a.scale * o[c][e] + gate * (v[c][e] * q * gp[e]));
        }
        store8(static_cast<TI*>(a.out) + row + i * 8, o[c]);
      }
    }
    if (!a.gamma) continue;
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (tid + c * TPR >= nch) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq += o[c][e] * o[c][e];
    }
    const float r = 1.0f / sqrtf(row_sum<TPR>(sq, sh) * inv_d + a.eps);
    if (tid == 0 && a.rstd) a.rstd[t] = r;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      float gm[8];
      load8(a.gamma + i * 8, gm);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[c][e] = o[c][e] * r * gm[e];
      store8(static_cast<TI*>(a.u) + row + i * 8, o[c]);
    }
  }
}

// Gradient. As above; acc[0..2]: this thread's column sums of dgamma, dgamma_post and the
// per-channel dgate over its rows, which the workgroup writes to partial[workgroup][3][d],
// those that are asked for.
template <typename TI, int TPR, int CH>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_grad_kernel(NormGradArgs a) {
  constexpr int ROWS = TPR > 256 ? 1 : 256 / TPR;
  __shared__ float sh[TPR / 64];
  const int tid = threadIdx.x % TPR, nch = a.d / 8;
  const int64_t group = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  const int64_t groups = (int64_t)gridDim.x * ROWS;
  const float inv_d = 1.0f / (float)a.d;
  float acc[3][CH][8] = {};
  for (int64_t t = group; t < a.T; t += groups) {
    const size_t row = (size_t)t * a.d;
    float D[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
#pragma unroll
      for (int e = 0; e < 8; ++e) D[c][e] = 0.f;
      if (i < nch && a.d_out) load8(static_cast<const TI*>(a.d_out) + row + i * 8, D[c]);
    }
    if (a.d_u) {
      const float r = a.rstd[t];
      float z[CH][8], dz[CH][8];
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i >= nch) continue;
        float gm[8];
        load8(static_cast<const TI*>(a.out) + row + i * 8, z[c]);
        load8(static_cast<const TI*>(a.d_u) + row + i * 8, dz[c]);
        load8(a.gamma + i * 8, gm);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[c][e] *= r;
          acc[0][c][e] += dz[c][e] * z[c][e];
          dz[c][e] *= gm[e];
          dot += dz[c][e] * z[c][e];
        }
      }
      const float m = row_sum<TPR>(dot, sh) * inv_d;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (tid + c * TPR >= nch) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) D[c][e] += r * (dz[c][e] - z[c][e] * m);
      }
    }
    if (a.dx) {
      const float scale = a.y ? a.scale : 1.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i >= nch) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = scale * D[c][e];
        store8(static_cast<TI*>(a.dx) + row + i * 8, v);
      }
    }
    if (!a.y) continue;
    const float q = a.rstd_post[t];
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.f;
    float n[CH][8], dn[CH][8];
    float dot = 0.f, dg = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      float gp[8], gc[8];
      load8(a.y + row + i * 8, n[c]);
      load8(a.gamma_post + i * 8, gp);
      if (a.gate_kind == MOE_GATE_CHANNEL) load8(a.gate + i * 8, gc);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gate = a.gate_kind == MOE_GATE_CHANNEL ? gc[e] : gt;
        n[c][e] *= q;
        const float dnn = D[c][e] * n[c][e];  // D n
        acc[1][c][e] += gate * dnn;
        acc[2][c][e] += dnn * gp[e];
        dg += dnn * gp[e];
        dn[c][e] = gate * D[c][e] * gp[e];
        dot += dn[c][e] * n[c][e];
      }
    }
    const float m = row_sum<TPR>(dot, sh) * inv_d;
    if (a.gate_kind == MOE_GATE_TOKEN && a.dgate) {
      dg = row_sum<TPR>(dg, sh);
      if (tid == 0) a.dgate[t] = dg;
    }
    if (!a.dy) continue;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) dn[c][e] = q * (dn[c][e] - n[c][e] * m);
      store8(static_cast<TI*>(a.dy) + row + i * 8, dn[c]);
    }
  }
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    if (s == 0 ? !a.dgamma : s == 1 ? !a.dgamma_post : !a.dgate || a.gate_kind != MOE_GATE_CHANNEL) continue;
    float* out = a.partial + ((size_t)blockIdx.x * 3 + s) * a.d;
    if constexpr (ROWS == 1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i < nch) store8(out + i * 8, acc[s][c]);
      }
    } else {  // the waves' sums first, in order
      __shared__ __attribute__((aligned(16))) float cols[ROWS][CH * TPR * 8];
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c) store8(cols[threadIdx.x / TPR] + (tid + c * TPR) * 8, acc[s][c]);
      __syncthreads();
      for (int i = threadIdx.x; i < a.d; i += ROWS * TPR) {
        float v = cols[0][i];
#pragma unroll
        for (int r = 1; r < ROWS; ++r) v += cols[r][i];
        out[i] = v;
      }
    }
  }
}

// Column sums of the partials: 64 columns per workgroup, sixteen threads per column on a
// sixteenth of the groups each, in order, then those in order.
constexpr int kSumParts = 16;
__global__ __launch_bounds__(64 * kSumParts) void norm_grad_sum_kernel(const float* __restrict__ partial,
                                                            int64_t groups, int d, float* o0,
                                                            float* o1, float* o2) {
  __shared__ float sh[kSumParts][64];
  const int which = blockIdx.y;
  float* out = which == 0 ? o0 : which == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  const int64_t per = (groups + kSumParts - 1) / kSumParts, g0 = part * per;
  const int64_t g1 = g0 + per < groups ? g0 + per : groups;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int64_t g = g0; g < g1; ++g) v += partial[((size_t)g * 3 + which) * d + c];
  }
  sh[part][threadIdx.x & 63] = v;
  __syncthreads();
  if (part || c >= d) return;
  v = sh[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < kSumParts; ++i) v += sh[i][threadIdx.x];
  out[c] = v;
}

// Rows of up to 1024 values are a wave's, four to a workgroup.
constexpr int kWaveRow = 1024;
// Workgroups of the gradient: as many as are resident together (their registers say how many),
// and half as many as there are rounds of rows, so that the partial sums stay few (us, by
// workgroups: 2048 rows of 4096: 43 with 1024, 36 with 512; 8192 of 3584: 130 with 585, 98
// with 512; 8192 of 8192: 245 with 1024, 214 with 256; 8192 of 2048: 54 with 1024, 67 with 512).
// 512 threads per row of 2049 to 4096 values, a chunk each: 16384 rows of 4096 262 -> 213 us
// against 256 threads with two chunks, whose registers left two waves per SIMD.
int64_t grad_groups(int64_t T, int d) {
  const int64_t rounds = d <= kWaveRow ? (T + 3) / 4 : T;
  const int64_t most = d <= 512 ? 1024 : d <= kWaveRow ? 512 : d <= 2048 ? 1024 : d <= 4096 ? 512 : 256;
  const int64_t few = rounds < 256 ? rounds : 256;
  int64_t n = rounds / 2 > few ? rounds / 2 : few;
  n = n < most ? n : most;
  return n > 0 ? n : 1;
}

template <typename TI>
hipError_t launch_fwd(const NormArgs& a, hipStream_t s) {
  const int64_t T = a.T;
  if (a.d <= 512) block_norm_kernel<TI, 64, 1><<<capped_grid((T + 3) / 4), 256, 0, s>>>(a);
  else if (a.d <= kWaveRow) block_norm_kernel<TI, 64, 2><<<capped_grid((T + 3) / 4), 256, 0, s>>>(a);
  else if (a.d <= 2048) block_norm_kernel<TI, 256, 1><<<capped_grid(T), 256, 0, s>>>(a);
  else if (a.d <= 4096) block_norm_kernel<TI, 256, 2><<<capped_grid(T), 256, 0, s>>>(a);
  else if (a.d <= 8192) block_norm_kernel<TI, 1024, 1><<<capped_grid(T), 1024, 0, s>>>(a);
  else block_norm_kernel<TI, 1024, 2><<<capped_grid(T), 1024, 0, s>>>(a);
  return hipGetLastError();
}

template <typename TI>
hipError_t launch_bwd(const NormGradArgs& a, hipStream_t s) {
  const int64_t groups = grad_groups(a.T, a.d);
  const unsigned grid = (unsigned)groups;
  if (a.d <= 512) block_norm_grad_kernel<TI, 64, 1><<<grid, 256, 0, s>>>(a);
  else if (a.d <= kWaveRow) block_norm_grad_kernel<TI, 64, 2><<<grid, 256, 0, s>>>(a);
  else if (a.d <= 2048) block_norm_grad_kernel<TI, 256, 1><<<grid, 256, 0, s>>>(a);
  else if (a.d <= 4096) block_norm_grad_kernel<TI, 512, 1><<<grid, 512, 0, s>>>(a);
  else if (a.d <= 8192) block_norm_grad_kernel<TI, 1024, 1><<<grid, 1024, 0, s>>>(a);
  else block_norm_grad_kernel<TI, 1024, 2><<<grid, 1024, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* chan = a.gate_kind == MOE_GATE_CHANNEL ? a.dgate : nullptr;
  if (!a.dgamma && !a.dgamma_post && !chan) return hipSuccess;
  norm_grad_sum_kernel<<<dim3((a.d + 63) / 64, 3), 64 * kSumParts, 0, s>>>(a.partial, groups, a.d, a.dgamma,
                                                               a.dgamma_post, chan);
  return hipGetLastError();
}

}  // namespace

size_t norm_grad_workspace(int64_t T, int d) {
  return (size_t)grad_groups(T, d) * 3 * (size_t)d;
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  return a.bf16 ? launch_fwd<bf16>(a, s) : launch_fwd<float>(a, s);
}

hipError_t launch_block_norm_grad(const NormGradArgs& a, hipStream_t s) {
  return a.bf16 ? launch_bwd<bf16>(a, s) : launch_bwd<float>(a, s);
}

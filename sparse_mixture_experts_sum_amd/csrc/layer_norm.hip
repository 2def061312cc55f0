// Layer norm of the residual sum, and its gradient.
//
// Forward: out = rs x + y, rounded to its type; u = (out - mean) r gamma + beta with
// r = 1 / sqrt(var + eps). A row is held in registers, so every tensor is read or written once:
// bound by HBM (bf16, 16384 x 4096 with y: 119 us, 5.6 TB/s, where a copy reaches 5.1; 8 rows of 4096:
// 4.5 us, one row's latency). The variance is that of differences from a mean: a wave takes its part's mean
// and the squares around it, and the waves' means and squares are joined by
// M2 = sum M2_w + n_w (mean_w - mean)^2, so that one pair of barriers gives both, without the
// cancellation of a difference of squares.
// Gradient: z = (out - mean) r, dz = d_u gamma, D = d_out + r (dz - mean(dz) - z mean(dz z)),
// dx = rs D, dy = D; both row means in one reduction. The column sums (dgamma, dbeta) stay in
// registers while a workgroup walks its rows and go out once per workgroup as partial sums,
// which a second kernel adds in workgroup order: no atomics, one fixed order. They need the row's
// mean and rstd alone, which are inputs: where rows are few, workgroups of their own take them in the
// same launch, 64 columns of all rows each. bf16, 16384 x 4096 with d_out and dy: 130 us, 5.1 TB/s; fp32,
// 8191 x 2048: 49-57 us (52 at a copy's rate); 4096 x 1024: 14.6 us in two launches (6.5): one wave a SIMD,
// whose four rows' loads wait for each other; 300 x 2048: 5 us.
// All values and sums are fp32; outputs are rounded once.
#include "step_kernels.h"
#include "train_common.h"

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

// 8 elements as they are stored, loaded before they are needed.
template <typename TI>
struct Stored8 {
  f32x4 v[sizeof(TI) / 2];
  __device__ __forceinline__ void load(const TI* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(TI) / 2; ++i) v[i] = reinterpret_cast<const f32x4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&o)[8]) const { load8(reinterpret_cast<const TI*>(v), o); }
};

// Sum over the L lanes of a row's part in one wave.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A row's threads: TPR of them, CH chunks of 8 values each (chunk c of thread i is i + c TPR).
// TPR < 64: several rows to a wave; TPR > 64: the row is the workgroup's.
template <int TPR_, int CH_>
struct Row {
  static constexpr int TPR = TPR_, CH = CH_;
  static constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;  // rows per workgroup
  static constexpr int LANES = TPR < 64 ? TPR : 64, WAVES = TPR / LANES;
  static_assert(TPR <= 64 || ROWS == 1, "a row is a wave's, a part of one, or the workgroup's");
  // values that wave w of a row holds
  static __device__ __forceinline__ int values(int w, int nch) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) n += 8 * min(max(nch - c * TPR - w * LANES, 0), LANES);
    return n;
  }
};

// Two sums over the threads of a row. sh: 2 * WAVES floats; two barriers, so that it can be
// used again at once.
template <class R>
__device__ __forceinline__ void row_sums(float& a, float& b, float* sh) {
  a = lanes_sum<R::LANES>(a);
  b = lanes_sum<R::LANES>(b);
  if constexpr (R::WAVES > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sh[2 * wave] = a;
      sh[2 * wave + 1] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < R::WAVES; ++i) {
      a += sh[2 * i];
      b += sh[2 * i + 1];
    }
    __syncthreads();
  }
}

// Mean and variance of a row.
template <class R>
__device__ __forceinline__ void row_moments(const float (&o)[R::CH][8], int tid, int nch, float inv_d,
                                            float* sh, float& mean, float& var) {
  const int wave = R::WAVES > 1 ? threadIdx.x >> 6 : 0;
  const int n = R::values(wave, nch);
  float sum = 0.f, m2 = 0.f;
#pragma unroll
  for (int c = 0; c < R::CH; ++c) {
    if (tid + c * R::TPR >= nch) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += o[c][e];
  }
  sum = lanes_sum<R::LANES>(sum);
  mean = R::WAVES > 1 ? sum / (float)max(n, 1) : sum * inv_d;
#pragma unroll
  for (int c = 0; c < R::CH; ++c) {
    if (tid + c * R::TPR >= nch) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) m2 += (o[c][e] - mean) * (o[c][e] - mean);
  }
  m2 = lanes_sum<R::LANES>(m2);
  if constexpr (R::WAVES > 1) {
    if ((threadIdx.x & 63) == 0) {
      sh[2 * wave] = mean;
      sh[2 * wave + 1] = m2;
    }
    __syncthreads();
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < R::WAVES; ++w) total += (float)R::values(w, nch) * sh[2 * w];
    mean = total * inv_d;
    m2 = 0.f;
#pragma unroll
    for (int w = 0; w < R::WAVES; ++w) {
      const float off = sh[2 * w] - mean;
      // (a wave without values has a mean of 0 and no weight)
      m2 += sh[2 * w + 1] + (float)R::values(w, nch) * off * off;
    }
    __syncthreads();
  }
  var = m2 * inv_d;
}

// Rows in strides of the grid.
template <typename TI, class R>
__global__ __launch_bounds__(R::THREADS) void layer_norm_kernel(LayerNormArgs a) {
  constexpr int TPR = R::TPR, CH = R::CH;
  __shared__ float sh[2 * R::WAVES];
  const int tid = threadIdx.x % TPR, nch = a.d / 8;
  const float inv_d = 1.0f / (float)a.d;
  for (int64_t t0 = (int64_t)blockIdx.x * R::ROWS; t0 < a.T; t0 += (int64_t)gridDim.x * R::ROWS) {
    // (rows of one wave: all lanes stay for the shuffles, those past the end on the last row)
    const int64_t mine = t0 + threadIdx.x / TPR, t = R::ROWS > 1 && mine >= a.T ? a.T - 1 : mine;
    const bool real = R::ROWS == 1 || mine < a.T;
    float o[CH][8];
    const size_t row = (size_t)t * a.d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      load8(static_cast<const TI*>(a.x) + row + i * 8, o[c]);
      if (!a.y) continue;
      float v[8];
      load8(a.y + row + i * 8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[c][e] = (float)(TI)(a.scale * o[c][e] + v[e]);
    }
    if (a.y && real) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i < nch) store8(static_cast<TI*>(a.out) + row + i * 8, o[c]);
      }
    }
    float mean, var;
    row_moments<R>(o, tid, nch, inv_d, sh, mean, var);
    const float r = 1.0f / sqrtf(var + a.eps);
    if (!real) continue;
    if (tid == 0) {
      if (a.mean) a.mean[t] = mean;
      if (a.rstd) a.rstd[t] = r;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      float gm[8], bt[8] = {};
      load8(a.gamma + i * 8, gm);
      if (a.beta) load8(a.beta + i * 8, bt);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[c][e] = (o[c][e] - mean) * r * gm[e] + bt[e];
      store8(static_cast<TI*>(a.u) + row + i * 8, o[c]);
    }
  }
}

// dgamma and dbeta of 64 columns from c0 on: thread i takes columns c0 + 8 (i % 8) .. + 7 of every
// THREADS / 8th row, and the threads' sums are added in order.
template <typename TI, int THREADS>
__device__ __forceinline__ void column_sums(const LayerNormGradArgs& a, int c0) {
  constexpr int LANES = THREADS / 8;
  __shared__ __attribute__((aligned(16))) float cols[LANES][64];
  const int c = c0 + threadIdx.x % 8 * 8, lane = threadIdx.x / 8;
  float acc[2][8] = {};
  if (c < a.d) {
#pragma unroll 4
    for (int t = lane; t < a.T; t += LANES) {
      const size_t at = (size_t)t * a.d + c;
      float z[8], du[8];
      load8(static_cast<const TI*>(a.out) + at, z);
      load8(static_cast<const TI*>(a.d_u) + at, du);
      const float mean = a.mean[t], r = a.rstd[t];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[0][e] += du[e] * ((z[e] - mean) * r);
        acc[1][e] += du[e];
      }
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float* out = s == 0 ? a.dgamma : a.dbeta;
    if (!out) continue;
    store8(&cols[lane][threadIdx.x % 8 * 8], acc[s]);
    __syncthreads();
    if (threadIdx.x < 64 && c0 + (int)threadIdx.x < a.d) {
      float v = cols[0][threadIdx.x];
#pragma unroll 8
      for (int i = 1; i < LANES; ++i) v += cols[i][threadIdx.x];
      out[c0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// Gradient. acc[0], acc[1]: this thread's column sums of dgamma and dbeta over its rows, which
// the workgroup writes to partial[workgroup][2][d], those that are asked for. FEW: workgroups from
// `groups` on take the column sums.
template <typename TI, class R, bool FEW>
__global__ __launch_bounds__(R::THREADS) void layer_norm_grad_kernel(LayerNormGradArgs a, int groups) {
  constexpr int TPR = R::TPR, CH = R::CH, ROWS = R::ROWS;
  __shared__ float sh[2 * R::WAVES];
  if constexpr (FEW) {
    if ((int)blockIdx.x >= groups) {
      column_sums<TI, R::THREADS>(a, ((int)blockIdx.x - groups) * 64);
      return;
    }
  }
  const int tid = threadIdx.x % TPR, nch = a.d / 8;
  const float inv_d = 1.0f / (float)a.d;
  float gm[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * TPR;
    if (i < nch) load8(a.gamma + i * 8, gm[c]);
  }
  float acc[2][CH][8] = {};
  // Where a CU holds one workgroup of a row, the next row's values are loaded while this one is worked on (8192
  // rows of 6000 bf16 105, so 96 us; 2000 of 8192 36, 33; where several are resident they do that for each
  // other, and the registers cost more: 16384 of 4096 129, 135).
  constexpr bool AHEAD = !FEW && TPR == 1024 && CH == 1;
  Stored8<TI> so[CH], su[CH], sd[CH];
  float s_mean = 0.f, s_rstd = 0.f;
  auto fetch = [&](int64_t t) {
    const size_t row = (size_t)t * a.d;
    s_mean = a.mean[t];
    s_rstd = a.rstd[t];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      so[c].load(static_cast<const TI*>(a.out) + row + i * 8);
      su[c].load(static_cast<const TI*>(a.d_u) + row + i * 8);
      if (a.d_out) sd[c].load(static_cast<const TI*>(a.d_out) + row + i * 8);
    }
  };
  const int64_t step = (int64_t)groups * ROWS;
  int64_t t0 = (int64_t)blockIdx.x * ROWS;
  if (AHEAD && t0 < a.T) fetch(t0);
  for (; t0 < a.T; t0 += step) {
    const int64_t mine = t0 + threadIdx.x / TPR, t = ROWS > 1 && mine >= a.T ? a.T - 1 : mine;
    const bool real = ROWS == 1 || mine < a.T;
    const size_t row = (size_t)t * a.d;
    float mean = s_mean, r = s_rstd;
    if constexpr (!AHEAD) {
      mean = a.mean[t];
      r = a.rstd[t];
    }
    float z[CH][8], dz[CH][8], D[CH][8];
    if constexpr (AHEAD) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (tid + c * TPR >= nch) continue;
        so[c].get(z[c]);
        su[c].get(dz[c]);
        if (a.d_out) sd[c].get(D[c]);
      }
      if (t0 + step < a.T) fetch(t0 + step);
    }
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      if constexpr (!AHEAD) {
        load8(static_cast<const TI*>(a.out) + row + i * 8, z[c]);
        load8(static_cast<const TI*>(a.d_u) + row + i * 8, dz[c]);
        if (a.d_out) load8(static_cast<const TI*>(a.d_out) + row + i * 8, D[c]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[c][e] = (z[c][e] - mean) * r;
        if (!FEW && real) {
          acc[0][c][e] += dz[c][e] * z[c][e];
          acc[1][c][e] += dz[c][e];
        }
        dz[c][e] *= gm[c][e];
        s0 += dz[c][e];
        s1 += dz[c][e] * z[c][e];
      }
    }
    row_sums<R>(s0, s1, sh);
    s0 *= inv_d;
    s1 *= inv_d;
    if (!real) continue;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = tid + c * TPR;
      if (i >= nch) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = r * (dz[c][e] - s0 - z[c][e] * s1);
        D[c][e] = a.d_out ? D[c][e] + g : g;
        v[e] = a.scale * D[c][e];
      }
      if (a.dx) store8(static_cast<TI*>(a.dx) + row + i * 8, v);
      if (a.dy) store8(static_cast<TI*>(a.dy) + row + i * 8, D[c]);
    }
  }
  if constexpr (FEW) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s == 0 ? !a.dgamma : !a.dbeta) continue;
    float* out = a.partial + ((size_t)blockIdx.x * 2 + s) * a.d;
    if constexpr (ROWS == 1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = tid + c * TPR;
        if (i < nch) store8(out + i * 8, acc[s][c]);
      }
    } else {  // the rows' sums first, in order
      __shared__ __attribute__((aligned(16))) float cols[ROWS][CH * TPR * 8];
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c) store8(cols[threadIdx.x / TPR] + (tid + c * TPR) * 8, acc[s][c]);
      __syncthreads();
      for (int i = threadIdx.x; i < a.d; i += R::THREADS) {
        float v = cols[0][i];
#pragma unroll
        for (int k = 1; k < ROWS; ++k) v += cols[k][i];
        out[i] = v;
      }
    }
  }
}

// Column sums of the partials: 64 columns per workgroup, sixteen threads per column on a
// sixteenth of the groups each, in order, then those in order.
constexpr int kSumParts = 16;
__global__ __launch_bounds__(64 * kSumParts) void layer_norm_sum_kernel(const float* __restrict__ partial,
                                                                       int64_t groups, int d, float* o0,
                                                                       float* o1) {
  __shared__ float sh[kSumParts][64];
  const int which = blockIdx.y;
  float* out = which == 0 ? o0 : o1;
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  const int64_t per = (groups + kSumParts - 1) / kSumParts, g0 = part * per;
  const int64_t g1 = g0 + per < groups ? g0 + per : groups;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int64_t g = g0; g < g1; ++g) v += partial[((size_t)g * 2 + which) * d + c];
  }
  sh[part][threadIdx.x & 63] = v;
  __syncthreads();
  if (part || c >= d) return;
  v = sh[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < kSumParts; ++i) v += sh[i][threadIdx.x];
  out[c] = v;
}

constexpr int kWaveRow = 1024;  // rows of up to so many values are a wave's or less

int rows_per_group(int d) { return d <= 128 ? 16 : d <= 256 ? 8 : d <= kWaveRow ? 4 : 1; }

// Workgroups of the gradient: as many as are resident together, and a quarter as many as there are
// rounds of rows, so that the partial sums stay few (us, by rounds of rows a workgroup: 2048 rows of
// 2048: two 17.0, four 14.4, eight 16.2; 1000 rows of 4096: two 16.9, four 15.8; 8192 rows of 1024: two and four
// 18.6, eight 21.3).
int64_t grad_groups(int64_t T, int d) {
  const int per = rows_per_group(d);
  const int64_t rounds = (T + per - 1) / per;
  const int64_t most = d <= 512 ? 1024 : d <= kWaveRow ? 512 : d <= 2048 ? 1024 : d <= 4096 ? 512 : 256;
  const int64_t few = rounds < 256 ? rounds : 256;
  int64_t n = rounds / 4 > few ? rounds / 4 : few;
  n = n < most ? n : most;
  return n > 0 ? n : 1;
}

template <typename TI, class R>
hipError_t fwd(const LayerNormArgs& a, hipStream_t s) {
  layer_norm_kernel<TI, R><<<capped_grid((a.T + R::ROWS - 1) / R::ROWS), R::THREADS, 0, s>>>(a);
  return hipGetLastError();
}
template <typename TI>
hipError_t launch_fwd(const LayerNormArgs& a, hipStream_t s) {
  if (a.d <= 128) return fwd<TI, Row<16, 1>>(a, s);
  if (a.d <= 256) return fwd<TI, Row<32, 1>>(a, s);
  if (a.d <= 512) return fwd<TI, Row<64, 1>>(a, s);
  if (a.d <= kWaveRow) return fwd<TI, Row<64, 2>>(a, s);
  if (a.d <= 2048) return fwd<TI, Row<256, 1>>(a, s);
  // (us: 16384 rows of 4096 with y, 119 against 124 with 256 threads of two chunks; 8192 rows of 8192 with
  // y, 124 against 149 with 1024 threads of one)
  if (a.d <= 4096) return fwd<TI, Row<512, 1>>(a, s);
  if (a.d <= 8192) return fwd<TI, Row<512, 2>>(a, s);
  return fwd<TI, Row<1024, 2>>(a, s);
}

// Rows so few that the column sums are taken in the same launch; in one before it where the rows'
// results go over what the sums read.
constexpr int64_t kFewRows = 512;

template <typename TI, class R>
hipError_t bwd(const LayerNormGradArgs& a, int64_t groups, hipStream_t s) {
  if (a.T <= kFewRows) {
    const int64_t rows = a.dx || a.dy ? (a.T + R::ROWS - 1) / R::ROWS : 0;
    const int64_t columns = a.dgamma || a.dbeta ? (a.d + 63) / 64 : 0;
    if (rows + columns == 0) return hipSuccess;
    auto over = [&](const void* p) { return p && (p == a.d_u || p == a.out); };
    if (columns && (over(a.dx) || over(a.dy))) {
      layer_norm_grad_kernel<TI, R, true><<<(unsigned)columns, R::THREADS, 0, s>>>(a, 0);
      if (rows) layer_norm_grad_kernel<TI, R, true><<<(unsigned)rows, R::THREADS, 0, s>>>(a, (int)rows);
    } else {
      layer_norm_grad_kernel<TI, R, true><<<(unsigned)(rows + columns), R::THREADS, 0, s>>>(a, (int)rows);
    }
  } else {
    layer_norm_grad_kernel<TI, R, false><<<(unsigned)groups, R::THREADS, 0, s>>>(a, (int)groups);
  }
  return hipGetLastError();
}
template <typename TI>
hipError_t launch_bwd(const LayerNormGradArgs& a, hipStream_t s) {
  const int64_t n = grad_groups(a.T, a.d);
  const hipError_t e = a.d <= 128        ? bwd<TI, Row<16, 1>>(a, n, s)
                       : a.d <= 256      ? bwd<TI, Row<32, 1>>(a, n, s)
                       : a.d <= 512      ? bwd<TI, Row<64, 1>>(a, n, s)
                       : a.d <= kWaveRow ? bwd<TI, Row<64, 2>>(a, n, s)
                       : a.d <= 2048     ? bwd<TI, Row<256, 1>>(a, n, s)
                       : a.d <= 4096     ? bwd<TI, Row<512, 1>>(a, n, s)
                       : a.d <= 8192     ? bwd<TI, Row<1024, 1>>(a, n, s)
                                         : bwd<TI, Row<1024, 2>>(a, n, s);
  if (e != hipSuccess || a.T <= kFewRows || (!a.dgamma && !a.dbeta)) return e;
  layer_norm_sum_kernel<<<dim3((a.d + 63) / 64, 2), 64 * kSumParts, 0, s>>>(a.partial, n, a.d, a.dgamma, a.dbeta);
  return hipGetLastError();
}

}  // namespace

size_t layer_norm_grad_workspace(int64_t T, int d) {
  return T <= kFewRows ? 0 : (size_t)grad_groups(T, d) * 2 * (size_t)d;
}

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
  return a.bf16 ? launch_fwd<bf16>(a, s) : launch_fwd<float>(a, s);
}

hipError_t launch_layer_norm_grad(const LayerNormGradArgs& a, hipStream_t s) {
  return a.bf16 ? launch_bwd<bf16>(a, s) : launch_bwd<float>(a, s);
}

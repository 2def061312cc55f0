// Products of rows grouped by expert, with ragged group sizes: NN (a b_e), NT (a b_e^T) and
// TN (the group's a^T b), fp32 sums.
//
// One workgroup per 64 x 64 tile of the output, 16 of the summed axis at a time through LDS.
#include "train_common.h"
#include "train_kernels.h"

#include "moe.h"

namespace {

constexpr int kT = 64, kK = 16;

// The tile of a workgroup: group e, summed range / output rows.
template <typename TI, typename TO, int FORM>
__global__ __launch_bounds__(256) void matmul_kernel(MatmulArgs a, int mtiles, int ntiles) {
  __shared__ float As[kK][kT + 1], Bs[kK][kT + 1];
  __shared__ int sh[4];
  const int tid = threadIdx.x, R = (int)a.R, K = (int)a.K, N = (int)a.N;
  const int nt = blockIdx.x % ntiles, mt = blockIdx.x / ntiles;
  int start, end;
  group_bounds(a.offsets, a.E, R, start, end);
  if (FORM == MOE_MATMUL_TN) {
    if (tid == mt / mtiles) { sh[0] = start; sh[1] = end; }
  } else {
    // tile mt of the groups' row tiles, group after group
    const int tiles = (end - start + kT - 1) / kT;
    int incl = tiles;
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if ((tid & 63) >= o) incl += v;
    }
    if (tid == 0) sh[2] = -1;
    __syncthreads();
    if (tid < a.E && mt >= incl - tiles && mt < incl) {
      sh[0] = start + (mt - (incl - tiles)) * kT;
      sh[1] = end;
      sh[2] = tid;
    }
  }
  __syncthreads();
  const int e = FORM == MOE_MATMUL_TN ? mt / mtiles : sh[2];
  if (e < 0) return;
  const int r0 = sh[0], r1 = sh[1], n0 = nt * kT;
  const int m0 = FORM == MOE_MATMUL_TN ? (mt % mtiles) * kT : r0;  // first output row
  const int len = FORM == MOE_MATMUL_TN ? r1 - r0 : K;             // summed
  const int mend = FORM == MOE_MATMUL_TN ? K : r1;
  const TI* A = static_cast<const TI*>(a.a);
  const TI* B = static_cast<const TI*>(a.b) + (FORM == MOE_MATMUL_TN ? 0 : (size_t)e * K * N);
  auto arow = [&](int r) -> int64_t {
    return a.gather_a ? min(max((int64_t)a.gather_a[r], (int64_t)0), a.rows_a - 1) : r;
  };
  auto brow = [&](int r) -> int64_t {
    return a.gather_b ? min(max((int64_t)a.gather_b[r], (int64_t)0), a.rows_b - 1) : r;
  };
  float acc[4][4] = {};
  const int tx = tid % 16, ty = tid / 16;
  for (int k0 = 0; k0 < len; k0 += kK) {
    for (int i = tid; i < kK * kT; i += 256) {
      if (FORM == MOE_MATMUL_TN) {
        const int kk = i / kT, m = i % kT;
        const bool in = k0 + kk < len;
        As[kk][m] = in && m0 + m < K ? (float)A[arow(r0 + k0 + kk) * K + m0 + m] : 0.f;
        Bs[kk][m] = in && n0 + m < N ? (float)B[brow(r0 + k0 + kk) * N + n0 + m] : 0.f;
      } else {
        const int kk = i % kK, m = i / kK;
        const bool in = k0 + kk < len;
        As[kk][m] = in && m0 + m < r1 ? (float)A[arow(m0 + m) * K + k0 + kk] : 0.f;
        if (FORM == MOE_MATMUL_NT) {
          Bs[kk][m] = in && n0 + m < N ? (float)B[(size_t)(n0 + m) * K + k0 + kk] : 0.f;
        } else {
          const int kb = i / kT, n = i % kT;
          Bs[kb][n] = k0 + kb < len && n0 + n < N ? (float)B[(size_t)(k0 + kb) * N + n0 + n] : 0.f;
        }
      }
    }
    __syncthreads();
    for (int kk = 0; kk < kK; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += As[kk][ty + 16 * i] * Bs[kk][tx + 16 * j];
    __syncthreads();
  }
  TO* out = static_cast<TO*>(a.out) + (FORM == MOE_MATMUL_TN ? (size_t)e * K * N : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= mend || n >= N) continue;
      TO* o = out + (size_t)m * N + n;
      *o = (TO)(a.accumulate ? (float)*o + acc[i][j] : acc[i][j]);
    }
}

template <typename TI, typename TO>
hipError_t launch(const MatmulArgs& a, hipStream_t s) {
  const int ntiles = (int)((a.N + kT - 1) / kT);
  const int mtiles = (int)((a.K + kT - 1) / kT);
  if (a.form == MOE_MATMUL_TN) {
    matmul_kernel<TI, TO, MOE_MATMUL_TN><<<a.E * mtiles * ntiles, 256, 0, s>>>(a, mtiles, ntiles);
  } else {
    const int64_t mt = a.R / kT + a.E;
    if (a.form == MOE_MATMUL_NN)
      matmul_kernel<TI, TO, MOE_MATMUL_NN><<<(unsigned)(mt * ntiles), 256, 0, s>>>(a, 0, ntiles);
    else
      matmul_kernel<TI, TO, MOE_MATMUL_NT><<<(unsigned)(mt * ntiles), 256, 0, s>>>(a, 0, ntiles);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_matmul(const MatmulArgs& a, hipStream_t s) {
  if (!a.bf16_in) return launch<float, float>(a, s);
  return a.bf16_out ? launch<bf16, bf16>(a, s) : launch<bf16, float>(a, s);
}

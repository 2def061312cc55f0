// Gradient of the token-choice router: of the selected weights, the load-balancing loss and
// the z-loss, with respect to the tokens, W_g and the bias.
//
// Per token, over its kept slots (w != 0) with S = sum of their probabilities,
//   dp_e = (dw_j - sum_i dw_i w_i) / S at e = idx_j (or dw_j), + loss_grad E f_e / (k T),
//   ds_e = p_e (dp_e - sum_c p_c dp_c) + z_loss_grad 2 lse p_e / T;
//   dx = ds W_g^T (+ the token's expert rows), dW_g = x^T ds, db = sum_t ds.
// x, dx and the rows are read or written once each, which bounds both passes (HBM).
// All values and sums are fp32. dW_g and db are summed per chunk of tokens into partial
// sums and those in chunk order: no atomics, one fixed order.
#include "train_common.h"
#include "train_kernels.h"

namespace {

constexpr int kTok = 16;     // tokens per workgroup of the ds / dx pass
// Partial sums of dW_g and db: chunks of tokens, at least kChunk each and at most kChunks.
constexpr int kChunk = 256, kChunks = 1024;
__host__ __device__ inline int64_t chunk_len(int64_t T) {
  const int64_t n = (T + kChunks - 1) / kChunks;
  return n < kChunk ? kChunk : n;
}

// ds of the workgroup's 16 tokens into LDS (row stride 64) and dlogits. 16 lanes per token,
// lane `sub` owning experts sub + 16 i.
template <typename TI>
__device__ __forceinline__ void token_ds(const RouteGradArgs& a, int64_t t0, float (&ds)[kTok][64]) {
  const int tok = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const int64_t t = t0 + tok < a.T ? t0 + tok : a.T - 1;  // (past the end: a copy, not stored)
  const int E = a.E, k = a.k;
  const float inv_T = 1.0f / (float)a.T;
  float p[4], dp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = sub + 16 * i;
    p[i] = e < E ? a.probs[t * E + e] : 0.f;
    dp[i] = (a.loss_grad != 0.f && e < E) ? a.loss_grad * ((float)E / (float)k) * inv_T * a.f[e] : 0.f;
  }
  if (a.dw) {
    float S = 0.f, dot = 0.f;
    float g[8];
    int ex[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = 0.f;
      ex[j] = -1;
      if (j >= k) continue;
      const float w = a.w[t * k + j];
      if (w == 0.f) continue;  // dropped (or a probability of 0, whose gradient is 0 too)
      if (a.dw_by_row) {
        const int r = a.pos[t * k + j];
        if (r < 0 || r >= a.R) continue;
        g[j] = a.dw[r];
      } else {
        g[j] = a.dw[t * k + j];
      }
      ex[j] = min(max(a.idx[t * k + j], 0), E - 1);
      S += a.probs[t * E + ex[j]];
      dot += g[j] * w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (ex[j] < 0) continue;
      const float v = a.renorm ? (g[j] - dot) / S : g[j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ex[j] == sub + 16 * i) dp[i] += v;
    }
  }
  float mean = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) mean += p[i] * dp[i];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) mean += __shfl_xor(mean, o);
  float zc = 0.f;
  if (a.z_loss_grad != 0.f) {
    // lse = s - log p at the most probable expert (p >= 1 / E there, so log p is exact to
    // about an ulp); the 16 lanes split the dot product
    float best = -1.f;
    int be = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (sub + 16 * i < E && p[i] > best) {
        best = p[i];
        be = sub + 16 * i;
      }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const float ob = __shfl_xor(best, o);
      const int oe = __shfl_xor(be, o);
      if (ob > best || (ob == best && oe < be)) {
        best = ob;
        be = oe;
      }
    }
    constexpr int N = Chunk<TI>::N;
    typedef typename Chunk<TI>::vec vec;
    const TI* x = static_cast<const TI*>(a.x) + t * a.d;
    const TI* W = static_cast<const TI*>(a.Wg) + be;
    float s = 0.f;
    for (int c = sub * N; c < a.d; c += 16 * N) {
      const vec v = *reinterpret_cast<const vec*>(x + c);
#pragma unroll
      for (int i = 0; i < N; ++i) s += (float)v[i] * (float)W[(size_t)(c + i) * E];
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (a.bias) s += a.bias[be];
    zc = a.z_loss_grad * 2.0f * inv_T * (s - logf(best));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = sub + 16 * i;
    const float v = p[i] * (dp[i] - mean + zc);
    ds[tok][e] = v;
    if (t0 + tok < a.T && e < E) a.dlogits[t * E + e] = v;
  }
  __syncthreads();
}

template <typename TI>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  __shared__ float ds[kTok][64];
  for (int64_t t0 = (int64_t)blockIdx.x * kTok; t0 < a.T; t0 += (int64_t)gridDim.x * kTok) {
  token_ds<TI>(a, t0, ds);
  if (a.dx) {
  constexpr int N = Chunk<TI>::N;
  typedef typename Chunk<TI>::vec vec;
  const TI* W = static_cast<const TI*>(a.Wg);
  for (int c = threadIdx.x * N; c < a.d; c += 256 * N) {
    float acc[kTok][N] = {};
    for (int e = 0; e < a.E; ++e) {
      float w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = (float)W[(size_t)(c + i) * a.E + e];
#pragma unroll
      for (int q = 0; q < kTok; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[q][i] += ds[q][e] * w[i];
    }
#pragma unroll
    for (int q = 0; q < kTok; ++q) {
      const int64_t t = t0 + q;
      if (t >= a.T) continue;
      if (a.rows)
        for (int j = 0; j < a.k; ++j) {
          const int r = a.pos[t * a.k + j];
          if (r < 0 || r >= a.R) continue;
          const vec v = *reinterpret_cast<const vec*>(static_cast<const TI*>(a.rows) + (size_t)r * a.d + c);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[q][i] += (float)v[i];
        }
      vec o;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = (TI)acc[q][i];
      *reinterpret_cast<vec*>(static_cast<TI*>(a.dx) + t * a.d + c) = o;
    }
  }
  }
  __syncthreads();  // ds is written again
  }
}

// partial[chunk][d + 1][E]: x^T ds over the chunk's tokens, and (row d) the sum of ds.
template <typename TI>
__global__ __launch_bounds__(256) void route_wgrad_kernel(RouteGradArgs a) {
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
  const int64_t t0 = blockIdx.y * chunk_len(a.T);
  const int64_t t1 = t0 + chunk_len(a.T) < a.T ? t0 + chunk_len(a.T) : a.T;
  if (c > a.d) return;
  float acc[16] = {};
  for (int64_t t = t0; t < t1; ++t) {
    const float x = c < a.d ? (float)static_cast<const TI*>(a.x)[t * a.d + c] : 1.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (part + 4 * i < a.E) acc[i] += x * a.dlogits[t * a.E + part + 4 * i];
  }
  float* out = a.partial + ((size_t)blockIdx.y * (a.d + 1) + c) * a.E;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (part + 4 * i < a.E) out[part + 4 * i] = acc[i];
}

template <typename TI>
__global__ __launch_bounds__(256) void route_wgrad_sum_kernel(RouteGradArgs a, int64_t chunks) {
  const size_t n = (size_t)(a.d + 1) * a.E, i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int64_t c = 0; c < chunks; ++c) v += a.partial[c * n + i];
  const size_t nw = (size_t)a.d * a.E;
  if (i < nw) {
    if (a.dWg) static_cast<TI*>(a.dWg)[i] = (TI)v;
  } else if (a.db) {
    a.db[i - nw] = v;
  }
}

int64_t chunks_of(int64_t T) { return (T + chunk_len(T) - 1) / chunk_len(T); }

template <typename TI>
hipError_t launch(const RouteGradArgs& a, hipStream_t s) {
  if (a.T > 0) {
    route_grad_kernel<TI><<<capped_grid((a.T + kTok - 1) / kTok), 256, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dWg && !a.db) return hipSuccess;
  const int64_t chunks = chunks_of(a.T);
  if (chunks > 0) {
    route_wgrad_kernel<TI><<<dim3(a.d / 64 + 1, (unsigned)chunks), 256, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t n = (size_t)(a.d + 1) * a.E;
  route_wgrad_sum_kernel<TI><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, chunks);
  return hipGetLastError();
}

}  // namespace

size_t route_grad_workspace(int64_t T, int64_t d, int E) {
  return (size_t)chunks_of(T) * (size_t)(d + 1) * (size_t)E;
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s) {
  return a.bf16 ? launch<bf16>(a, s) : launch<float>(a, s);
}

// Gradient of the token-choice router: of the selected weights, the load-balancing loss and
// the z-loss, with respect to the tokens, W_g and the bias.
//
// Per token, over its kept slots (w != 0) with S = sum of their probabilities,
//   dp_e = (dw_j - sum_i dw_i w_i) / S at e = idx_j (or dw_j), + loss_grad E f_e / (k T),
//   ds_e = p_e (dp_e - sum_c p_c dp_c) + z_loss_grad 2 lse p_e / T;
// the slots' part of it from w itself: as w = p / S (or p), p_e dp_e = w_j (dw_j - sum_i dw_i
// w_i), whose sum over e is 0 (or w_j dw_j, and sum_i dw_i w_i). No division by an S that may
// be as small as the smallest kept probability, and no load of p_e behind idx's.
//   dx = ds W_g^T (+ the token's expert rows), dW_g = x^T ds, db = sum_t ds.
// x, dx and the rows are read or written once each (x twice with the z-loss, whose lse takes
// a dot product first): bound by HBM, and by the launches at small sizes. Four kernels: W_g
// transposed (z-loss only), ds, then dx and partial sums of dW_g and db side by side in one
// launch, and the partial sums' sum in chunk order: no atomics, one fixed order. bf16, both
// losses: 4096 tokens of 1024, 8 experts, 21 us (ds 8.0, products 9.1, sum 3.5: latencies, a
// copy of those bytes takes 3.4); 8191 tokens of 2048, 64 experts, top-4 with the rows'
// gradients added, 77 us (traced: transpose 4.8, ds 11, products 60 at 4.2 TB/s, sum 5; a copy
// 40). fp32: 32 and 168 us.
//
// Both products run on the matrix cores. fp32: v_mfma_f32_32x32x2_f32 on the values. bf16:
// v_mfma_f32_32x32x16_bf16 with ds as a sum of three bf16 terms, which is ds to its last bit: ds
// sums to zero over a token's experts, and a weight's gradient over tokens nearly so, so dx and
// dW_g may be far smaller than their terms (two terms, off by 2^-17, take 167 against 174 us for
// 16384 tokens of 4096, 8 experts, rows added, and the same time within 2% at the sizes above).
// x and W_g are bf16 already. The ds kernel leaves ds in fp32 rows of EP = 32 or 64 experts,
// zeros past E.
#include "train_common.h"
#include "train_kernels.h"

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// The z-loss's dot products read W_g transposed: in LDS, where a workgroup of the ds kernel
// puts it itself, up to this size; from HBM, by a kernel of its own, beyond (mid-size layer,
// 16 KB: picking each expert's column out of W_g's rows instead took 14 us, this 9).
constexpr size_t kLdsWg = 65536;
constexpr int kTile = 64;    // tokens that the dW_g workgroups take at a time
constexpr int kSlab = 128;   // columns of x per dW_g workgroup: 32 per wave
constexpr int kDxCols = 256; // columns of dx per workgroup: 64 per wave
constexpr int kRun = 4;      // tiles of 32 tokens per dx workgroup
// Partial sums of dW_g and db: at most kChunks chunks of whole tiles of tokens, so that
// d / kSlab times that many workgroups cover the chip and the partial sums stay small.
constexpr int kChunks = 32;
__host__ __device__ inline int64_t chunk_len(int64_t T) {
  const int64_t tiles = (T + kTile - 1) / kTile;
  return (tiles + kChunks - 1) / kChunks * kTile;
}
int64_t chunks_of(int64_t T) { return T > 0 ? (T + chunk_len(T) - 1) / chunk_len(T) : 0; }
int padded_experts(int E) { return E <= 32 ? 32 : 64; }

// Workspace: padded rows of ds, W_g transposed, the partial sums, [E][d] of dW_g and [E] of db per
// chunk. Whole 256-byte pieces.
struct Layout {
  size_t ds, wt, partial, total;
};
Layout layout(int64_t T, int64_t d, int E) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  Layout l;
  l.ds = 0;
  l.wt = up((size_t)T * padded_experts(E) * 4);
  l.partial = l.wt + up(T > 0 ? (size_t)d * E * 4 : 0);
  l.total = l.partial + up((size_t)chunks_of(T) * (d + 1) * E * 4);
  return l;
}

__global__ __launch_bounds__(256) void transpose_kernel(const uint16_t* __restrict__ w16,
                                                        const uint32_t* __restrict__ w32, int d, int E,
                                                        void* __restrict__ out) {
  const int i = blockIdx.x * 256 + threadIdx.x;  // (d E <= 2^26)
  if (i >= d * E) return;
  const int e = i / d, c = i - e * d;
  if (w16) static_cast<uint16_t*>(out)[i] = w16[(size_t)c * E + e];
  else static_cast<uint32_t*>(out)[i] = w32[(size_t)c * E + e];
}

// ds of 256 / LANES tokens, LANES lanes per token, lane `sub` owning experts sub + LANES i: into
// dlogits and the padded rows.
template <typename TI, int EP, int LANES>
__device__ __forceinline__ void token_ds(const RouteGradArgs& a, const TI* wt, int64_t t0) {
  const int tok = threadIdx.x / LANES, sub = threadIdx.x % LANES;
  const int64_t t = t0 + tok < a.T ? t0 + tok : a.T - 1;  // (past the end: a copy, not stored)
  const int E = a.E, k = a.k;
  const float inv_T = 1.0f / (float)a.T;
  constexpr int PE = 64 / LANES;  // experts per lane
  float p[PE], dp[PE], sel[PE] = {};  // sel: the slots' part of ds
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < PE; ++i) {
    const int e = sub + LANES * i;
    p[i] = e < E ? a.probs[t * E + e] : 0.f;
    dp[i] = (a.loss_grad != 0.f && e < E) ? a.loss_grad * ((float)E / (float)k) * inv_T * a.f[e] : 0.f;
  }
  if (a.dw) {
    // every slot's loads first (a slot past k, and one without a row, reads another's)
    float w[8], g[8];
    int ex[8], at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t slot = t * k + (j < k ? j : 0);
      w[j] = a.w[slot];
      ex[j] = min(max(a.idx[slot], 0), E - 1);
      at[j] = a.dw_by_row ? a.pos[slot] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool row = at[j] >= 0 && at[j] < a.R;
      g[j] = 0.f;
      if (!a.dw_by_row) g[j] = a.dw[t * k + (j < k ? j : 0)];
      else if (a.R > 0) g[j] = a.dw[row ? at[j] : 0];
      // w = 0: dropped (or a probability of 0, whose gradient is 0 too)
      if (j >= k || w[j] == 0.f || (a.dw_by_row && !row)) ex[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (ex[j] >= 0) dot += g[j] * w[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (ex[j] < 0) continue;
      const float v = w[j] * (a.renorm ? g[j] - dot : g[j]);
#pragma unroll
      for (int i = 0; i < PE; ++i)
        if (ex[j] == sub + LANES * i) sel[i] += v;
    }
    if (a.renorm) dot = 0.f;  // (of sel's sum)
  }
  float mean = 0.f;
#pragma unroll
  for (int i = 0; i < PE; ++i) mean += p[i] * dp[i];
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) mean += __shfl_xor(mean, o);
  mean += dot;
  float zc = 0.f;
  if (a.z_loss_grad != 0.f) {
    // lse = s - log p at the most probable expert (p >= 1 / E there, so log p is exact to
    // about an ulp); the lanes split the dot product
    float best = -1.f;
    int be = 0;
#pragma unroll
    for (int i = 0; i < PE; ++i)
      if (sub + LANES * i < E && p[i] > best) {
        best = p[i];
        be = sub + LANES * i;
      }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
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
    const TI* W = wt + (size_t)be * a.d;
    float s = 0.f;
#pragma unroll 8
    for (int c = sub * N; c < a.d; c += LANES * N) {
      const vec v = *reinterpret_cast<const vec*>(x + c), u = *reinterpret_cast<const vec*>(W + c);
#pragma unroll
      for (int i = 0; i < N; ++i) s += (float)v[i] * (float)u[i];
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (a.bias) s += a.bias[be];
    zc = a.z_loss_grad * 2.0f * inv_T * (s - logf(best));
  }
  if (t0 + tok >= a.T) return;
#pragma unroll
  for (int i = 0; i < EP / LANES; ++i) {
    const int e = sub + LANES * i;
    const float v = sel[i] + p[i] * (dp[i] - mean + zc);  // (0 past E: both are)
    if (e < E) a.dlogits[t * E + e] = v;
    a.ds[t * EP + e] = v;
  }
}

// LDS_WG: W_g transposed into (dynamic) LDS first.
template <typename TI, int EP, bool LDS_WG, int LANES>
__global__ __launch_bounds__(256) void ds_kernel(RouteGradArgs a) {
  extern __shared__ __attribute__((aligned(16))) char wg_lds[];
  constexpr int TOK = 256 / LANES;
  if constexpr (LDS_WG) {
    constexpr int N = Chunk<TI>::N;
    TI* W = reinterpret_cast<TI*>(wg_lds);
    const int chunks = a.d * a.E / N;  // (d is a multiple of 64)
    for (int p = threadIdx.x; p < chunks; p += 256) {
      const auto v = *reinterpret_cast<const typename Chunk<TI>::vec*>(static_cast<const TI*>(a.Wg) + p * N);
      int c = p * N / a.E, e = p * N - c * a.E;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        W[e * a.d + c] = v[i];
        if (++e == a.E) {
          e = 0;
          ++c;
        }
      }
    }
    __syncthreads();
    for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.T; t0 += (int64_t)gridDim.x * TOK)
      token_ds<TI, EP, LANES>(a, W, t0);
  } else {
    for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.T; t0 += (int64_t)gridDim.x * TOK)
      token_ds<TI, EP, LANES>(a, static_cast<const TI*>(a.wt), t0);
  }
}

// Operands of the two products. A fragment covers 32 indices (lane % 32) and a piece of the
// summed axis: bf16 16 deep, lanes below 32 the first eight; fp32 two deep, lane / 32 the
// place. Accumulator value 4 q + i: first operand's index 8 q + 4 (lane / 32) + i, second
// operand's index lane % 32.
__device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(float a, float b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}
// Eight values as bf16 terms hi + mid + lo, each cut off instead of rounded: eight of the 24 bits
// a term, so that the sum is the value (to 2^-126, the smallest normal) and hi is finite where it
// is. A non-finite value is hi alone.
struct Terms {
  s16x8 t[3];
};
__device__ __forceinline__ Terms split(f32x4 a, f32x4 b) {
  Terms t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = i < 4 ? a[i % 4] : b[i % 4];
    const uint32_t hi = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
    const float r = (hi & 0x7f800000u) == 0x7f800000u ? 0.f : v - __builtin_bit_cast(float, hi);
    const uint32_t mid = __builtin_bit_cast(uint32_t, r) & 0xffff0000u;
    t.t[0][i] = (short)(hi >> 16);
    t.t[1][i] = (short)(mid >> 16);
    t.t[2][i] = (short)(__builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, mid)) >> 16);
  }
  return t;
}
__device__ __forceinline__ f32x16 zero16() {
  f32x16 v;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  return v;
}

// The routed rows of a dx tile: 32 tokens of up to KM slots, 64 columns, in passes of 32 /
// PASSES tokens whose loads are all in flight together. STREAM: non-temporal loads.
template <typename TI, int KM, bool STREAM>
struct RowTile {
  static constexpr int N = Chunk<TI>::N, PIECES = 64 / N, RPI = 64 / PIECES;  // tokens per load
  static constexpr int ITS = 32 / RPI, PASSES = KM > 4 ? ITS : ITS > 4 ? ITS / 4 : 1;
  static constexpr int PER = ITS / PASSES;
  typedef typename Chunk<TI>::vec vec;
  vec v[PER][KM ? KM : 1];
  uint32_t in[PER];  // bit j: slot j has a row

  // pass p; pos: the 32 tokens' rows in LDS, KM per token
  __device__ __forceinline__ void load(const RouteGradArgs& a, int p, const int* pos, int c, int ln) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = (p * PER + i) * RPI + ln / PIECES;
      in[i] = 0;
#pragma unroll
      for (int j = 0; j < KM; ++j) {
        const int at = pos[r * KM + j];
        in[i] |= (at >= 0 ? 1u : 0u) << j;
        // (a slot without a row reads row 0 and drops it: no branch between the loads)
        const vec* p = reinterpret_cast<const vec*>(static_cast<const TI*>(a.rows) + (size_t)max(at, 0) * a.d + c);
        v[i][j] = STREAM ? __builtin_nontemporal_load(p) : *p;
      }
    }
  }
};

// The columns' rows of W_g as first operands, 64 columns from c0: kept over a wave's tiles.
template <typename TI, int EP>
struct WgFrags;
template <int EP>
struct WgFrags<bf16, EP> {
  s16x8 f[2][EP / 16];
  __device__ __forceinline__ void load(const RouteGradArgs& a, int c0, int x, int h) {
    const int E = a.E;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const short* w = static_cast<const short*>(a.Wg) + (size_t)min(c0 + 32 * b + x, a.d - 1) * E;
#pragma unroll
      for (int s = 0; s < EP / 16; ++s) {
        const int e0 = 16 * s + 8 * h;
        f[b][s] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
        if (E % 8 == 0) {
          if (e0 < E) f[b][s] = *reinterpret_cast<const s16x8*>(w + e0);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e0 + i < E) f[b][s][i] = w[e0 + i];
        }
      }
    }
  }
  __device__ __forceinline__ void product(const RouteGradArgs& a, int64_t t, int h, f32x16 (&acc)[2]) const {
    const f32x4* row = reinterpret_cast<const f32x4*>(a.ds + t * EP + 8 * h);
#pragma unroll
    for (int s = 0; s < EP / 16; ++s) {
      const Terms d = split(row[4 * s], row[4 * s + 1]);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < 3; ++n) acc[b] = mma(f[b][s], d.t[n], acc[b]);
    }
  }
};
// fp32: summed in the order e, EP / 2 + e, so that each lane's values are consecutive
template <int EP>
struct WgFrags<float, EP> {
  float f[2][EP / 2];
  __device__ __forceinline__ void load(const RouteGradArgs& a, int c0, int x, int h) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float* w = static_cast<const float*>(a.Wg) + (size_t)min(c0 + 32 * b + x, a.d - 1) * a.E;
#pragma unroll
      for (int i = 0; i < EP / 2; ++i) {
        const int e = h * (EP / 2) + i;
        f[b][i] = e < a.E ? w[e] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void product(const RouteGradArgs& a, int64_t t, int h, f32x16 (&acc)[2]) const {
    const float* row = a.ds + t * EP + h * (EP / 2);
#pragma unroll
    for (int i = 0; i < EP / 2; ++i) {
      const float v = row[i];
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[b] = mma(f[b][i], v, acc[b]);
    }
  }
};

// The rows of a tile's slots, KM per token: entry ln + 64 i of the tile, -1 for none.
template <int KM>
struct TilePos {
  int v[KM ? (32 * KM + 63) / 64 : 1];
  __device__ __forceinline__ void fetch(const RouteGradArgs& a, int64_t t0, int ln) {
    if constexpr (KM > 0) {
#pragma unroll
      for (int i = 0; i < (32 * KM + 63) / 64; ++i) {
        const int at = ln + 64 * i, j = at % KM;
        const int64_t tt = t0 + at / KM;
        const int r = at < 32 * KM && tt < a.T && j < a.k ? a.pos[tt * a.k + j] : -1;
        v[i] = r < a.R ? r : -1;
      }
    }
  }
};

// dx of 32 tokens (t0 ..) and 64 columns (c0 ..), one wave: ds W_g^T with the columns as the
// first operand, then through the wave's piece of LDS, so that rows and dx move in 16-byte
// pieces, 128 or 256 contiguous bytes per row. The rows' loads go out first; `next` fetches the
// following tile's slots behind them.
template <typename TI, int EP, int KM, bool STREAM>
__device__ __forceinline__ void dx_tile(const RouteGradArgs& a, int64_t t0, int64_t t_next, int c0,
                                        const WgFrags<TI, EP>& wg, TilePos<KM>& slots, float* buf, int* pos) {
  const int ln = threadIdx.x & 63, x = ln & 31, h = ln >> 5;
  const int64_t t = min(t0 + x, a.T - 1);
  typedef RowTile<TI, KM, STREAM> Rows;
  constexpr int N = Rows::N, PIECES = Rows::PIECES, RPI = Rows::RPI;
  const int c = c0 + (ln % PIECES) * N, c_in = min(c, a.d - N);
  Rows rows;
  if constexpr (KM > 0) {
#pragma unroll
    for (int i = 0; i < (32 * KM + 63) / 64; ++i)
      if (ln + 64 * i < 32 * KM) pos[ln + 64 * i] = slots.v[i];
    rows.load(a, 0, pos, c_in, ln);
    slots.fetch(a, t_next, ln);
  }
  f32x16 acc[2] = {zero16(), zero16()};
  wg.product(a, t, h, acc);
  // [32 tokens][64 columns], 16-byte piece p of token row r at p ^ (r % 16)
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = (32 * b + 8 * q + 4 * h) / 4;
      *reinterpret_cast<f32x4*>(buf + x * 64 + (p ^ (x & 15)) * 4) =
          f32x4{acc[b][4 * q], acc[b][4 * q + 1], acc[b][4 * q + 2], acc[b][4 * q + 3]};
    }
  typedef typename Rows::vec vec;
#pragma unroll
  for (int p = 0; p < Rows::PASSES; ++p) {
    if constexpr (KM > 0) {
      if (p) rows.load(a, p, pos, c_in, ln);
    }
#pragma unroll
    for (int it = 0; it < Rows::PER; ++it) {
      const int r = (p * Rows::PER + it) * RPI + ln / PIECES;
      float v[N];
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const int piece = (ln % PIECES) * (N / 4) + i;
        const f32x4 u = *reinterpret_cast<const f32x4*>(buf + r * 64 + (piece ^ (r & 15)) * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[4 * i + q] = u[q];
      }
#pragma unroll
      for (int j = 0; j < KM; ++j) {
        const bool in = rows.in[it] >> j & 1;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += in ? (float)rows.v[it][j][i] : 0.f;
      }
      vec o;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = (TI)v[i];
      if (t0 + r < a.T && c < a.d) *reinterpret_cast<vec*>(static_cast<TI*>(a.dx) + (t0 + r) * a.d + c) = o;
    }
  }
}

// x^T ds over a chunk's tokens for kSlab columns: a wave's 32 columns by EP experts.
template <typename TI, int EP>
__device__ __forceinline__ void dw_chunk(const RouteGradArgs& a, int64_t chunk, int slab, char* lds) {
  const int tid = threadIdx.x, ln = tid & 63, wave = tid >> 6, x = ln & 31, h = ln >> 5;
  const int64_t t0 = chunk * chunk_len(a.T), t1 = min(t0 + chunk_len(a.T), a.T);
  const int c0 = slab * kSlab;
  constexpr int NE = EP / 32;
  f32x16 acc[NE];
#pragma unroll
  for (int n = 0; n < NE; ++n) acc[n] = zero16();
  if constexpr (sizeof(TI) == 2) {
    // x [64][128] and the terms of ds, [64][EP] each, bf16, read back transposed (a 16-lane
    // group's four rows give each lane four tokens of one column); 16-byte pieces swizzled by the row
    char* xs = lds;
    char* ds = lds + kTile * kSlab * 2;
    const bf16* X = static_cast<const bf16*>(a.x);
    auto sw = [](int row, int pieces) { return ((0xCA60 >> (4 * (row & 3))) & 15) % pieces; };
    auto frag = [&](const char* base, int width, int k0, int col0) {  // rows k0 .. + 15, 32 columns
      const int g = ln >> 4, r = (ln & 15) >> 2, cc = ln & 3;
      const int n = col0 + (g & 1) * 16 + 4 * cc, k = k0 + (g >> 1) * 8 + r;
      const char* p = base + k * width * 2 + ((n >> 3) ^ sw(k, width / 8)) * 16 + ((n >> 2) & 1) * 8;
      const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * width * 2));
      return s16x8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
    };
    constexpr int ND = EP / 32;  // eight experts of a token per thread, ND times
    u32x4 xv[4];
    f32x4 dv[ND][2];
    auto load = [&](int64_t t) {  // tokens past the chunk's end are zeros in both operands
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = tid + 256 * i, r = p / 16, c = c0 + (p % 16) * 8;
        xv[i] = t + r < t1 && c < a.d ? ld16(X + (t + r) * a.d + c) : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const int p = tid + 256 * i, r = p / (EP / 8);
        const f32x4* d = reinterpret_cast<const f32x4*>(a.ds + (t + r) * EP + (p % (EP / 8)) * 8);
#pragma unroll
        for (int n = 0; n < 2; ++n) dv[i][n] = t + r < t1 ? d[n] : f32x4{0, 0, 0, 0};
      }
    };
    load(t0);
    for (int64_t t = t0; t < t1; t += kTile) {
      __syncthreads();  // the last tile is no longer read
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = tid + 256 * i, r = p / 16;
        st16(xs + r * kSlab * 2 + ((p % 16) ^ sw(r, 16)) * 16, xv[i]);
      }
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const int p = tid + 256 * i, r = p / (EP / 8);
        const Terms d = split(dv[i][0], dv[i][1]);
#pragma unroll
        for (int n = 0; n < 3; ++n)
          st16(ds + (n * kTile + r) * EP * 2 + ((p % (EP / 8)) ^ sw(r, EP / 8)) * 16, __builtin_bit_cast(u32x4, d.t[n]));
      }
      __syncthreads();
      if (t + kTile < t1) load(t + kTile);  // in flight over this tile's products
#pragma unroll
      for (int s = 0; s < kTile / 16; ++s) {
        const s16x8 f = frag(xs, kSlab, 16 * s, wave * 32);
#pragma unroll
        for (int n = 0; n < NE; ++n)
#pragma unroll
          for (int i = 0; i < 3; ++i)
            acc[n] = mma(frag(ds + i * kTile * EP * 2, EP, 16 * s, 32 * n), f, acc[n]);
      }
    }
  } else {
    const float* X = static_cast<const float*>(a.x) + min(c0 + wave * 32 + x, a.d - 1);
    const float* D = a.ds + x;
    for (int64_t t = t0; t < t1; t += 16) {
      float xv[8], dv[8][NE];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t tt = t + 2 * i + h;
        const bool in = tt < t1;
        xv[i] = in ? X[tt * a.d] : 0.f;
#pragma unroll
        for (int n = 0; n < NE; ++n) dv[i][n] = in ? D[tt * EP + 32 * n] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int n = 0; n < NE; ++n) acc[n] = mma(dv[i][n], xv[i], acc[n]);
    }
  }
  const int c = c0 + wave * 32 + x;
  float* out = a.partial + (size_t)chunk * (a.d + 1) * a.E;
  if (c < a.d) {
#pragma unroll
    for (int n = 0; n < NE; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = 32 * n + 8 * (i / 4) + 4 * h + i % 4;
        if (e < a.E) out[(size_t)e * a.d + c] = acc[n][i];
      }
  }
  // db's partial sum, in the first slab's workgroup: a wave takes every fourth token
  if (slab) return;
  __syncthreads();
  float* sh = reinterpret_cast<float*>(lds);
  float v = 0.f;
  if (ln < a.E) {
#pragma unroll 4
    for (int64_t t = t0 + wave; t < t1; t += 4) v += a.dlogits[t * a.E + ln];
  }
  sh[tid] = v;
  __syncthreads();
  if (tid < a.E) out[(size_t)a.d * a.E + tid] = ((sh[tid] + sh[64 + tid]) + sh[128 + tid]) + sh[192 + tid];
}

// Workgroups [0, dw_blocks): partial sums of dW_g and db, column slabs within a chunk; the
// others: dx tiles, columns within 32 tokens.
template <typename TI, int EP, int KM, bool STREAM>
__global__ __launch_bounds__(256) void route_products_kernel(RouteGradArgs a, int dw_blocks) {
  // dx: 8 KB per wave; dW_g (bf16): x and ds tiles
  constexpr int kTiles = sizeof(TI) == 2 ? kTile * kSlab * 2 + 3 * kTile * EP * 2 : 0;
  __shared__ __attribute__((aligned(16))) char lds[kTiles > 32768 ? kTiles : 32768];
  __shared__ int pos[4][KM ? 32 * KM : 1];
  if ((int)blockIdx.x < dw_blocks) {
    const int slabs = (a.d + kSlab - 1) / kSlab;
    dw_chunk<TI, EP>(a, blockIdx.x / slabs, blockIdx.x % slabs, lds);
    return;
  }
  // kRun consecutive token tiles of a column block per workgroup, while W_g's rows are kept
  const int wave = threadIdx.x >> 6, ln = threadIdx.x & 63;
  const int64_t cols = (a.d + kDxCols - 1) / kDxCols, tiles = (a.T + 31) / 32;
  const int64_t runs = (tiles + kRun - 1) / kRun * cols;
  for (int64_t i = blockIdx.x - dw_blocks; i < runs; i += gridDim.x - dw_blocks) {
    const int c0 = (int)(i % cols) * kDxCols + wave * 64;
    if (c0 >= a.d) continue;
    WgFrags<TI, EP> wg;
    wg.load(a, c0, ln & 31, ln >> 5);
    const int64_t first = i / cols * kRun, last = min(first + kRun, tiles);
    TilePos<KM> slots;
    slots.fetch(a, first * 32, ln);
    for (int64_t n = first; n < last; ++n)
      dx_tile<TI, EP, KM, STREAM>(a, n * 32, (n + 1) * 32, c0, wg, slots, reinterpret_cast<float*>(lds) + wave * 2048,
                          pos[wave]);
  }
}

// dW_g and db from the partial sums, chunks in order.
template <typename TI>
__global__ __launch_bounds__(256) void route_sum_kernel(RouteGradArgs a, int chunks) {
  const size_t n = (size_t)(a.d + 1) * a.E, i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
#pragma unroll 8
  for (int c = 0; c < chunks; ++c) v += a.partial[c * n + i];
  const size_t nw = (size_t)a.d * a.E;
  if (i < nw) {
    const size_t e = i / a.d, c = i - e * a.d;
    if (a.dWg) static_cast<TI*>(a.dWg)[c * a.E + e] = (TI)v;
  } else if (a.db) {
    a.db[i - nw] = v;
  }
}

template <typename TI, int EP, bool STREAM>
void launch_products(const RouteGradArgs& a, int km, unsigned grid, int dw_blocks, hipStream_t s) {
  if (km <= 2) route_products_kernel<TI, EP, 2, STREAM><<<grid, 256, 0, s>>>(a, dw_blocks);
  else if (km <= 4) route_products_kernel<TI, EP, 4, STREAM><<<grid, 256, 0, s>>>(a, dw_blocks);
  else route_products_kernel<TI, EP, 8, STREAM><<<grid, 256, 0, s>>>(a, dw_blocks);
}

template <typename TI, int EP>
hipError_t launch(RouteGradArgs a, hipStream_t s) {
  const Layout l = layout(a.T, a.d, a.E);
  a.ds = reinterpret_cast<float*>(a.ws + l.ds);
  a.wt = a.ws + l.wt;
  a.partial = reinterpret_cast<float*>(a.ws + l.partial);
  const bool dw = a.dWg || a.db;
  const int chunks = (int)chunks_of(a.T);
  hipError_t e = hipSuccess;
  if (a.T > 0) {
    const size_t wg_bytes = (size_t)a.d * a.E * sizeof(TI);
    // Lanes per token: 32 where the z-loss's dot product is a chain of loads that more waves
    // hide (us of the whole gradient with 16 -> 32: 8191 tokens of 2048, 64 experts, 48.6 -> 46.3;
    // 200 of 1024, 8 experts, 14.7 -> 14.0), 16 without it, and where the workgroups come back
    // for more tokens (16384 of 4096, 8 experts, 97.7 against 103.6).
    constexpr int64_t kLdsGroups = 512;  // two per CU: each brings W_g into its LDS once
    const auto groups = [&](int lanes) { return capped_grid((a.T + 256 / lanes - 1) / (256 / lanes)); };
    if (a.z_loss_grad == 0.f) {
      ds_kernel<TI, EP, false, 16><<<groups(16), 256, 0, s>>>(a);
    } else if (wg_bytes <= kLdsWg) {
      if (a.T <= kLdsGroups * 8)
        ds_kernel<TI, EP, true, 32><<<groups(32), 256, wg_bytes, s>>>(a);
      else
        ds_kernel<TI, EP, true, 16><<<kLdsGroups < groups(16) ? kLdsGroups : groups(16), 256, wg_bytes, s>>>(a);
    } else {
      const bool b16 = sizeof(TI) == 2;
      transpose_kernel<<<(a.d * a.E + 255) / 256, 256, 0, s>>>(
          b16 ? static_cast<const uint16_t*>(a.Wg) : nullptr,
          b16 ? nullptr : static_cast<const uint32_t*>(a.Wg), a.d, a.E, a.wt);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      ds_kernel<TI, EP, false, 32><<<groups(32), 256, 0, s>>>(a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int dw_blocks = dw ? chunks * ((a.d + kSlab - 1) / kSlab) : 0;
    const int64_t dx_blocks = a.dx ? (a.T + 32 * kRun - 1) / (32 * kRun) * ((a.d + kDxCols - 1) / kDxCols) : 0;
    if (dw_blocks || dx_blocks) {
      const unsigned grid = dw_blocks + (dx_blocks ? capped_grid(dx_blocks) : 0);
      const int km = a.rows && a.R > 0 ? a.k : 0;
      // Rows that fill half of the last-level cache or more push out what is read again; fewer
      // stay there from the kernel that wrote them. us of the gradient without the hint -> with,
      // rows long written / with the cast that writes them right before: 8192 rows of 2048, 33 MB,
      // 42.1 -> 44.0 / 61.3 -> 60.9; 24576, 100 MB, 71.3 -> 67.7 / 117.4 -> 119.2; 32764, 134 MB,
      // 81.4 -> 77.9 / 146.2 -> 144.4; 49152, 201 MB, 116 -> 110 / 217 -> 208; 16384 of 4096, 134
      // MB, 100.8 -> 98.2 / 170.1 -> 166.1; 65536 of 1024, 134 MB, 55.9 -> 53.8 / 114.0 -> 114.9.
      const bool stream = (double)a.R * a.d * sizeof(TI) > 128e6;
      if (km == 0) route_products_kernel<TI, EP, 0, false><<<grid, 256, 0, s>>>(a, dw_blocks);
      else if (stream) launch_products<TI, EP, true>(a, km, grid, dw_blocks, s);
      else launch_products<TI, EP, false>(a, km, grid, dw_blocks, s);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (!dw) return hipSuccess;
  const size_t n = (size_t)(a.d + 1) * a.E;
  route_sum_kernel<TI><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, chunks);
  return hipGetLastError();
}

template <typename TI>
hipError_t launch_type(const RouteGradArgs& a, hipStream_t s) {
  return padded_experts(a.E) == 32 ? launch<TI, 32>(a, s) : launch<TI, 64>(a, s);
}

}  // namespace

size_t route_grad_workspace(int64_t T, int64_t d, int E) { return layout(T, d, E).total; }

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s) {
  return a.bf16 ? launch_type<bf16>(a, s) : launch_type<float>(a, s);
}

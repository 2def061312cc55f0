// Newton-Schulz orthogonalisation of E matrices, and the update step around it.
//
// X = G / (|G| + eps); a step is X <- P X with A = X X^T and P = a I + b A + c A^2 (X^T X, of the short
// side, and X P where G is tall). All polynomials of A commute, so two steps share the long products:
// with A' = (P X) (P X)^T = P^2 A and P' of it, X <- P' P X.
// Per pair of steps, with s and l the short and the long side, 3 s^2 l + 5 s^3 operations in place of
// 6 s^2 l + 2 s^3; every product but the last is symmetric, and only the tiles on and below its
// diagonal are computed, each stored a second time as its own transpose.
// P and P' P are kept with their diagonals, as they are multiplied: a I apart and b A + c A^2 rounded
// by itself would cancel where P is small, at the large singular values.
//
// Products: one workgroup of four waves per square tile, v_mfma_f32_32x32x16_f16, stages of 32 of the
// summed axis through a ring of four LDS buffers, tile after tile as one stream. All matrices of the
// iteration are padded with zeros to multiples of 128, so that a sum is a whole number of ring turns
// and no value of an operand has to be masked.
// They are kept in panels of 32 columns, [columns / 32][rows][32]: what a load instruction of a stage
// takes (16 rows of 64 bytes) is then one run of 1 KB of whole cache lines, whichever axis of the
// matrix is summed over, and so is what a store leaves. With rows as they are, half lines, the L2s
// gave a CU no more than the half (1.05 TB/s an XCD), and that bound the products.
// Tiles that would leave most CUs without one in the last round have their sums in parts,
// which a second kernel joins in order.
//
// What is kept between products: fp16, of values scaled to lie in its range (X times a power of
// two near the square root of its long side; A and P as they are, of order 1). G itself enters
// as G 2^p (bf16 values of 2^-14 and more then exactly, smaller ones to 2^-25, and so what the momentum makes of
// them in fp32 to 2^-11 of a value), and the rest of its norm as a factor of the first products' sums.
// bf16 matrices: one fp16 term (2^-11 of a value at most, 2^-25 below 2^-14, where values are 1 / sqrt(short side)
// at the start: rows 1e-5 times the others are off by 7% of themselves; with bf16 terms a full-rank matrix would be
// off by 1%, not by 0.2%), for as many steps as bear it: each multiplies what was rounded before it.
// fp32 matrices, bf16 ones of more steps (one_term_bears) and bf16 ones of short sides (few large singular values,
// whose roundings do not average out: 64 x 128 is 0.7% off with one term, 700 x 700 0.2%; the products
// are too small there to be what counts): two terms, hi + lo / 2048 (22 bits; lo is scaled so that
// it stays normal where hi is), and three products: lo hi and hi lo first, their sum divided by
// 2048, then hi hi.
// Bound by the matrix cores where matrices are large (8 of 4096 x 14336 bf16 with the update: 22.1 ms, the long
// products at 1190 TFLOP/s, where a large fp16 product reaches 1172; 64 of 2048 x 1408: 5.4 ms), by tiles
// that do not fill the chip evenly in between (8 of 1024 x 4096: 0.6 ms), and by launches where small.
#include <math.h>

#include <type_traits>

#include "matmul_tile.h"
#include "step_kernels.h"
#include "train_common.h"

namespace {

typedef _Float16 f16;
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kPad = 128;           // sides of the iteration's matrices
constexpr int kXcds = 8;
constexpr int kCus = 256;
constexpr int kColBlock = 4;        // columns of tiles walked together
constexpr float kLo = 1.0f / 2048;  // scale of the second term
constexpr int kNormBlocks = 256;    // most partial sums of a matrix's squares
constexpr int kMaxParts = 16;       // of a product's sum
constexpr int kOneTerm = 128;       // bf16 matrices with short sides past it may be kept in one term (terms_of)
constexpr double kMostGrowth = 256;  // what steps in one term may multiply a rounding by, added over the steps
constexpr double kMostValue = 1.25;  // singular values that they may reach

// Place of a value of a matrix of the iteration: panels of 32 columns, each with all rows.
__device__ __forceinline__ int64_t in_panels(int64_t rows, int64_t r, int64_t c) {
  return ((c >> 5) * rows + r) * 32 + (c & 31);
}

// The same for matrices that are loaded as fragments: of 32 rows and 16 columns one run of 1 KB, lane l's
// 16 bytes (row l % 32, columns 8 (l / 32) ..) at 16 l.
__device__ __forceinline__ int64_t in_fragments(int64_t rows, int64_t r, int64_t c) {
  return (((c >> 4) * (rows >> 5) + (r >> 5)) * 64 + (c >> 3 & 1) * 32 + (r & 31)) * 8 + (c & 7);
}

// ---- the matrix in, and its norm -------------------------------------------------------
// u, what is orthogonalised: g, or its momentum step, from g and the momentum before
// (`fresh`) or after it.
__device__ __forceinline__ float momentum_of(const OrthArgs& a, float m, float g) { return a.mu * m + g; }
__device__ __forceinline__ float update_of(const OrthArgs& a, float m, float g) {
  return a.nesterov ? a.mu * m + g : m;
}
template <typename TI>
__device__ __forceinline__ void load_row(const TI* p, int n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
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
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)p[i] : 0.f;
  }
}
template <typename TI>
__device__ __forceinline__ void store_row(TI* p, int n, bool vec, const float (&v)[8]) {
  if (vec && n >= 8) {
    if constexpr (sizeof(TI) == 2) {
      bf16x8 t;
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = (bf16)v[i];
      *reinterpret_cast<bf16x8*>(p) = t;
    } else {
      *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (TI)v[i];
  }
}

__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  v = ((sh[0] + sh[1]) + sh[2]) + sh[3];
  __syncthreads();
  return v;
}

// The momentum's step, and sums of u^2 (fp64: no finite fp32 matrix overflows or vanishes).
// Workgroup x of matrix y. vec: whole chunks of 8 values, 16-byte aligned.
template <typename TI>
__global__ __launch_bounds__(256) void square_kernel(OrthArgs a, bool vec, double* partial) {
  __shared__ double sh[4];
  const int64_t size = a.m * a.n, at = (int64_t)blockIdx.y * size;
  const TI* g = static_cast<const TI*>(a.g) + at;
  float* mom = a.momentum ? a.momentum + at : nullptr;
  double sum = 0;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < size; i += (int64_t)gridDim.x * 2048) {
    const int n = (int)min((int64_t)8, size - i);
    float u[8];
    load_row(g + i, n, vec, u);
    if (mom) {
      float m[8];
      load_row(mom + i, n, vec, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = momentum_of(a, m[e], u[e]);
        u[e] = update_of(a, m[e], u[e]);
      }
      store_row(mom + i, n, vec, m);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)u[e] * (double)u[e];
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) partial[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// v in two terms. (v is hidden from the compiler: where it is a product's sum, the compiler may
// take hi a second time, from that sum and in one rounding, and store another hi than the one that
// lo was taken against; the value was then off by 2^-11, once in some thousands.)
__device__ __forceinline__ void split(float v, f16& hi, f16& lo) {
  asm("" : "+v"(v));
  hi = (f16)v;
  lo = (f16)((v - (float)hi) * 2048.f);
}

// How a matrix of norm `norm` (eps included) is brought to values of X times about `scale`: by 2^p,
// and X = first times that. A norm that is not finite: no value of the result is.
struct Scale {
  double by;
  float first;
  __device__ __forceinline__ Scale(double norm, double scale) {
    int p = 0;
    first = __builtin_nanf("");
    if (norm == 0.0) {
      first = 0.f;
    } else if (norm < __builtin_huge_val()) {
      frexp(scale / norm, &p);
      --p;
      first = (float)(ldexp(1.0, -p) / norm);
    }
    by = ldexp(1.0, p);
  }
};

// u 2^p in fp16 terms, padded with zeros to rows x cols and in panels of 32 columns (and in `frags`, where
// given, as fragments), and each matrix's Scale::first. Eight threads take 64 columns of a row: whole lines of g, half lines of two panels.
template <typename TI, int TERMS>
__global__ __launch_bounds__(256) void scale_kernel(OrthArgs a, bool vec, const double* partial, int blocks,
                                                    double scale, f16* x, f16* frags, int64_t rows, int64_t cols,
                                                    int64_t plane, float* first) {
  __shared__ double sh[4];
  const int e = blockIdx.y;
  const double sq = block_sum((int)threadIdx.x < blocks ? partial[(int64_t)e * blocks + threadIdx.x] : 0.0, sh);
  const Scale sc(sqrt(sq) + (double)a.eps, scale);
  if (blockIdx.x == 0 && threadIdx.x == 0) first[e] = sc.first;
  const int64_t at = (int64_t)e * a.m * a.n;
  const uint32_t chunks = (uint32_t)rows * (uint32_t)(cols / 8), column = (uint32_t)rows * 8;  // (at most 2^31)
  const TI* g = static_cast<const TI*>(a.g) + at;
  const float* mom = a.momentum ? a.momentum + at : nullptr;
  f16* out = x + (int64_t)e * rows * cols;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < chunks; i += gridDim.x * 256) {
    const int64_t r = i % column / 8, c = (int64_t)(i / column) * 64 + i % 8 * 8;
    const int n = r < a.m ? (int)max(min((int64_t)8, a.n - c), (int64_t)0) : 0;
    float u[8] = {};
    if (n > 0) {
      load_row(g + r * a.n + c, n, vec, u);
      if (mom) {
        float m[8];
        load_row(mom + r * a.n + c, n, vec, m);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = update_of(a, m[k], u[k]);
      }
    }
    f16x8 hi, lo;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f16 h, l;
      split((float)((double)u[k] * sc.by), h, l);
      hi[k] = h;
      lo[k] = l;
    }
    f16* to = out + in_panels(rows, r, c);
    *reinterpret_cast<f16x8*>(to) = hi;
    if constexpr (TERMS == 2) {
      *reinterpret_cast<f16x8*>(to + plane) = lo;
      if (frags) {
        to = frags + (int64_t)e * rows * cols + in_fragments(rows, r, c);
        *reinterpret_cast<f16x8*>(to) = hi;
        *reinterpret_cast<f16x8*>(to + plane) = lo;
      }
    }
  }
}

// ---- products --------------------------------------------------------------------------
// Matrices of the iteration: rows x columns in panels, `mat` values each, their second terms
// `plane` values behind the first ones.
struct Operands {
  const f16* at;
  int64_t plane, mat;
  int rows;
};
// d[i][j] = f sum_k A(i, k) B(j, k) (+ p c[i][j] + q I), f times first[e]^power, of E matrices. An
// operand is summed over its columns (A[i][k]) or over its rows (A[k][i]).
struct ProductArgs {
  Operands a, b, c;
  int64_t K, rows, cols;  // padded
  f16* d;                 // rows x cols in fp16 terms, or
  int64_t d_plane;
  void* out;              // the result of the iteration, [m][n]
  int64_t m, n;
  int E, power, vec;
  float f, p, q, keep, rate;
  const float* first;
  // set by the launch: the parts that a tile's sum is in, and the most tiles that an XCD has
  int parts, rest;
  float* sums;
};

// One operand's stage in LDS: X of its output axis by 32 of the summed axis, as rows of 64 bytes,
// 16-byte chunk c of a row at c ^ swz(row): free of bank conflicts for both kinds of reads below. A
// direct load instruction moves 16 rows, lane l into slot l.
// Summed over columns (KS false): X rows of a panel. Summed over rows: 32 rows of each of X / 32 panels.
template <bool KS_, int X_>
struct Operand {
  static constexpr bool KS = KS_;
  static constexpr int X = X_, BYTES = X * 64, PW = BYTES / 1024 / 4;  // loads per wave and stage
  static_assert(PW >= 1, "whole loads per wave");
  static __device__ __forceinline__ int swz(int row) { return (row >> 2) & 3; }
  // LDS row of load j of a wave for this lane, and the source chunk that goes into its slot
  static __device__ __forceinline__ int row(int j, int wave, int ln) { return (wave * PW + j) * 16 + ln / 4; }
  static __device__ __forceinline__ int chunk(int j, int wave, int ln) { return (ln % 4) ^ swz(row(j, wave, ln)); }
  // byte offset of this lane's fragment of the 32 rows (columns) from x0 (substep 0)
  static __device__ __forceinline__ int frag(int x0, int ln) {
    if constexpr (!KS) {
      const int m = x0 + (ln & 31);
      return m * 64 + ((ln >> 5) ^ swz(m)) * 16;
    } else {
      const int g = ln >> 4, k = (g >> 1) * 8 + ((ln & 15) >> 2), n = (g & 1) * 16 + 4 * (ln & 3);
      return (x0 + k) * 64 + ((n >> 3) ^ swz(k)) * 16 + ((n >> 2) & 1) * 8;
    }
  }
  // The fragment of substep s, k = 16 s + 8 h .. + 7 (h = lane / 32); over rows by transposing reads.
  static __device__ __forceinline__ u32x4 read(const char* st, int at, int s) {
    if constexpr (!KS) {
      return *reinterpret_cast<const u32x4*>(st + (at ^ (32 * s)));
    } else {
      // (swz of rows 4 on is that of these, which is even, and 1)
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(st + at + 1024 * s));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(st + (at ^ 16) + 256 + 1024 * s));
      return __builtin_bit_cast(u32x4, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
  }
};

template <int BM_, bool AKS, bool BKS, int TERMS_>
struct Tile {
  static constexpr int BM = BM_, BK = 32, TERMS = TERMS_;
  typedef Operand<AKS, BM> A;
  typedef Operand<BKS, BM> B;
  static constexpr int WM = BM / 2, MB = WM / 32, SUB = BK / 16;  // 2 x 2 waves
  // a stage: A's terms, then B's
  static constexpr int STAGE = TERMS * (A::BYTES + B::BYTES), LPS = TERMS * (A::PW + B::PW);
  static constexpr int OUT_BYTES = BM == 64 ? 4096 : 32 * WM * 2;  // LDS of each wave for its output
  static constexpr int LDS = kStages * STAGE + 4 * OUT_BYTES, PER_CU = 160 * 1024 / LDS;
  static constexpr int SLOTS = PER_CU * (kCus / kXcds);  // workgroups of an XCD that are resident
  static constexpr int MFMAS = TERMS == 2 ? 3 : 1;     // per pair of fragments
};

template <class G>
struct Frags {
  u32x4 a[G::TERMS][G::SUB][G::MB], b[G::TERMS][G::SUB][G::MB];
};

template <class G>
struct Wave {
  int a_at[G::MB], b_at[G::MB];
  f32x16 acc[G::MB][G::MB];  // [columns][rows]; two terms: hi hi of one ring turn
  f32x16 cross[G::TERMS == 2 ? G::MB : 1][G::TERMS == 2 ? G::MB : 1];
  f32x16 sum[G::TERMS == 2 ? G::MB : 1][G::TERMS == 2 ? G::MB : 1];

  // LDS read r of a stage's fragments (r constant at every call)
  __device__ __forceinline__ void read(int r, const char* st, Frags<G>& F) const {
    const int s = r / (2 * G::TERMS * G::MB), i = r % (2 * G::TERMS * G::MB), t = i / G::MB % G::TERMS, b = i % G::MB;
    if (i < G::TERMS * G::MB) F.a[t][s][b] = G::A::read(st + t * G::A::BYTES, a_at[b], s);
    else F.b[t][s][b] = G::B::read(st + G::TERMS * G::A::BYTES + t * G::B::BYTES, b_at[b], s);
  }
  __device__ __forceinline__ void mfma(int i, const Frags<G>& F) {
    const int s = i / (G::MB * G::MB * G::MFMAS), nb = i / (G::MB * G::MFMAS) % G::MB, mb = i / G::MFMAS % G::MB;
    const int k = i % G::MFMAS;  // hi hi, lo hi, hi lo
    const u32x4 b = F.b[k == 2 ? 1 : 0][s][nb], a = F.a[k == 1 ? 1 : 0][s][mb];
    f32x16& to = k ? cross[nb][mb] : acc[nb][mb];
    to = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), to, 0, 0, 0);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nb = 0; nb < G::MB; ++nb)
#pragma unroll
      for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          acc[nb][mb][r] = 0.f;
          if constexpr (G::TERMS == 2) cross[nb][mb][r] = sum[nb][mb][r] = 0.f;
        }
  }
  // two terms: a turn's sums go to the others (last: with the cross terms, back into acc)
  __device__ __forceinline__ void flush(bool last) {
    if constexpr (G::TERMS == 2) {
#pragma unroll
      for (int nb = 0; nb < G::MB; ++nb)
#pragma unroll
        for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float v = sum[nb][mb][r] + acc[nb][mb][r];
            if (last) {
              acc[nb][mb][r] = v + kLo * cross[nb][mb][r];
            } else {
              sum[nb][mb][r] = v;
              acc[nb][mb][r] = 0.f;
            }
          }
    }
  }
};

// A tile's sources: where its operands begin (uniform), each lane's offsets of its loads from
// there, in bytes, and the bytes per stage and from term to term.
template <class G>
struct Loader {
  const char *a, *b;
  uint32_t va[G::A::PW], vb[G::B::PW];
  int64_t sa, sb, pa, pb;
  int wave;
};

// One tile of a matrix, ring turns [u0, u1) of its sum; part: where the sum of these goes, -1:
// it is the whole one.
struct Item {
  int e, i, j, u0, u1, part;
};

// Stage J of a turn: wait for this wave's loads of the next stage and its own LDS reads of this
// one, then the barrier: after it the next stage is whole in LDS and this stage's buffer is
// free. Then the stage's MFMAs, with the reads of the next stage into Fn and the refill of this
// buffer (stage J of the turn that begins at ra, rb) spread between them.
template <class G, int J>
struct Step {
  static __device__ __forceinline__ void load(const Loader<G>& ld, int g, const char* ra, const char* rb, char* st) {
    constexpr int NA = G::TERMS * G::A::PW;
    const bool is_a = g < NA;
    const int i = is_a ? g : g - NA, pw = is_a ? G::A::PW : G::B::PW, t = i / pw, l = i % pw;
    const char* p = is_a ? ra + (J * ld.sa + t * ld.pa) + ld.va[l] : rb + (J * ld.sb + t * ld.pb) + ld.vb[l];
    char* to = is_a ? st + t * G::A::BYTES + (ld.wave * G::A::PW + l) * 1024
                    : st + G::TERMS * G::A::BYTES + t * G::B::BYTES + (ld.wave * G::B::PW + l) * 1024;
    __builtin_amdgcn_global_load_lds(p, (lds_void*)to, 16, 0, 0);
  }
  // IDLE: a wave without values of the tile only loads (and reads the next item's first fragments).
  template <bool IDLE>
  static __device__ __forceinline__ void run(char* const (&ring)[kStages], const Loader<G>& ld, const char* ra,
                                             const char* rb, Wave<G>& w, Frags<G>& Fc, Frags<G>& Fn) {
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<(kStages - 2) * G::LPS>();
    wait_lgkmcnt0();
    sync_point();
    constexpr int NM = G::SUB * G::MB * G::MB * G::MFMAS, NR = G::SUB * 2 * G::TERMS * G::MB, NG = G::LPS;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int m = NM * g / NG; m < NM * (g + 1) / NG; ++m) {
        if constexpr (!IDLE) w.mfma(m, Fc);
      }
#pragma unroll
      for (int r = NR * g / NG; r < NR * (g + 1) / NG; ++r) {
        if constexpr (!IDLE || J == kStages - 1) w.read(r, ring[(J + 1) % kStages], Fn);
      }
      load(ld, g, ra, rb, ring[J]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Tiles of a matrix: all, column block after column block, rows outer and the block's columns
// inner; or, SYM, those on and below the diagonal in the same order.
template <bool SYM>
__device__ __forceinline__ void locate_tile(int at, int Mt, int Nt, Item& t) {
  if constexpr (SYM) {
    const int per = Mt * (Mt + 1) / 2;
    t.e = at / per;
    int r = at - t.e * per, c0 = 0;
    for (;; c0 += kColBlock) {
      const int left = Mt - c0, w = min(left, kColBlock), n = w * (w + 1) / 2 + (left - w) * w;
      if (r < n) {
        int row = 0;
        while (row < w && r > row) r -= ++row;  // the block's corner: rows of 1, 2, .. tiles
        if (row < w) {
          t.i = c0 + row;
          t.j = c0 + r;
        } else {
          t.i = c0 + w + r / w;
          t.j = c0 + r % w;
        }
        return;
      }
      r -= n;
    }
  } else {
    const int per = Mt * Nt;
    t.e = at / per;
    const int r = at - t.e * per, blk = r / (Mt * kColBlock), cols = min(kColBlock, Nt - blk * kColBlock);
    const int in = r - blk * Mt * kColBlock;
    t.i = in / cols;
    t.j = blk * kColBlock + in % cols;
  }
}
// The grid of tiles, and the XCD's eighth of all of them.
template <class G, bool SYM>
struct Share {
  int Mt, Nt, lo, n, turns;
  __device__ __forceinline__ Share(const ProductArgs& a, int xcd) {
    Mt = (int)((a.rows + G::BM - 1) / G::BM);
    Nt = (int)((a.cols + G::BM - 1) / G::BM);
    const int64_t all = (int64_t)a.E * (SYM ? Mt * (Mt + 1) / 2 : Mt * Nt);
    lo = (int)(all * xcd / kXcds);
    n = (int)(all * (xcd + 1) / kXcds) - lo;
    turns = (int)(a.K / (kStages * G::BK));
  }
  // items: the tiles, or their parts, a tile's one after another
  __device__ __forceinline__ int items(const ProductArgs& a) const { return n * a.parts; }
  __device__ __forceinline__ Item locate(const ProductArgs& a, int xcd, int at) const {
    Item t;
    t.part = -1;
    t.u0 = 0;
    t.u1 = turns;
    if (a.parts > 1) {
      const int tile = at / a.parts, part = at - tile * a.parts;
      t.u0 = turns * part / a.parts;
      t.u1 = turns * (part + 1) / a.parts;
      t.part = (xcd * a.rest + tile) * a.parts + part;
      at = tile;
    }
    locate_tile<SYM>(lo + at, Mt, Nt, t);
    return t;
  }
};

template <class G>
__device__ __forceinline__ void make_loader(const ProductArgs& a, const Item& t, int lane, Loader<G>& ld) {
  const int ln = here(lane);
  auto side = [&](auto op, const Operands& o, int x0, int64_t size, const char*& base, uint32_t* v, int64_t& step) {
    typedef decltype(op) Op;
    const int last = (int)size - 1 - x0;  // (256-row tiles: the last row or panel again past the end)
    step = Op::KS ? 32 * 64 : (int64_t)o.rows * 64;
    base = reinterpret_cast<const char*>(o.at + t.e * o.mat + (Op::KS ? (int64_t)x0 * o.rows : (int64_t)x0 * 32)) +
           t.u0 * kStages * step;
#pragma unroll
    for (int j = 0; j < Op::PW; ++j) {
      const int row = Op::row(j, ld.wave, ln), chunk = Op::chunk(j, ld.wave, ln) * 16;
      v[j] = Op::KS ? (uint32_t)(min(row >> 5, last >> 5) * o.rows + (row & 31)) * 64 + chunk
                    : (uint32_t)min(row, last) * 64 + chunk;
    }
  };
  side(typename G::A{}, a.a, t.i * G::BM, a.rows, ld.a, ld.va, ld.sa);
  side(typename G::B{}, a.b, t.j * G::BM, a.cols, ld.b, ld.vb, ld.sb);
}

// A wave whose quarter of the tile lies past the matrix (256-row tiles), or above the diagonal of
// a symmetric one: that quarter is the transpose of another wave's.
template <class G, bool SYM>
__device__ __forceinline__ bool idle(const ProductArgs& a, const Item& t, int wm, int wn) {
  const int m0 = t.i * G::BM + wm * G::WM, n0 = t.j * G::BM + wn * G::WM;
  return m0 >= a.rows || n0 >= a.cols || (SYM && m0 < n0);
}

// The values of a chunk of 8 in fp16 terms.
template <int TERMS>
struct Terms {
  u32x4 hi, lo;
  __device__ __forceinline__ void load(const Operands& o, int e, int64_t row, int64_t col) {
    const f16* p = o.at + e * o.mat + in_panels(o.rows, row, col);
    hi = ld16(p);
    if constexpr (TERMS == 2) lo = ld16(p + o.plane);
  }
  __device__ __forceinline__ float value(int k) const {
    const float h = (float)__builtin_bit_cast(f16x8, hi)[k];
    if constexpr (TERMS == 2) return h + (float)__builtin_bit_cast(f16x8, lo)[k] * kLo;
    return h;
  }
};

// A chunk of 8 of the weights, where its row is whole chunks.
template <typename TO>
struct Weights {
  u32x4 v[sizeof(TO) / 2];
  __device__ __forceinline__ void load(const TO* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(TO) / 2; ++i) v[i] = ld16(p + i * (16 / sizeof(TO)));
  }
  __device__ __forceinline__ float value(int k) const {
    if constexpr (sizeof(TO) == 2) return (float)__builtin_bit_cast(bf16x8, v[0])[k];
    else return __builtin_bit_cast(f32x4, v[k / 4])[k % 4];
  }
};

// What a product does with its sums: f S, as fragments; f S; f S + p c + q I; the result; it into the weights.
enum { kFragments, kProduct, kPolynomial, kLast, kUpdate };

// acc[nb][mb][4 q + i] is row lane % 32 of block mb, column 8 q + 4 (lane / 32) + i of block nb.
// 32 rows at a time go through a piece of LDS of the wave's own (16-byte chunk c of a row at
// c ^ (row % chunks)) and leave as whole row segments; c's values, and the weights that the result is
// applied to, are loaded a pass ahead.
// The transposed tile leaves by the same piece of LDS, column by column.
// (only: that pass alone)
template <class G>
struct Passes {
  static constexpr int SEG = G::OUT_BYTES / 32, CHUNKS = SEG / 16, COLS = SEG / 4, BLOCKS = COLS / 32;
  static constexpr int PER = COLS / 8, RPS = 64 / PER, N = 32 / RPS, ALL = G::MB * (G::MB / BLOCKS);
};
template <class G, bool SYM, int KIND, typename TO>
__device__ __forceinline__ void store_tile(const ProductArgs& a, const Item& t, int wm, int wn, int lane, char* buf,
                                           const Wave<G>& w, int only = -1) {
  typedef Passes<G> S;
  constexpr int TERMS = G::TERMS, SEG = S::SEG, CHUNKS = S::CHUNKS, COLS = S::COLS, BLOCKS = S::BLOCKS;
  constexpr int PER = S::PER, RPS = S::RPS, N = S::N, PASSES = S::ALL;
  const int ln = here(lane);
  const int64_t m0 = (int64_t)t.i * G::BM + wm * G::WM, n0 = (int64_t)t.j * G::BM + wn * G::WM;
  float f = a.f;
  for (int i = 0; i < a.power; ++i) f *= a.first[t.e];
  const int r0 = ln / PER, c0 = ln % PER;
  constexpr bool AHEAD = KIND == kPolynomial || KIND == kUpdate;
  Terms<TERMS> old[KIND == kPolynomial ? 2 : 1][N];
  Weights<TO> weights[KIND == kUpdate ? 2 : 1][N];
  auto place = [&](int64_t r, int64_t c) {
    return KIND == kFragments ? in_fragments(a.rows, r, c) : in_panels(a.rows, r, c);
  };
  auto row_of = [&](int pass, int i) { return m0 + pass / (G::MB / BLOCKS) * 32 + i * RPS + r0; };
  auto col_of = [&](int pass) { return n0 + pass % (G::MB / BLOCKS) * COLS + c0 * 8; };
  auto fetch = [&](int pass) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t row = row_of(pass, i), col = col_of(pass);
      if constexpr (KIND == kPolynomial) old[pass % 2][i].load(a.c, t.e, row, col);
      if constexpr (KIND == kUpdate) {
        // (past the end the first ones, which nobody takes)
        const bool in = row < a.m && col < a.n;
        if (a.vec) weights[pass % 2][i].load(static_cast<const TO*>(a.out) + (in ? ((int64_t)t.e * a.m + row) * a.n + col : 0));
      }
    }
  };
  if constexpr (AHEAD) {
    if (only < 0) fetch(0);
  }
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
    if (only >= 0 && pass != only) continue;
    __builtin_amdgcn_sched_barrier(0);  // (one pass's registers at a time)
    const int mb = pass / (G::MB / BLOCKS), nb0 = pass % (G::MB / BLOCKS) * BLOCKS, r = ln & 31;
    if constexpr (AHEAD) {
      if (only >= 0) fetch(pass);
      else if (pass + 1 < PASSES) fetch(pass + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int nb = 0; nb < BLOCKS; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = nb * 8 + 2 * q + (ln >> 5);
        const f32x16& v = w.acc[nb0 + nb][mb];
        *reinterpret_cast<f32x4*>(buf + r * SEG + ((c ^ (r % CHUNKS)) << 4)) =
            f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    f16x8 hi[N], lo[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = i * RPS + r0;
      f32x4 s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s[h] = *reinterpret_cast<const f32x4*>(buf + row * SEG + (((2 * c0 + h) ^ (row % CHUNKS)) << 4));
      const int64_t gr = row_of(pass, i), gc = col_of(pass);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = f * s[k / 4][k % 4];
        if constexpr (KIND == kPolynomial)
          v[k] += a.p * old[pass % 2][i].value(k) + (gr == gc + k ? a.q : 0.f);
      }
      if constexpr (KIND >= kLast) {
        if (gr >= a.m || gc >= a.n) continue;
        const int n = (int)min((int64_t)8, a.n - gc);
        TO* o = static_cast<TO*>(a.out) + ((int64_t)t.e * a.m + gr) * a.n + gc;
        if constexpr (KIND == kUpdate) {
          float w[8];
          if (!a.vec) load_row(o, n, false, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = a.keep * (a.vec ? weights[pass % 2][i].value(k) : w[k]) - a.rate * v[k];
        }
        store_row(o, n, a.vec, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          f16 h, l;
          split(v[k], h, l);
          hi[i][k] = h;
          lo[i][k] = l;
        }
        f16* d = a.d + t.e * a.rows * a.cols + place(gr, gc);
        *reinterpret_cast<f16x8*>(d) = hi[i];
        if constexpr (TERMS == 2) *reinterpret_cast<f16x8*>(d + a.d_plane) = lo[i];
      }
    }
    if constexpr (SYM && KIND < kLast) {
      if (m0 != n0) {
        // [32 rows][columns] of fp16, chunk c of a row at c ^ swz(row), and out of there in columns
        // by transposing reads: 16 columns at a time, lane l with rows 8 (l / 16) .. + 7 of column l % 16
        auto swz = [](int row) { return ((0xCA60 >> (4 * (row & 3))) & 15) % PER; };
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int row = i * RPS + r0;
            *reinterpret_cast<f16x8*>(buf + row * (COLS * 2) + ((c0 ^ swz(row)) << 4)) = term ? lo[i] : hi[i];
          }
#pragma unroll
          for (int i = 0; i < COLS / 16; ++i) {
            const int row = 8 * (ln >> 4) + (ln & 15) / 4, col = 16 * i + 4 * (ln & 3);
            const char* p = buf + row * (COLS * 2) + (((col >> 3) ^ swz(row)) << 4) + (col & 4) * 2;
            const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
            const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * COLS * 2));
            const s16x8 v{v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
            const int64_t gr = n0 + pass % (G::MB / BLOCKS) * COLS + 16 * i + (ln & 15), gc = m0 + mb * 32 + 8 * (ln >> 4);
            st16(a.d + t.e * a.rows * a.cols + place(gr, gc) + term * a.d_plane, __builtin_bit_cast(u32x4, v));
          }
        }
      }
    }
  }
}

// A part's sums, as they lie in the registers: 16 bytes of every lane at a time.
template <class G>
__device__ __forceinline__ float* part_at(const ProductArgs& a, int64_t part, int wave, int lane) {
  return a.sums + (part * G::BM * G::BM + wave * G::WM * G::WM) + lane * 4;
}
template <class G>
__device__ __forceinline__ void put_part(const ProductArgs& a, int part, int wave, int lane, const Wave<G>& w) {
  float* p = part_at<G>(a, part, wave, here(lane));
#pragma unroll
  for (int nb = 0; nb < G::MB; ++nb)
#pragma unroll
    for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& v = w.acc[nb][mb];
        *reinterpret_cast<f32x4*>(p + ((nb * G::MB + mb) * 4 + q) * 256) =
            f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
}

// Workgroups take their XCD's items in strides of the XCD's workgroups, as one stream of
// stages: the last ring turn of an item loads the first one of the next. The 256-row tiles take all 512 registers:
// six of them keep one value in scratch, read at a tile's end, and the one of operands summed over rows five,
// in the last turn of a tile; the turns before it have no scratch accesses.
template <class G, bool SYM, int KIND, typename TO>
__global__ __launch_bounds__(256, 1) void product_kernel(ProductArgs a) {
  // (an array of its own for each stage: the compiler then sees that the reads of one stage
  // do not wait for the loads into another)
  __shared__ __attribute__((aligned(1024))) char s0[G::STAGE], s1[G::STAGE], s2[G::STAGE], s3[G::STAGE];
  __shared__ __attribute__((aligned(1024))) char outs[4 * G::OUT_BYTES];
  char* const ring[kStages] = {s0, s1, s2, s3};
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / 2, wn = wave % 2;
  const int xcd = blockIdx.x % kXcds, slots = gridDim.x / kXcds;
  const Share<G, SYM> share(a, xcd);
  const int items = share.items(a);
  int at = blockIdx.x / kXcds;
  if (at >= items) return;

  Wave<G> w;
#pragma unroll
  for (int j = 0; j < G::MB; ++j) {
    w.a_at[j] = G::A::frag(wm * G::WM + j * 32, ln);
    w.b_at[j] = G::B::frag(wn * G::WM + j * 32, ln);
  }
  Loader<G> ld;
  ld.wave = wave;
  ld.pa = a.a.plane * 2;
  ld.pb = a.b.plane * 2;
  Item t = share.locate(a, xcd, at);
  make_loader<G>(a, t, ln, ld);
  Frags<G> F0, F1;
#pragma unroll
  for (int g = 0; g < G::LPS; ++g) Step<G, 0>::load(ld, g, ld.a, ld.b, s0);
#pragma unroll
  for (int g = 0; g < G::LPS; ++g) Step<G, 1>::load(ld, g, ld.a, ld.b, s1);
#pragma unroll
  for (int g = 0; g < G::LPS; ++g) Step<G, 2>::load(ld, g, ld.a, ld.b, s2);
#pragma unroll
  for (int g = 0; g < G::LPS; ++g) Step<G, 3>::load(ld, g, ld.a, ld.b, s3);
  wait_vmcnt<(kStages - 1) * G::LPS>();
  sync_point();
#pragma unroll
  for (int r = 0; r < G::SUB * 2 * G::TERMS * G::MB; ++r) w.read(r, s0, F0);

  for (;;) {
    w.clear();
    const Item cur = t;
    at += slots;
    const bool more = at < items;
    if (more) t = share.locate(a, xcd, at);
#define MOE_TURN(IDLE, RA, RB)                                         \
  {                                                                    \
    const char *const ra = (RA), *const rb = (RB);                     \
    Step<G, 0>::template run<IDLE>(ring, ld, ra, rb, w, F0, F1);       \
    Step<G, 1>::template run<IDLE>(ring, ld, ra, rb, w, F1, F0);       \
    Step<G, 2>::template run<IDLE>(ring, ld, ra, rb, w, F0, F1);       \
    Step<G, 3>::template run<IDLE>(ring, ld, ra, rb, w, F1, F0);       \
  }
    // the last turn loads the next item's first (without one, this item's, never used)
    if (idle<G, SYM>(a, cur, wm, wn)) {
      for (int u = 1; u < cur.u1 - cur.u0; ++u)
        MOE_TURN(true, ld.a + u * kStages * ld.sa, ld.b + u * kStages * ld.sb);
      if (more) make_loader<G>(a, t, ln, ld);
      MOE_TURN(true, ld.a, ld.b);
    } else {
      for (int u = 1; u < cur.u1 - cur.u0; ++u) {
        MOE_TURN(false, ld.a + u * kStages * ld.sa, ld.b + u * kStages * ld.sb);
        w.flush(false);
      }
      if (more) make_loader<G>(a, t, ln, ld);
      MOE_TURN(false, ld.a, ld.b);
      w.flush(true);
      if (cur.part >= 0) put_part<G>(a, cur.part, wave, ln, w);
      else store_tile<G, SYM, KIND, TO>(a, cur, wm, wn, ln, outs + wave * G::OUT_BYTES, w);
    }
#undef MOE_TURN
    if (!more) break;
  }
  wait_vmcnt<0>();  // the loads that nobody reads have landed before the LDS is given back
}

// The sums of the tiles that are in parts, in order: one pass of what one of the product's waves
// holds of a tile per workgroup.
template <class G, bool SYM, int KIND, typename TO>
__global__ __launch_bounds__(64, 1) void join_kernel(ProductArgs a) {
  typedef Passes<G> S;
  __shared__ __attribute__((aligned(1024))) char buf[G::OUT_BYTES];
  const int pass = blockIdx.x % S::ALL, quarter = blockIdx.x / S::ALL, ln = threadIdx.x;
  const int wave = quarter % 4, tile = quarter / 4 / kXcds, xcd = quarter / 4 % kXcds;
  const Share<G, SYM> share(a, xcd);
  if (tile >= share.n) return;
  const Item t = share.locate(a, xcd, tile * a.parts);
  if (idle<G, SYM>(a, t, wave / 2, wave % 2)) return;
  Wave<G> w;
#pragma unroll
  for (int p = 0; p < S::ALL; ++p) {
    if (p != pass) continue;
    constexpr int WIDE = G::MB / S::BLOCKS, AHEAD = 8;  // (parts in flight: each waits for memory)
    f32x4 sum[S::BLOCKS * 4] = {};
    for (int i = 0; i < a.parts; i += AHEAD) {
      f32x4 v[AHEAD][S::BLOCKS * 4];
#pragma unroll
      for (int h = 0; h < AHEAD; ++h) {
        const float* from = part_at<G>(a, t.part + min(i + h, a.parts - 1), wave, ln);
#pragma unroll
        for (int k = 0; k < S::BLOCKS * 4; ++k) {
          const int block = (p % WIDE * S::BLOCKS + k / 4) * G::MB + p / WIDE;
          v[h][k] = *reinterpret_cast<const f32x4*>(from + (block * 4 + k % 4) * 256);
        }
      }
#pragma unroll
      for (int h = 0; h < AHEAD; ++h) {
        if (i + h >= a.parts) continue;
#pragma unroll
        for (int k = 0; k < S::BLOCKS * 4; ++k) sum[k] += v[h][k];
      }
    }
#pragma unroll
    for (int k = 0; k < S::BLOCKS * 4; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x) w.acc[p % WIDE * S::BLOCKS + k / 4][p / WIDE][k % 4 * 4 + x] = sum[k][x];
  }
  store_tile<G, SYM, KIND, TO>(a, t, wave / 2, wave % 2, ln, buf, w, pass);
}

// Whether the next two steps of a matrix kept in two terms share a Gram matrix. Of few singular values
// a rounding of A is not averaged away, and the first pair multiplies it most: with up to kFewValues of
// them an odd step comes first, alone (off by, in 1e-7 of the norm, pairs first and so: 16 x 680 30, 13;
// 24 x 2000 13, 12; but 32 x 380 9, 12; 64 x 128 11, 17; plain fp32 13, 10, 11, 12).
constexpr int kFewValues = 24;
__host__ __device__ inline bool pair_in_two_terms(int64_t side, int left) {
  return side > kFewValues ? left >= 2 : left > 0 && left % 2 == 0;
}

// ---- small matrices --------------------------------------------------------------------
// Products of matrices that stay in LDS, by one workgroup of eight waves per matrix: what a launch
// of its own for every product costs (5 us where nothing else counts) would be most of their time.

constexpr int kWaves = 8, kThreads = 64 * kWaves;

// A matrix in two fp16 terms in LDS, rows of `row` bytes (a multiple of 128). 16-byte chunk c of a
// row lies at c ^ swz(row): free of bank conflicts for 32 rows' chunks as for transposing reads.
struct InLds {
  char* hi;
  char* lo;
  int row;
  static __device__ __forceinline__ int swz(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }
  __device__ __forceinline__ int at(int r, int c) const { return r * row + (((c >> 3) ^ swz(r)) << 4) + (c & 7) * 2; }
  // fragment of 32 rows from x0, columns k0 .. k0 + 15 of the summed axis
  static __device__ __forceinline__ f16x8 rows(const char* p, const InLds& m, int x0, int k0, int ln) {
    return *reinterpret_cast<const f16x8*>(p + m.at(x0 + (ln & 31), k0 + 8 * (ln >> 5)));
  }
  // fragment of 32 columns from x0, rows k0 .. k0 + 15 of the summed axis
  static __device__ __forceinline__ f16x8 columns(const char* p, const InLds& m, int x0, int k0, int ln) {
    const int g = ln >> 4, k = k0 + 8 * (g >> 1) + ((ln & 15) >> 2), n = x0 + 16 * (g & 1) + 4 * (ln & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + m.at(k, n)));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + m.at(k + 4, n)));
    return __builtin_bit_cast(f16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
  }
  // four values of row r from column c (a multiple of 4)
  __device__ __forceinline__ void put(int r, int c, const float (&v)[4]) const {
    f16x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16 a, b;
      split(v[i], a, b);
      h[i] = a;
      l[i] = b;
    }
    *reinterpret_cast<f16x4*>(hi + at(r, c)) = h;
    *reinterpret_cast<f16x4*>(lo + at(r, c)) = l;
  }
  __device__ __forceinline__ void get(int r, int c, float (&v)[4]) const {
    const f16x4 h = *reinterpret_cast<const f16x4*>(hi + at(r, c)), l = *reinterpret_cast<const f16x4*>(lo + at(r, c));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)h[i] + kLo * (float)l[i];
  }
};

// N blocks of 32 rows of A from i0 and 32 columns from j0 on, of A B^T (or, COLUMNS, A B) over K:
// value 4 q + t of lane l is row l % 32, column 8 q + 4 (l / 32) + t of a block.
template <bool COLUMNS, int N>
__device__ __forceinline__ void lds_blocks(const InLds& A, const InLds& B, int i0, int j0, int K, int lane,
                                           f32x16 (&out)[N]) {
  const int ln = here(lane);
  f32x16 cross[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    out[n] = f32x16{};
    cross[n] = f32x16{};
  }
  for (int k1 = 0; k1 < K; k1 += 64) {  // (sums of hi hi of 64 terms, as in the tiles above)
    f32x16 acc[N];
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = f32x16{};
#pragma unroll
    for (int k = 0; k < 64; k += 16) {
      const f16x8 ah = InLds::rows(A.hi, A, i0, k1 + k, ln), al = InLds::rows(A.lo, A, i0, k1 + k, ln);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        f16x8 bh, bl;
        if constexpr (COLUMNS) {
          bh = InLds::columns(B.hi, B, j0 + 32 * n, k1 + k, ln);
          bl = InLds::columns(B.lo, B, j0 + 32 * n, k1 + k, ln);
        } else {
          bh = InLds::rows(B.hi, B, j0 + 32 * n, k1 + k, ln);
          bl = InLds::rows(B.lo, B, j0 + 32 * n, k1 + k, ln);
        }
        acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bh, ah, acc[n], 0, 0, 0);
        cross[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bh, al, cross[n], 0, 0, 0);
        cross[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bl, ah, cross[n], 0, 0, 0);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) out[n] += acc[n];
  }
#pragma unroll
  for (int n = 0; n < N; ++n) out[n] += kLo * cross[n];
}

// d = u v, or a I + b u + c u^2 (POLY), of SIDE x SIDE symmetric matrices that commute; d may be u or v.
// All waves call it; it ends with d whole.
template <int SIDE, bool POLY>
__device__ __forceinline__ void lds_square(const OrthArgs& a, const InLds& u, const InLds& v, const InLds& d, int wave,
                                           int ln) {
  constexpr int BLOCKS = SIDE * SIDE / 1024, EACH = BLOCKS >= kWaves ? BLOCKS / kWaves : 1;
  f32x16 r[EACH];
  float old[POLY ? EACH : 1][4][4];
  const bool mine = wave * EACH < BLOCKS;
  const int i0 = wave * EACH / (SIDE / 32) * 32;
  auto j0 = [&](int n) { return (wave * EACH + n) % (SIDE / 32) * 32; };
  const int row = i0 + (ln & 31), col = 4 * (ln >> 5);
  if (mine) {
    lds_blocks<false>(u, v, i0, j0(0), SIDE, ln, r);
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
      if constexpr (POLY) {
#pragma unroll
        for (int q = 0; q < 4; ++q) u.get(row, j0(n) + 8 * q + col, old[n][q]);
      }
    }
  }
  __syncthreads();  // (everyone has read what d is written over)
  if (mine) {
#pragma unroll
    for (int n = 0; n < EACH; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float w[4];
        const int c = j0(n) + 8 * q + col;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          w[t] = r[n][4 * q + t];
          if constexpr (POLY) w[t] = a.c * w[t] + a.b * old[n][q][t] + (row == c + t ? a.a : 0.f);
        }
        d.put(row, c, w);
      }
  }
  __syncthreads();
}

// Everything between a Gram matrix, in U, and what X is multiplied by, to P: P(A), or with `two` P' P.
template <int SIDE>
__device__ __forceinline__ void lds_polynomial(const OrthArgs& a, bool two, const InLds& U, const InLds& P, int wave,
                                               int ln) {
  lds_square<SIDE, true>(a, U, U, P, wave, ln);
  if (two) {
    lds_square<SIDE, false>(a, P, U, U, wave, ln);
    lds_square<SIDE, false>(a, P, U, U, wave, ln);  // A'
    lds_square<SIDE, true>(a, U, U, U, wave, ln);   // P'
    lds_square<SIDE, false>(a, U, P, P, wave, ln);
  }
}
// The same from and to global memory, for short sides of 65 to 128: 17 us with `two`, in place of five launches of 5 us.
__global__ __launch_bounds__(kThreads) void polynomial_kernel(OrthArgs a, bool two, const f16* A, f16* out,
                                                              int64_t plane) {
  constexpr int SIDE = kPad;
  __shared__ __attribute__((aligned(1024))) char lds[2][2][SIDE * SIDE * 2];
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const InLds U{lds[0][0], lds[0][1], SIDE * 2}, P{lds[1][0], lds[1][1], SIDE * 2};
  const int64_t at = (int64_t)blockIdx.x * SIDE * SIDE;
  constexpr int CHUNKS = SIDE / 8;
#pragma unroll
  for (int i = threadIdx.x; i < SIDE * CHUNKS; i += kThreads) {
    const int r = i / CHUNKS, c = i % CHUNKS * 8;
    *reinterpret_cast<u32x4*>(U.hi + U.at(r, c)) = ld16(A + at + in_panels(SIDE, r, c));
    *reinterpret_cast<u32x4*>(U.lo + U.at(r, c)) = ld16(A + plane + at + in_panels(SIDE, r, c));
  }
  __syncthreads();
  lds_polynomial<SIDE>(a, two, U, P, wave, ln);
#pragma unroll
  for (int i = threadIdx.x; i < SIDE * CHUNKS; i += kThreads) {
    const int r = i / CHUNKS, c = i % CHUNKS * 8;
    st16(out + at + in_panels(SIDE, r, c), *reinterpret_cast<const u32x4*>(P.hi + P.at(r, c)));
    st16(out + plane + at + in_panels(SIDE, r, c), *reinterpret_cast<const u32x4*>(P.lo + P.at(r, c)));
  }
}

// X of up to 64 x 384 in LDS, of a matrix whose short side is at most 64, or of 384 of its longer side.
constexpr int kSmallSide = 64, kSmallLong = 384;

// Value (i, j) of X, i of the short side, is value (i, j) or (j, i) of the matrix.
struct Shape {
  int m, n;
  bool tall;
  __device__ __forceinline__ explicit Shape(const OrthArgs& a) : m((int)a.m), n((int)a.n), tall(a.m > a.n) {}
  __device__ __forceinline__ int64_t at(int i, int j) const { return tall ? (int64_t)j * n + i : (int64_t)i * n + j; }
};

// Columns c0 .. c0 + w - 1 of X 2^p into LDS (of l columns, zeros behind w). All threads; ends with it whole.
template <typename TI>
__device__ __forceinline__ void lds_load(const OrthArgs& a, const Shape& sh, const TI* g, const float* mom, double by, int c0,
                                         int w, int l, const InLds& X) {
  for (int i = threadIdx.x; i < kSmallSide * l / 8; i += kThreads) {
    *reinterpret_cast<u32x4*>(X.hi + i * 16) = u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(X.lo + i * 16) = u32x4{0, 0, 0, 0};
  }
  __syncthreads();
  // (along the matrix's rows)
  const int s = sh.tall ? sh.n : sh.m, in = sh.tall ? s : w, size = s * w;
  int r = threadIdx.x / in, c = threadIdx.x - r * in;
  for (int k = threadIdx.x; k < size; k += kThreads) {
    const int i = sh.tall ? c : r, j = sh.tall ? r : c;
    const int64_t at = sh.at(i, c0 + j);
    float u = (float)g[at];
    if (mom) u = update_of(a, mom[at], u);
    f16 h, lo;
    split((float)((double)u * by), h, lo);
    const int to = X.at(i, j);
    *reinterpret_cast<f16*>(X.hi + to) = h;
    *reinterpret_cast<f16*>(X.lo + to) = lo;
    r += kThreads / in;
    c += kThreads % in;
    if (c >= in) {
      c -= in;
      ++r;
    }
  }
  __syncthreads();
}

// f P X: the whole is computed, all waves wait for it, then put(i, j, values j .. j + 3).
template <class Put>
__device__ __forceinline__ void lds_times(const InLds& P, const InLds& X, int l, float f, int wave, int ln, Put put) {
  // block columns wave, wave + 8, .. of X, both block rows of each
  constexpr int EACH = (kSmallLong / 32 + kWaves - 1) / kWaves;
  const int row = here(ln) & 31, col = 4 * (here(ln) >> 5);
  f32x16 r[EACH][2];
#pragma unroll
  for (int b = 0; b < EACH; ++b) {
    const int j0 = (wave + b * kWaves) * 32;
    if (j0 >= l) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x16 one[1];
      lds_blocks<true>(P, X, i * 32, j0, kSmallSide, ln, one);
      r[b][i] = f * one[0];
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < EACH; ++b) {
    const int j0 = (wave + b * kWaves) * 32;
    if (j0 >= l) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {r[b][i][4 * q], r[b][i][4 * q + 1], r[b][i][4 * q + 2], r[b][i][4 * q + 3]};
        put(i * 32 + row, j0 + 8 * q + col, v);
      }
  }
}
// X X^T, a block for each of four waves: put(i, j, values j .. j + 3).
template <class Put>
__device__ __forceinline__ void lds_gram(const InLds& X, int l, int wave, int ln, Put put) {
  if (wave >= 4) return;
  const int i0 = wave / 2 * 32, j0 = wave % 2 * 32, row = here(ln) & 31, col = 4 * (here(ln) >> 5);
  f32x16 r[1];
  lds_blocks<false>(X, X, i0, j0, l, ln, r);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float v[4] = {r[0][4 * q], r[0][4 * q + 1], r[0][4 * q + 2], r[0][4 * q + 3]};
    put(i0 + row, j0 + 8 * q + col, v);
  }
}
// Four values of the result, (i, j) on, to where they belong.
template <typename TI>
__device__ __forceinline__ void put_result(const OrthArgs& a, const Shape& sh, TI* out, int i, int j, const float (&v)[4]) {
  const int s = sh.tall ? sh.n : sh.m, l = sh.tall ? sh.m : sh.n;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (i >= s || j + k >= l) continue;
    TI* o = out + sh.at(i, j + k);
    *o = (TI)(a.momentum ? a.keep * (float)*o - a.rate * v[k] : v[k]);
  }
}

// The whole of it for matrices of at most 64 x 384: X and the square matrices in LDS (8 of 64 x 128 fp32: 27 us, bound
// by LDS round trips between dependent products; in launches of their own these took 86). Few singular values:
// single steps (16 x 16: off by 0.8 in 1e-6, pairs 1.4), which cost nothing here where a side is short.
template <typename TI>
__global__ __launch_bounds__(kThreads) void small_kernel(OrthArgs a, double scale) {
  __shared__ __attribute__((aligned(1024))) char xs[2][kSmallSide * kSmallLong * 2];
  __shared__ __attribute__((aligned(1024))) char sq[2][2][kSmallSide * kSmallSide * 2];
  __shared__ double sums[kWaves];
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Shape sh(a);
  const int size = sh.m * sh.n, w = max(sh.m, sh.n), l = (w + 63) / 64 * 64;
  const int64_t at = (int64_t)blockIdx.x * size;
  const TI* g = static_cast<const TI*>(a.g) + at;
  TI* out = static_cast<TI*>(a.out) + at;
  float* mom = a.momentum ? a.momentum + at : nullptr;
  const InLds X{xs[0], xs[1], l * 2}, A{sq[0][0], sq[0][1], kSmallSide * 2}, P{sq[1][0], sq[1][1], kSmallSide * 2};

  double sum = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < size; i += kThreads) {
    float u = (float)g[i];
    if (mom) {
      const float v = momentum_of(a, mom[i], u);
      mom[i] = v;
      u = update_of(a, v, u);
    }
    sum += (double)u * (double)u;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (ln == 0) sums[wave] = sum;
  __syncthreads();  // (and the momentum is written, which other threads read below)
  sum = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) sum += sums[i];
  const Scale sc(sqrt(sum) + (double)a.eps, scale);
  lds_load(a, sh, g, mom, sc.by, 0, w, l, X);

  const float unit = (float)(1.0 / scale);
  for (int done = 0; done < a.steps;) {
    const bool begin = done == 0, two = min(sh.m, sh.n) > kFewValues && a.steps - done >= 2;
    const float t = begin ? sc.first : unit;  // X = t X^
    lds_gram(X, l, wave, ln, [&](int i, int j, const float(&v)[4]) {
      const float r[4] = {t * t * v[0], t * t * v[1], t * t * v[2], t * t * v[3]};
      A.put(i, j, r);
    });
    __syncthreads();
    lds_polynomial<kSmallSide>(a, two, A, P, wave, ln);
    done += two ? 2 : 1;
    if (done == a.steps)
      lds_times(P, X, l, t, wave, ln, [&](int i, int j, const float(&v)[4]) { put_result(a, sh, out, i, j, v); });
    else
      lds_times(P, X, l, begin ? t * (float)scale : 1.f, wave, ln,
                [&](int i, int j, const float(&v)[4]) { X.put(i, j, v); });
    __syncthreads();
  }
}

// Matrices of at most 64 x 12288: workgroup (c, e) has up to 384 columns of X in LDS. Between two launches of
// this kernel the Gram matrix's parts, one of every workgroup, are joined and P is computed.
// 8 of 40 x 1000: 49 us, 66 by the tiles above; 64 of 60 x 8000: 428, 657.
// FIRST: X from g (else X <- f P X from the one that the launch before left); LAST: X is the result
// (else it is left for the next launch, with its part of the Gram matrix).
struct ThinArgs {
  const double* partial;  // of the squares, `blocks` per matrix
  float* first;           // per matrix
  char* x;                // [E][columns / each][2][64 x 384], as in LDS
  const char* P;          // [E][2][64 x 64], as in LDS
  float* parts;           // [E][columns / each][64][64]
  double scale;
  int each;               // columns of a workgroup
  int blocks, power;
  float f;                // times first^power
};
constexpr int kThinLong = 32 * kSmallLong;
template <typename TI, bool FIRST, bool LAST>
__global__ __launch_bounds__(kThreads) void thin_kernel(OrthArgs a, ThinArgs t) {
  __shared__ __attribute__((aligned(1024))) char xs[2][kSmallSide * kSmallLong * 2];
  __shared__ __attribute__((aligned(1024))) char sq[2][kSmallSide * kSmallSide * 2];
  __shared__ double sums[kWaves];
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Shape sh(a);
  const int e = blockIdx.y, all = max(sh.m, sh.n), c0 = blockIdx.x * t.each, w = min(all - c0, t.each);
  const int l = (w + 63) / 64 * 64, bytes = kSmallSide * l * 2;
  const int64_t at = (int64_t)e * a.m * a.n, part = (int64_t)e * gridDim.x + blockIdx.x;
  const InLds X{xs[0], xs[1], l * 2}, P{sq[0], sq[1], kSmallSide * 2};
  char* image = t.x + part * (2 * kSmallSide * kSmallLong * 2);
  if constexpr (FIRST) {
    double v = (int)threadIdx.x < t.blocks ? t.partial[(int64_t)e * t.blocks + threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if (ln == 0) sums[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += sums[i];
    const Scale sc(sqrt(v) + (double)a.eps, t.scale);
    if (blockIdx.x == 0 && threadIdx.x == 0) t.first[e] = sc.first;
    lds_load(a, sh, static_cast<const TI*>(a.g) + at, a.momentum ? a.momentum + at : nullptr, sc.by, c0, w, l, X);
  } else {
    const char* from = t.P + (int64_t)e * (2 * kSmallSide * kSmallSide * 2);
#pragma unroll
    for (int i = threadIdx.x * 16; i < kSmallSide * kSmallSide * 2; i += kThreads * 16) {
      *reinterpret_cast<u32x4*>(P.hi + i) = ld16(from + i);
      *reinterpret_cast<u32x4*>(P.lo + i) = ld16(from + kSmallSide * kSmallSide * 2 + i);
    }
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16) {
      *reinterpret_cast<u32x4*>(X.hi + i) = ld16(image + i);
      *reinterpret_cast<u32x4*>(X.lo + i) = ld16(image + bytes + i);
    }
    __syncthreads();
    const float f = t.power ? t.f * t.first[e] : t.f;
    if constexpr (LAST) {
      TI* out = static_cast<TI*>(a.out) + at;
      lds_times(P, X, l, f, wave, ln, [&](int i, int j, const float(&v)[4]) { put_result(a, sh, out, i, c0 + j, v); });
    } else {
      lds_times(P, X, l, f, wave, ln, [&](int i, int j, const float(&v)[4]) { X.put(i, j, v); });
      __syncthreads();
    }
  }
  if constexpr (!LAST) {
    float* to = t.parts + part * (kSmallSide * kSmallSide);
    lds_gram(X, l, wave, ln, [&](int i, int j, const float(&v)[4]) {
      *reinterpret_cast<f32x4*>(to + i * kSmallSide + j) = f32x4{v[0], v[1], v[2], v[3]};
    });
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16) {
      st16(image + i, *reinterpret_cast<const u32x4*>(X.hi + i));
      st16(image + bytes + i, *reinterpret_cast<const u32x4*>(X.lo + i));
    }
  }
}
// The sum of the parts, in order, times f (times first^power), and what X is multiplied by.
__global__ __launch_bounds__(kThreads) void thin_polynomial_kernel(OrthArgs a, ThinArgs t, int parts, bool two, char* out) {
  __shared__ __attribute__((aligned(1024))) char sq[2][2][kSmallSide * kSmallSide * 2];
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const InLds A{sq[0][0], sq[0][1], kSmallSide * 2}, P{sq[1][0], sq[1][1], kSmallSide * 2};
  float f = t.f;
  for (int i = 0; i < t.power; ++i) f *= t.first[blockIdx.x];
  constexpr int N = kSmallSide * kSmallSide, EACH = N / 4 / kThreads, AHEAD = 8;
  const float* from = t.parts + (int64_t)blockIdx.x * parts * N + threadIdx.x * 4;
  f32x4 sum[EACH] = {};
  for (int i = 0; i < parts; i += AHEAD) {
    f32x4 v[AHEAD][EACH];
#pragma unroll
    for (int h = 0; h < AHEAD; ++h)
#pragma unroll
      for (int k = 0; k < EACH; ++k)
        v[h][k] = *reinterpret_cast<const f32x4*>(from + (int64_t)min(i + h, parts - 1) * N + k * kThreads * 4);
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) {
      if (i + h >= parts) continue;
#pragma unroll
      for (int k = 0; k < EACH; ++k) sum[k] += v[h][k];
    }
  }
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int i = threadIdx.x * 4 + k * kThreads * 4;
    const float v[4] = {f * sum[k][0], f * sum[k][1], f * sum[k][2], f * sum[k][3]};
    A.put(i / kSmallSide, i % kSmallSide, v);
  }
  __syncthreads();
  lds_polynomial<kSmallSide>(a, two, A, P, wave, ln);
  char* to = out + (int64_t)blockIdx.x * (2 * kSmallSide * kSmallSide * 2);
#pragma unroll
  for (int i = threadIdx.x * 16; i < kSmallSide * kSmallSide * 2; i += kThreads * 16) {
    st16(to + i, *reinterpret_cast<const u32x4*>(P.hi + i));
    st16(to + kSmallSide * kSmallSide * 2 + i, *reinterpret_cast<const u32x4*>(P.lo + i));
  }
}

// ---- short sides of 129 to 256 -----------------------------------------------------------
// Where launches are what counts, a step is two: the Gram matrix by the tiles above, and this one, which
// takes 32 rows of P and, without leaving LDS, their product with 128 columns of X (every workgroup of
// a row of them computes the same rows of P). X is kept with its long side along the rows, [long][256],
// wide matrices turned: then both products' right operands are rows, whose fragments only one wave
// uses. It loads them itself, those of A into registers and those of X into its own piece of LDS while
// it computes P; A, and X a second time, are kept as those fragments. 5 of 201 x 333 fp32: 12 us a launch,
// twelve launches in place of nineteen.
constexpr int kStrip = 256;      // the padded short side
constexpr int kStripRows = 32;   // of P, of a workgroup
constexpr int kStripLong = 128;  // of the long side, of a workgroup

// u 2^p in fp16 terms as scale_kernel leaves it, of the transposed matrix: 32 x 64 of it by way of LDS.
template <typename TI>
__global__ __launch_bounds__(256) void scale_turned_kernel(OrthArgs a, bool vec, const double* partial, int blocks,
                                                           double scale, f16* x, f16* frags, int64_t rows, int64_t plane,
                                                           float* first) {
  __shared__ double sh[4];
  __shared__ __attribute__((aligned(16))) f16 tile[2][64][40];
  const int e = blockIdx.y;
  const double sq = block_sum((int)threadIdx.x < blocks ? partial[(int64_t)e * blocks + threadIdx.x] : 0.0, sh);
  const Scale sc(sqrt(sq) + (double)a.eps, scale);
  if (blockIdx.x == 0 && threadIdx.x == 0) first[e] = sc.first;
  const int64_t r0 = (int64_t)(blockIdx.x % (kStrip / 32)) * 32, c0 = (int64_t)(blockIdx.x / (kStrip / 32)) * 64;
  const int64_t r = r0 + threadIdx.x / 8, c = c0 + threadIdx.x % 8 * 8, at = ((int64_t)e * a.m + r) * a.n + c;
  const int n = r < a.m ? (int)max(min((int64_t)8, a.n - c), (int64_t)0) : 0;
  float u[8] = {};
  if (n > 0) {
    load_row(static_cast<const TI*>(a.g) + at, n, vec, u);
    if (a.momentum) {
      float m[8];
      load_row(a.momentum + at, n, vec, m);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = update_of(a, m[k], u[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    f16 h, l;
    split((float)((double)u[k] * sc.by), h, l);
    tile[0][c - c0 + k][r - r0] = h;
    tile[1][c - c0 + k][r - r0] = l;
  }
  __syncthreads();
  const int64_t mat = (int64_t)e * rows * kStrip, i = c0 + threadIdx.x / 4, j = r0 + threadIdx.x % 4 * 8;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const f16x8 v = *reinterpret_cast<const f16x8*>(&tile[t][threadIdx.x / 4][threadIdx.x % 4 * 8]);
    *reinterpret_cast<f16x8*>(x + mat + in_panels(rows, i, j) + t * plane) = v;
    *reinterpret_cast<f16x8*>(frags + mat + in_fragments(rows, i, j) + t * plane) = v;
  }
}

struct StripArgs {
  const f16* A;  // [E][256 x 256], as fragments
  const f16* x;  // [E][rows x 256], as fragments
  f16 *to, *panels;  // the next X, as fragments and in panels
  const float* first;
  int64_t a_plane, x_plane;
  int rows, power;
  float f;  // times first^power
};

// A product with 32 rows in LDS, of N steps of 16 from k0 on: lane l has row l % 32 of those in LDS and
// columns 8 q + 4 (l / 32) + t, or, TURNED, a row of the other operand and those columns of LDS's rows.
// frag(term, k): the other operand's fragments.
template <bool TURNED, int N, class Frag>
__device__ __forceinline__ f32x16 strip_times(const InLds& m, int k0, int lane, Frag frag) {
  const int ln = here(lane);
  auto mfma = [](f16x8 lds, f16x8 reg, f32x16 to) {
    return TURNED ? __builtin_amdgcn_mfma_f32_32x32x16_f16(lds, reg, to, 0, 0, 0)
                  : __builtin_amdgcn_mfma_f32_32x32x16_f16(reg, lds, to, 0, 0, 0);
  };
  f32x16 sum{}, cross{}, acc{};
  f16x8 hi[2], lo[2];  // (of one step ahead)
  auto read = [&](int k) {
    hi[k % 2] = InLds::rows(m.hi, m, 0, k0 + 16 * k, ln);
    lo[k % 2] = InLds::rows(m.lo, m, 0, k0 + 16 * k, ln);
  };
  read(0);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const f16x8 h = frag(0, k), l = frag(1, k);
    if (k + 1 < N) read(k + 1);
    __builtin_amdgcn_sched_barrier(0);
    acc = mfma(hi[k % 2], h, acc);
    cross = mfma(lo[k % 2], h, cross);
    cross = mfma(hi[k % 2], l, cross);
    __builtin_amdgcn_sched_barrier(0);
    if (k % 4 == 3) {  // (sums of hi hi of 64 terms, as above)
      sum += acc;
      acc = f32x16{};
    }
  }
  return sum + kLo * cross;
}

template <typename TI, bool LAST>
__global__ __launch_bounds__(kThreads) void strip_kernel(OrthArgs a, StripArgs t) {
  constexpr int STRIPS = kStrip / kStripRows, STEPS = kStrip / 16, BLOCKS = kStripLong / 32;
  // rows of A, then of P; and each wave's part of X: 32 rows, half of the summed axis
  __shared__ __attribute__((aligned(1024))) char ps[2][kStripRows * kStrip * 2];
  __shared__ __attribute__((aligned(1024))) char xs[kWaves][2][STEPS / 2][1024];
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = ln >> 5;
  // the workgroups of the same rows of X are on one XCD
  const int chunks = t.rows / kStripLong, group = blockIdx.x / kXcds;
  const int chunk = group / STRIPS * kXcds + blockIdx.x % kXcds, e = chunk / chunks;
  if (e >= a.E) return;
  const int i0 = group % STRIPS * kStripRows, l0 = chunk % chunks * kStripLong + wave % BLOCKS * 32;
  const int k0 = wave / BLOCKS * (STEPS / 2);
  const InLds P{ps[0], ps[1], kStrip * 2};
  const f16* const mat = t.A + (int64_t)e * kStrip * kStrip;
  constexpr int EACH = kStripRows * kStrip / 8 / kThreads;
  auto place = [&](int n, int& r, int& c) {
    const int i = threadIdx.x + n * kThreads;
    r = i % kStripRows;
    c = i / kStripRows * 8;
  };
  u32x4 rows[2][EACH];
  int r, c;
#pragma unroll
  for (int n = 0; n < EACH; ++n) {
    place(n, r, c);
#pragma unroll
    for (int term = 0; term < 2; ++term) rows[term][n] = ld16(mat + term * t.a_plane + in_fragments(kStrip, i0 + r, c));
  }
  f16x8 own[2][STEPS];  // this wave's 32 columns of A (which is its own transpose)
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
#pragma unroll
    for (int term = 0; term < 2; ++term)
      own[term][k] = __builtin_bit_cast(f16x8, ld16(mat + term * t.a_plane + in_fragments(kStrip, wave * 32, 16 * k) + ln * 8));
  const f16* const x = t.x + (int64_t)e * t.rows * kStrip;
#pragma unroll
  for (int k = 0; k < STEPS / 2; ++k)
#pragma unroll
    for (int term = 0; term < 2; ++term)
      __builtin_amdgcn_global_load_lds(x + term * t.x_plane + in_fragments(t.rows, l0, 16 * (k0 + k)) + ln * 8,
                                       (lds_void*)xs[wave][term][k], 16, 0, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int n = 0; n < EACH; ++n) {
    place(n, r, c);
#pragma unroll
    for (int term = 0; term < 2; ++term) *reinterpret_cast<u32x4*>(ps[term] + P.at(r, c)) = rows[term][n];
  }
  __syncthreads();
  const f32x16 sq = strip_times<false, STEPS>(P, 0, ln, [&](int term, int k) { return own[term][k]; });
  __syncthreads();  // (everyone has read A)
  r = ln & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    c = wave * 32 + 8 * q + 4 * half;
    f16x4* const at[2] = {reinterpret_cast<f16x4*>(P.hi + P.at(r, c)), reinterpret_cast<f16x4*>(P.lo + P.at(r, c))};
    const f16x4 h = *at[0], l = *at[1];
    f16x4 ph, pl;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float old = (float)h[k] + kLo * (float)l[k];
      f16 v0, v1;
      split(a.c * sq[4 * q + k] + a.b * old + (i0 + r == c + k ? a.a : 0.f), v0, v1);
      ph[k] = v0;
      pl[k] = v1;
    }
    *at[0] = ph;
    *at[1] = pl;
  }
  wait_vmcnt<0>();  // X
  __syncthreads();
  const bool tall = a.m > a.n, turned = !LAST || tall;
  auto times = [&](auto flag) {
    return strip_times<decltype(flag)::value, STEPS / 2>(P, 16 * k0, ln, [&](int term, int k) {
      return *reinterpret_cast<const f16x8*>(xs[wave][term][k] + ln * 16);
    });
  };
  f32x16 v = turned ? times(std::true_type{}) : times(std::false_type{});
  // Two waves have half of each sum: each takes half of the values.
  const bool upper = wave >= BLOCKS;
  {
    f32x4* const to = reinterpret_cast<f32x4*>(xs[wave][0][0]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = upper ? v[4 * q + k] : v[4 * (q + 2) + k];
      to[q * 64 + ln] = w;
    }
    __syncthreads();
    const f32x4* const from = reinterpret_cast<const f32x4*>(xs[wave ^ BLOCKS][0][0]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4 w = from[q * 64 + ln];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * q + k] = (upper ? v[4 * (q + 2) + k] : v[4 * q + k]) + w[k];
    }
  }
  float by = t.f;
  for (int i = 0; i < t.power; ++i) by *= t.first[e];
  const int j0 = (upper ? 16 : 0) + 4 * half;  // of value 0; value 4 q + k is 8 q + k behind it
  if constexpr (!LAST) {
    const int64_t at = (int64_t)e * t.rows * kStrip;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f16x4 h, l;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f16 v0, v1;
        split(by * v[4 * q + k], v0, v1);
        h[k] = v0;
        l[k] = v1;
      }
      const int64_t row = l0 + (ln & 31), col = i0 + j0 + 8 * q;
      f16 *to = t.to + at + in_fragments(t.rows, row, col), *panel = t.panels + at + in_panels(t.rows, row, col);
      *reinterpret_cast<f16x4*>(to) = h;
      *reinterpret_cast<f16x4*>(panel) = h;
      *reinterpret_cast<f16x4*>(to + t.x_plane) = l;
      *reinterpret_cast<f16x4*>(panel + t.x_plane) = l;
    }
  } else {
    const int row = (tall ? l0 : i0) + (ln & 31), col = (tall ? i0 : l0) + j0;
    if (row >= a.m) return;
    TI* out = static_cast<TI*>(a.out) + ((int64_t)e * a.m + row) * a.n + col;
    float w[2][4] = {};
    if (a.momentum) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (col + 8 * q + k < a.n) w[q][k] = (float)out[8 * q + k];
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float u = by * v[4 * q + k];
        if (col + 8 * q + k < a.n) out[8 * q + k] = (TI)(a.momentum ? a.keep * w[q][k] - a.rate * u : u);
      }
  }
}

// ---- host ------------------------------------------------------------------------------
int64_t padded(int64_t n) { return (n + kPad - 1) / kPad * kPad; }
size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

int64_t tiles_of(const ProductArgs& a, int bm, bool sym) {
  const int64_t mt = (a.rows + bm - 1) / bm, nt = (a.cols + bm - 1) / bm;
  return a.E * (sym ? mt * (mt + 1) / 2 : mt * nt);
}

// How a product is laid over the chip: parts of a tile and tiles of an XCD (ProductArgs), and
// about how long it takes, in ns.
struct Plan {
  int parts, rest;
  double ns;
};
// Parts where tiles do not fill the chip once, as many as do, of two ring turns at least.
template <class G>
Plan plan_for(const ProductArgs& a, bool sym) {
  // ns of a tile's stage of 32, where a CU has few tiles and (the clock and the L2s' share gone down)
  // many; of a tile's end, of a launch, and of a join. Fitted to kernel traces (us so, and measured: 256 rows: 8 of 4096 squared
  // 571, 541, times 4096 x 14336 3188, 3107; 128 rows in one term: 8 of 1024 squared 20.4, 21.6, 4 of 512 8.8, 10.2;
  // in two: 2048 squared times itself 50.8, 58.6, 64 of 2048 x 640 by 640 383, 360; 64 rows: 8 of 1024 squared 42.4, 42.8,
  // 4 of 512 7.2, 8.5, 2 of 384 over 8064 in ten parts with the join 19, 24.6); they choose, no result depends on them.
  struct Cost {
    double stage, busy, tile, launch, join;
    int few;
  };
  constexpr Cost c = G::BM == 256    ? Cost{750, 850, 5000, 2000, 0, 1}
                     : G::TERMS == 1 ? Cost{240, 340, 0, 5000, 7000, 8}
                     : G::BM == 128  ? Cost{700, 800, 3000, 3000, 0, 1}
                                     : Cost{200, 240, 0, 4000, 5000, 4};
  constexpr int cus = kCus / kXcds;
  const int64_t tiles = tiles_of(a, G::BM, sym), each = (tiles + kXcds - 1) / kXcds, turns = a.K / (kStages * G::BK);
  const int64_t per_cu = (each + cus - 1) / cus;
  const double sum = (double)(a.K / G::BK) * (per_cu > c.few ? c.busy : c.stage) + c.tile;
  Plan p{1, (int)each, c.launch + sum * (double)per_cu};
  if (c.join == 0 || each > G::SLOTS / 2) return p;
  int parts = G::SLOTS / (int)each;
  if (parts > turns / 2) parts = (int)(turns / 2);
  if (parts > kMaxParts) parts = kMaxParts;
  const double ns = c.launch + sum / parts * (double)((each * parts + cus - 1) / cus) + c.join;
  if (parts > 1 && ns < p.ns) p = Plan{parts, (int)each, ns};
  return p;
}

template <class G, bool SYM, int KIND, typename TO>
hipError_t launch_tile(const ProductArgs& args, hipStream_t s) {
  ProductArgs a = args;
  const Plan p = plan_for<G>(a, SYM);
  a.parts = p.parts;
  a.rest = p.rest;
  const int items = a.rest * a.parts;
  product_kernel<G, SYM, KIND, TO><<<(unsigned)((items < G::SLOTS ? items : G::SLOTS) * kXcds), 256, 0, s>>>(a);
  if (a.parts > 1)
    join_kernel<G, SYM, KIND, TO><<<(unsigned)(a.rest * kXcds * 4 * Passes<G>::ALL), 64, 0, s>>>(a);
  return hipGetLastError();
}
// The larger of the two tiles there are for one or two terms, or the smaller one.
template <bool AKS, bool BKS, int TERMS>
using Big = Tile<TERMS == 1 ? 256 : 128, AKS, BKS, TERMS>;
template <bool AKS, bool BKS, int TERMS>
using Small = Tile<TERMS == 1 ? 128 : 64, AKS, BKS, TERMS>;
template <int TERMS>
bool big(const ProductArgs& a, bool sym) {
  return plan_for<Big<false, false, TERMS>>(a, sym).ns < plan_for<Small<false, false, TERMS>>(a, sym).ns;
}
template <bool AKS, bool BKS, bool SYM, int TERMS, int KIND, typename TO>
hipError_t product(const ProductArgs& a, hipStream_t s) {
  if (big<TERMS>(a, SYM)) return launch_tile<Big<AKS, BKS, TERMS>, SYM, KIND, TO>(a, s);
  return launch_tile<Small<AKS, BKS, TERMS>, SYM, KIND, TO>(a, s);
}
// Bytes of its parts' sums.
template <int TERMS>
size_t sum_bytes(int E, int64_t K, int64_t rows, int64_t cols, bool sym) {
  typedef Small<false, false, TERMS> G;  // (the larger tiles have no parts)
  ProductArgs a{};
  a.E = E;
  a.K = K;
  a.rows = rows;
  a.cols = cols;
  const Plan p = plan_for<G>(a, sym);
  return big<TERMS>(a, sym) || p.parts == 1 ? 0 : (size_t)kXcds * p.rest * p.parts * G::BM * G::BM * sizeof(float);
}

// Matrices of one launch, and of workgroups that keep 384 columns.
int64_t long_side(const OrthArgs& a) { return a.m > a.n ? a.m : a.n; }
bool is_small(const OrthArgs& a) { return (a.m <= kSmallSide || a.n <= kSmallSide) && long_side(a) <= kSmallLong; }
bool is_thin(const OrthArgs& a) {
  return (a.m <= kSmallSide || a.n <= kSmallSide) && !is_small(a) && long_side(a) <= kThinLong;
}
// Columns of a workgroup: 128 or 256, so that it has soon done, where a matrix then has no more than 24
// parts of its Gram matrix and all workgroups are on the chip at once; else 384 (at most 32 parts, of 12288
// columns, and as many rounds of workgroups as there are).
int thin_columns(const OrthArgs& a) {
  for (int w = 128; w < kSmallLong; w += 128)
    if (long_side(a) <= 24 * w && a.E * ((long_side(a) + w - 1) / w) <= kCus) return w;
  return kSmallLong;
}
int64_t thin_groups(const OrthArgs& a) { return (long_side(a) + thin_columns(a) - 1) / thin_columns(a); }

// Matrices whose steps are two launches each: those whose workgroups are at most half of what the chip holds, in two
// terms whatever their type (us, by the tiles above and so: 5 of 201 x 333 fp32 113, 98; 2 of 200 x 1000 bf16 129 in one
// term, 109; past it 16 of 256 x 256 fp32 105, 118). What they read of L2, 384 KB of each workgroup, is the time
// then. (One term would be 92 for 109, but every step is a single one and rounds X: off by up to 3.7% of the norm at
// ranks of 1 to 64, where tiles, with pairs, are off by 1.2%.) Up to twice as many workgroups bf16 matrices are kept in
// two terms as well: their smaller tiles fill more of the chip (us by tiles, one term and two: 8 of 440 x 168 122, 104; 2 of
// 1500 x 200 133, 117; 1 of 200 x 4096 145, 131; past it 32 of 130 x 256 117, 139; 40 of 160 x 800 164, 214).
int64_t strip_groups(const OrthArgs& a) {
  return (int64_t)a.E * (kStrip / kStripRows) * (padded(long_side(a)) / kStripLong);
}
bool are_few(const OrthArgs& a) { return padded(a.m < a.n ? a.m : a.n) == kStrip && strip_groups(a) <= kCus; }
bool is_strip(const OrthArgs& a) { return are_few(a) && strip_groups(a) * 2 <= kCus; }

// Whether `steps` steps bear the roundings of one term: what a step is off by is multiplied in every later one by
// |p'| at most, p(s) = a s + b s^3 + c s^5, whose largest magnitude over the singular values there are is mostly a's, at
// 0 (the default coefficients' 3.44, which makes that 198 for five steps and 683 for six; off by up to 1.5% and 4.4%
// of the norm at ranks of 1 to 128, eight steps up to 51%). Singular values well past 1 are left to two terms.
bool one_term_bears(const OrthArgs& a) {
  double growth = 0, most = 0;
  for (int i = 0; i <= 64; ++i) {
    const double s = i / 64.0, t = s * s, d = fabs(a.a + t * (3.0 * a.b + t * 5.0 * a.c)), v = fabs(s * (a.a + t * (a.b + t * a.c)));
    growth = growth > d ? growth : d;
    most = most > v ? most : v;
  }
  double sum = 0;
  for (int i = 0; i < a.steps && sum <= kMostGrowth; ++i) sum = sum * growth + 1;
  return most <= kMostValue && sum <= kMostGrowth;
}
int terms_of(const OrthArgs& a) {
  return a.bf16 && (a.m < a.n ? a.m : a.n) > kOneTerm && !are_few(a) && one_term_bears(a) ? 1 : 2;
}

// Whether the next two steps share a Gram matrix. In one term what was rounded in A is multiplied by
// up to a^4 on the way to A', which costs most in the middle steps, where singular values of every size
// are left: there single steps, unless the long side is twice the short one and pairs save a
// fifth; then one single step between two pairs (off by, in 64-bit simulations of five steps with these
// roundings, of gradients 512 x 2048 in 1e-3: pairs first 3.1, one between 0.9, all single 1.1; 512 x 512:
// 2.4, 2.0, 1.3, and 1.0 with only the first two as a pair).
bool pair_next(const OrthArgs& a, int terms, int done) {
  const int left = a.steps - done;
  const int64_t s = a.m < a.n ? a.m : a.n, l = a.m < a.n ? a.n : a.m;
  if (terms == 2) return pair_in_two_terms(s, left);
  if (left < 2 || done == 0) return left >= 2;
  return l >= 2 * s && left % 2 == 0;
}

// Pieces of the workspace.
struct Layout {
  int64_t rows, cols, side;  // padded
  int blocks;                // partial sums per matrix
  size_t partial, first, sums, x[3], sq[3], bytes;
};
Layout layout_of(const OrthArgs& a) {
  Layout l{};  // (pieces that a path does not have: at 0, which nothing looks at)
  const int terms = terms_of(a);
  l.rows = padded(a.m);
  l.cols = padded(a.n);
  l.side = l.rows < l.cols ? l.rows : l.cols;
  const int64_t blocks = (a.m * a.n + 4095) / 4096;
  l.blocks = (int)(blocks < kNormBlocks ? blocks : kNormBlocks);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += aligned(n);
    return p;
  };
  if (is_small(a)) {  // (everything is in LDS)
    l.bytes = 256;
    return l;
  }
  l.partial = take((size_t)a.E * l.blocks * sizeof(double));
  l.first = take((size_t)a.E * sizeof(float));
  if (is_thin(a)) {
    const size_t groups = (size_t)a.E * (size_t)thin_groups(a);
    l.sums = take(groups * kSmallSide * kSmallSide * sizeof(float));
    l.x[0] = take(groups * kSmallSide * kSmallLong * 4);
    l.sq[0] = take((size_t)a.E * kSmallSide * kSmallSide * 4);
    l.bytes = at;
    return l;
  }
  const int64_t longer = l.rows < l.cols ? l.cols : l.rows;
  size_t sums = 0;
  auto product = [&](int64_t K, int64_t rows, int64_t cols, bool sym) {
    const size_t n = terms == 1 ? sum_bytes<1>(a.E, K, rows, cols, sym) : sum_bytes<2>(a.E, K, rows, cols, sym);
    if (n > sums) sums = n;
  };
  product(longer, l.side, l.side, true);
  const bool strip = is_strip(a);
  if (strip) {
    l.rows = longer;
    l.cols = l.side;
  } else {
    product(l.side, l.side, l.side, true);
    product(l.side, l.rows, l.cols, false);
  }
  l.sums = take(sums);
  const size_t x = (size_t)a.E * l.rows * l.cols * terms * 2, sq = (size_t)a.E * l.side * l.side * terms * 2;
  // (strips: X in panels, and as fragments before and after a step)
  for (int i = 0; i < 3; ++i) l.x[i] = i == 0 || (strip ? i == 1 || a.steps > 1 : i == 1 && a.steps > 2) ? take(x) : 0;
  for (int i = 0; i < 3; ++i) l.sq[i] = i == 0 || (!strip && (i == 1 || a.steps > 1)) ? take(sq) : 0;
  l.bytes = at;
  return l;
}

template <typename TI>
hipError_t run_thin(const OrthArgs& a, const Layout& l, double scale, hipStream_t s) {
  ThinArgs t{};
  t.partial = reinterpret_cast<const double*>(a.ws + l.partial);
  t.first = reinterpret_cast<float*>(a.ws + l.first);
  t.x = a.ws + l.x[0];
  t.P = a.ws + l.sq[0];
  t.parts = reinterpret_cast<float*>(a.ws + l.sums);
  t.scale = scale;
  t.blocks = l.blocks;
  const dim3 grid((unsigned)thin_groups(a), a.E);
  t.each = thin_columns(a);
  const float unit = (float)(1.0 / scale);
  thin_kernel<TI, true, false><<<grid, kThreads, 0, s>>>(a, t);
  for (int done = 0; done < a.steps;) {
    const bool begin = done == 0, two = pair_in_two_terms(a.m < a.n ? a.m : a.n, a.steps - done);
    t.power = begin ? 2 : 0;
    t.f = begin ? 1.f : unit * unit;
    thin_polynomial_kernel<<<a.E, kThreads, 0, s>>>(a, t, (int)grid.x, two, a.ws + l.sq[0]);
    done += two ? 2 : 1;
    t.power = begin ? 1 : 0;
    if (done == a.steps) {
      t.f = begin ? 1.f : unit;
      thin_kernel<TI, false, true><<<grid, kThreads, 0, s>>>(a, t);
    } else {
      t.f = begin ? (float)scale : 1.f;
      thin_kernel<TI, false, false><<<grid, kThreads, 0, s>>>(a, t);
    }
  }
  return hipGetLastError();
}

template <typename TI>
hipError_t run_strip(const OrthArgs& a, const Layout& l, double scale, bool aligned_in, hipStream_t s) {
  const double* partial = reinterpret_cast<const double*>(a.ws + l.partial);
  float* first = reinterpret_cast<float*>(a.ws + l.first);
  const int64_t x_plane = a.E * l.rows * l.cols, a_plane = (int64_t)a.E * kStrip * kStrip;
  f16* panels = reinterpret_cast<f16*>(a.ws + l.x[0]);
  f16* x[2] = {reinterpret_cast<f16*>(a.ws + l.x[1]), reinterpret_cast<f16*>(a.ws + l.x[2])};
  f16* A = reinterpret_cast<f16*>(a.ws + l.sq[0]);
  const bool vec = aligned_in && a.n % 8 == 0;
  if (a.m > a.n)
    scale_kernel<TI, 2><<<dim3((unsigned)(l.rows * l.cols / 8 / 256), a.E), 256, 0, s>>>(
        a, vec, partial, l.blocks, scale, panels, x[0], l.rows, l.cols, x_plane, first);
  else
    scale_turned_kernel<TI><<<dim3((unsigned)(kStrip / 32 * (l.rows / 64)), a.E), 256, 0, s>>>(
        a, vec, partial, l.blocks, scale, panels, x[0], l.rows, x_plane, first);
  hipError_t e = hipGetLastError();
  const float unit = (float)(1.0 / scale);
  const int64_t chunks = strip_groups(a) / (kStrip / kStripRows);
  const unsigned grid = (unsigned)((chunks + kXcds - 1) / kXcds * kXcds * (kStrip / kStripRows));
  for (int done = 0; done < a.steps && e == hipSuccess; ++done) {
    const bool begin = done == 0;
    ProductArgs r{};
    r.a = r.b = Operands{panels, x_plane, l.rows * l.cols, (int)l.rows};
    r.K = l.rows;
    r.rows = r.cols = kStrip;
    r.E = a.E;
    r.sums = reinterpret_cast<float*>(a.ws + l.sums);
    r.d = A;
    r.d_plane = a_plane;
    r.first = first;
    r.power = begin ? 2 : 0;
    r.f = begin ? 1.f : unit * unit;
    e = product<true, true, true, 2, kFragments, f16>(r, s);
    if (e != hipSuccess) return e;
    const bool last = done + 1 == a.steps;
    StripArgs t{};
    t.A = A;
    t.x = x[done & 1];
    t.to = x[(done + 1) & 1];
    t.panels = panels;
    t.first = first;
    t.a_plane = a_plane;
    t.x_plane = x_plane;
    t.rows = (int)l.rows;
    t.power = begin ? 1 : 0;
    t.f = last ? (begin ? 1.f : unit) : begin ? (float)scale : 1.f;
    if (last) strip_kernel<TI, true><<<grid, kThreads, 0, s>>>(a, t);
    else strip_kernel<TI, false><<<grid, kThreads, 0, s>>>(a, t);
    e = hipGetLastError();
  }
  return e;
}

template <typename TI, int TERMS>
hipError_t run(const OrthArgs& a, hipStream_t s) {
  const Layout l = layout_of(a);
  double* partial = reinterpret_cast<double*>(a.ws + l.partial);
  float* first = reinterpret_cast<float*>(a.ws + l.first);
  float* sums = reinterpret_cast<float*>(a.ws + l.sums);
  const bool tall = a.m > a.n;
  auto aligned16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool aligned_in = aligned16(a.g) && aligned16(a.momentum);
  const int64_t x_plane = a.E * l.rows * l.cols, sq_plane = a.E * l.side * l.side;
  f16* x[2] = {reinterpret_cast<f16*>(a.ws + l.x[0]), reinterpret_cast<f16*>(a.ws + l.x[1])};
  f16* sq[3] = {reinterpret_cast<f16*>(a.ws + l.sq[0]), reinterpret_cast<f16*>(a.ws + l.sq[1]),
                reinterpret_cast<f16*>(a.ws + l.sq[2])};
  // 2^k near the square root of the long side: X's values are of order 1 / sqrt(long side) at the end
  double scale = 1;
  while (scale * scale < (double)(a.m > a.n ? a.m : a.n)) scale *= 2;
  if (is_small(a)) {
    small_kernel<TI><<<a.E, kThreads, 0, s>>>(a, scale);
    return hipGetLastError();
  }

  square_kernel<TI><<<dim3(l.blocks, a.E), 256, 0, s>>>(a, aligned_in && a.m * a.n % 8 == 0, partial);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if constexpr (TERMS == 2) {
    if (is_thin(a)) return run_thin<TI>(a, l, scale, s);
    if (is_strip(a)) return run_strip<TI>(a, l, scale, aligned_in, s);
  }
  const int64_t chunks = (l.rows * l.cols / 8 + 255) / 256, most = (4096 + a.E - 1) / a.E;
  scale_kernel<TI, TERMS><<<dim3((unsigned)(chunks < most ? chunks : most), a.E), 256, 0, s>>>(
      a, aligned_in && a.n % 8 == 0, partial, l.blocks, scale, x[0], nullptr, l.rows, l.cols, x_plane, first);
  e = hipGetLastError();
  if (e != hipSuccess) return e;

  auto big = [&](const f16* p) { return Operands{p, x_plane, l.rows * l.cols, (int)l.rows}; };
  auto square = [&](const f16* p) { return Operands{p, sq_plane, l.side * l.side, (int)l.side}; };
  // of symmetric matrices that commute: d = u v, or a I + b u + c u^2
  auto symmetric = [&](const f16* u, const f16* v, f16* d) {
    ProductArgs r{};
    r.a = r.c = square(u);
    r.b = square(v ? v : u);
    r.K = r.rows = r.cols = l.side;
    r.E = a.E;
    r.sums = sums;
    r.d = d;
    r.d_plane = sq_plane;
    r.f = v ? 1.f : a.c;
    r.p = a.b;
    r.q = a.a;
    return v ? product<false, false, true, TERMS, kProduct, f16>(r, s)
             : product<false, false, true, TERMS, kPolynomial, f16>(r, s);
  };
  f16 *A = sq[0], *P = sq[1], *Y = sq[2];
  for (int done = 0, at = 0; done < a.steps; at ^= 1) {
    const bool begin = done == 0, two = pair_next(a, TERMS, done);
    const float unit = (float)(1.0 / scale);  // X = unit X^ (the first X^: first[e] X^)
    ProductArgs r{};
    r.a = r.b = big(x[at]);
    r.K = tall ? l.rows : l.cols;
    r.rows = r.cols = l.side;
    r.E = a.E;
    r.sums = sums;
    r.d = A;
    r.d_plane = sq_plane;
    r.first = first;
    r.power = begin ? 2 : 0;
    r.f = begin ? 1.f : unit * unit;
    e = tall ? product<true, true, true, TERMS, kProduct, f16>(r, s) : product<false, false, true, TERMS, kProduct, f16>(r, s);
    const f16* Q = P;
    if (l.side == kPad && TERMS == 2) {
      if (e != hipSuccess) return e;
      polynomial_kernel<<<a.E, kThreads, 0, s>>>(a, two, A, P, sq_plane);
      e = hipGetLastError();
    } else if (e == hipSuccess) {
      e = symmetric(A, nullptr, P);
    }
    if (two && !(l.side == kPad && TERMS == 2)) {
      if (e == hipSuccess) e = symmetric(P, A, Y);
      if (e == hipSuccess) e = symmetric(P, Y, A);        // A'
      if (e == hipSuccess) e = symmetric(A, nullptr, Y);  // P'
      if (e == hipSuccess) e = symmetric(Y, P, A);
      Q = A;
    }
    if (e != hipSuccess) return e;
    done += two ? 2 : 1;
    const bool last = done == a.steps;
    ProductArgs g{};
    g.a = tall ? big(x[at]) : square(Q);
    g.b = tall ? square(Q) : big(x[at]);
    g.K = l.side;
    g.rows = l.rows;
    g.cols = l.cols;
    g.E = a.E;
    g.sums = sums;
    g.first = first;
    g.power = begin ? 1 : 0;
    if (last) {
      g.f = begin ? 1.f : unit;
      g.out = a.out;
      g.m = a.m;
      g.n = a.n;
      g.vec = aligned16(a.out) && a.n % 8 == 0;
      g.keep = a.keep;
      g.rate = a.rate;
      if (a.momentum)
        e = tall ? product<false, false, false, TERMS, kUpdate, TI>(g, s)
                 : product<false, true, false, TERMS, kUpdate, TI>(g, s);
      else
        e = tall ? product<false, false, false, TERMS, kLast, TI>(g, s)
                 : product<false, true, false, TERMS, kLast, TI>(g, s);
    } else {
      g.f = begin ? (float)scale : 1.f;
      g.d = x[at ^ 1];
      g.d_plane = x_plane;
      e = tall ? product<false, false, false, TERMS, kProduct, f16>(g, s) : product<false, true, false, TERMS, kProduct, f16>(g, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t orthogonalize_workspace(const OrthArgs& a) { return layout_of(a).bytes; }

hipError_t launch_orthogonalize(const OrthArgs& a, hipStream_t s) {
  if (terms_of(a) == 1) return run<bf16, 1>(a, s);
  return a.bf16 ? run<bf16, 2>(a, s) : run<float, 2>(a, s);
}

// Products of rows grouped by expert, with ragged group sizes: NN (a b_e), NT (a b_e^T) and
// TN (the group's a^T b), fp32 sums.
//
// bf16: one workgroup of four waves per BM x BN tile of the output, v_mfma_f32_32x32x16_bf16.
// The summed axis advances in stages of BK through a ring of four LDS buffers filled by
// direct global -> LDS loads. An operand is either K-contiguous in memory (a of NN and NT,
// b of NT), and its fragments are 16-byte LDS reads, or K-strided (b of NN, both of TN), and
// its fragments come out of LDS with transposing reads: no operand is transposed in memory.
// Stages are software-pipelined: while the MFMAs of one stage run from registers, the
// fragments of the next are read from LDS and the stage just consumed is refilled.
// What is out of range is never loaded: addresses are clamped to the last row, column or
// chunk, and the values of the summed axis past its end are zeroed in both operands'
// fragments (the last stage only), so that a non-finite value there reaches no sum.
#include "train_common.h"
#include "train_kernels.h"

#include "moe.h"

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kStages = 4;    // LDS ring
constexpr int kTable = 2048;  // TN: rows of the summed axis whose indices are in LDS at once

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkmcnt0() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
}
// s_waitcnt vmcnt(n * PER) for a runtime n, 3 or more taken for 3
template <int PER>
__device__ __forceinline__ void wait_stages(int n) {
  if (n >= 3) wait_vmcnt<3 * PER>();
  else if (n == 2) wait_vmcnt<2 * PER>();
  else if (n == 1) wait_vmcnt<PER>();
  else wait_vmcnt<0>();
}
__device__ __forceinline__ void sync_point() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// One operand's stage in LDS: X rows (its output axis) by BK of the summed axis.
//   K-contiguous (KS false): [X][BK], 16-byte chunk c of a row stored at c ^ swz(row).
//   K-strided (KS true): [BK][X], 16-byte slot s of a row stored at s ^ swz(row).
// Both swizzles make the fragment reads free of bank conflicts. A direct load instruction
// moves 64 lanes x 16 bytes into 1 KB of LDS, lane l into slot l.
template <bool KS_, int X_, int BK_, int NW>
struct Operand {
  static constexpr bool KS = KS_;
  static constexpr int X = X_, BK = BK_;
  static constexpr int BYTES = X * BK * 2;
  static constexpr int PW = BYTES / 1024 / NW;         // loads per wave and stage
  static constexpr int ROW = KS ? X * 2 : BK * 2;      // bytes per LDS row
  static constexpr int SLOTS = ROW / 16;               // chunks per LDS row
  static constexpr int RPI = 1024 / ROW;               // LDS rows per load instruction
  static_assert(PW >= 1 && BYTES % (1024 * NW) == 0, "whole loads per wave");
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (KS) return ((0xCA60 >> (4 * (row & 3))) & 15) % SLOTS;
    else if constexpr (SLOTS == 4) return ((row >> 1) ^ (row >> 3)) & 3;
    else return (row ^ (row >> 3)) & 7;
  }
  // LDS row of load j of a wave for this lane, and the source chunk that goes into its slot
  static __device__ __forceinline__ int row(int j, int wave, int ln) {
    return (wave * PW + j) * RPI + ln / SLOTS;
  }
  static __device__ __forceinline__ int chunk(int j, int wave, int ln) {
    return (ln % SLOTS) ^ swz(row(j, wave, ln));
  }
  // byte offset of this lane's fragment of the 32 rows from x0 (substep 0)
  static __device__ __forceinline__ int frag(int x0, int ln) {
    if constexpr (KS) {
      const int g = ln >> 4, r = (ln & 15) >> 2, c = ln & 3;
      const int n = x0 + (g & 1) * 16 + 4 * c, k = (g >> 1) * 8 + r;
      return k * ROW + ((n >> 3) ^ swz(k)) * 16 + ((n >> 2) & 1) * 8;
    } else {
      const int m = x0 + (ln & 31);
      return m * ROW + ((ln >> 5) ^ swz(m)) * 16;
    }
  }
  // the fragment of substep s (k = 16 s + 8 (lane / 32) .. + 7)
  static __device__ __forceinline__ s16x8 read(const char* st, int at, int s) {
    if constexpr (KS) {
      const char* p = st + at + 16 * s * ROW;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ROW));
      return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    } else {
      return *reinterpret_cast<const s16x8*>(st + (at ^ (32 * s)));
    }
  }
};

// BM x BN tile, WGM x (4 / WGM) waves.
template <int FORM_, int BM_, int BN_, int BK_, int WGM>
struct Geo {
  static constexpr int FORM = FORM_, BM = BM_, BN = BN_, BK = BK_;
  static constexpr bool TN = FORM == MOE_MATMUL_TN;
  static constexpr int WGN = 4 / WGM, SUB = BK / 16;
  typedef Operand<TN, BM, BK, 4> A;
  typedef Operand<FORM != MOE_MATMUL_NT, BN, BK, 4> B;
  static constexpr int WM = BM / WGM, WN = BN / WGN, MB = WM / 32, NB = WN / 32;
  static constexpr int STAGE = A::BYTES + B::BYTES, LPS = A::PW + B::PW;
};

// Sources of a tile's direct loads. NN, NT: one pointer per load, advancing by a fixed step
// per stage. TN: the rows are the summed axis, so each load takes its row's index from a
// table in LDS (the gather, or the rows themselves; past the end the last row again).
template <class G>
struct Loader {
  const bf16* pa[G::A::PW];
  const bf16* pb[G::B::PW];
  size_t step_a, step_b;  // elements per stage (TN: per row)
  const int *ta, *tb;     // TN tables, this segment's first row at 0
  int len, wave, ln;

  template <class Op>
  __device__ __forceinline__ const bf16* at(const bf16* const* p, size_t step, const int* tab, int j,
                                            int kt) const {
    if constexpr (G::TN) return p[j] + (size_t)tab[kt * G::BK + Op::row(j, wave, ln)] * step;
    else return p[j] + (size_t)kt * step;
  }
  // NN, NT, a stage that ends past len: the last chunk (or row) again
  template <class Op>
  __device__ __forceinline__ const bf16* at_tail(const bf16* const* p, size_t step, int j, int kt) const {
    const int k = kt * G::BK + (Op::KS ? Op::row(j, wave, ln) : Op::chunk(j, wave, ln) * 8);
    const int back = min(0, len - (Op::KS ? 1 : 8) - k);
    return p[j] + (size_t)kt * step + (Op::KS ? (int64_t)back * (int64_t)(step / G::BK) : (int64_t)back);
  }
  // load j (A's, then B's; a constant at every call) of stage kt into st
  template <bool TAIL>
  __device__ __forceinline__ void issue(int j, int kt, char* st) const {
    if (j < G::A::PW) {
      const bf16* p = TAIL ? at_tail<typename G::A>(pa, step_a, j, kt)
                           : at<typename G::A>(pa, step_a, ta, j, kt);
      __builtin_amdgcn_global_load_lds(p, (lds_void*)(st + (wave * G::A::PW + j) * 1024), 16, 0, 0);
    } else {
      const int i = j - G::A::PW;
      const bf16* p = TAIL ? at_tail<typename G::B>(pb, step_b, i, kt)
                           : at<typename G::B>(pb, step_b, tb, i, kt);
      __builtin_amdgcn_global_load_lds(
          p, (lds_void*)(st + G::A::BYTES + (wave * G::B::PW + i) * 1024), 16, 0, 0);
    }
  }
  __device__ __forceinline__ void issue_stage(int kt, char* st) const {
    if (G::TN || (kt + 1) * G::BK <= len) {
#pragma unroll
      for (int j = 0; j < G::LPS; ++j) issue<false>(j, kt, st);
    } else {
#pragma unroll
      for (int j = 0; j < G::LPS; ++j) issue<true>(j, kt, st);
    }
  }
};

template <class G>
struct Frags {
  s16x8 a[G::SUB][G::MB], b[G::SUB][G::NB];
};

template <class G>
struct Wave {
  int a_at[G::MB], b_at[G::NB];
  f32x16 acc[G::NB][G::MB];

  // LDS read r of a stage's fragments (r constant at every call)
  __device__ __forceinline__ void read(int r, const char* st, Frags<G>& F) const {
    const int s = r / (G::MB + G::NB), i = r % (G::MB + G::NB);
    if (i < G::MB) F.a[s][i] = G::A::read(st, a_at[i], s);
    else F.b[s][i - G::MB] = G::B::read(st + G::A::BYTES, b_at[i - G::MB], s);
  }
  __device__ __forceinline__ void mfma(int i, const Frags<G>& F) {
    const int s = i / (G::NB * G::MB), nb = i / G::MB % G::NB, mb = i % G::MB;
    acc[nb][mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        __builtin_bit_cast(bf16x8, F.b[s][nb]), __builtin_bit_cast(bf16x8, F.a[s][mb]), acc[nb][mb],
        0, 0, 0);
  }
};

// Zero the summed axis past `left` (values left from the stage's first on), in both operands.
template <class G>
__device__ __forceinline__ void mask_frags(Frags<G>& F, int left, int ln) {
#pragma unroll
  for (int s = 0; s < G::SUB; ++s) {
    const int v = left - 16 * s - 8 * (ln >> 5);  // of this lane's 8
    u32x4 m;
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = v >= 2 * j + 2 ? ~0u : v == 2 * j + 1 ? 0xffffu : 0u;
#pragma unroll
    for (int i = 0; i < G::MB; ++i)
      F.a[s][i] = __builtin_bit_cast(s16x8, __builtin_bit_cast(u32x4, F.a[s][i]) & m);
#pragma unroll
    for (int i = 0; i < G::NB; ++i)
      F.b[s][i] = __builtin_bit_cast(s16x8, __builtin_bit_cast(u32x4, F.b[s][i]) & m);
  }
}

// Stage kt (J = kt % kStages). On entry its fragments are in Fc and the loads of the next
// kStages - 1 stages are in flight. Wait for this wave's loads of stage kt + 1 and its own LDS
// reads of stage kt, then the barrier: after it stage kt + 1 is whole in LDS and stage kt's
// buffer is free. Then the stage's MFMAs, with the reads of stage kt + 1 into Fn and the
// refill of stage kt's buffer (with stage kt + kStages) spread between them. FULL: both happen
// and the next stage and the refill lie inside len; otherwise they are tested.
template <class G, int J, bool FULL>
struct Step {
  static __device__ __forceinline__ void run(int kt, int nk, char* const (&ring)[kStages],
                                             const Loader<G>& ld, Wave<G>& w, Frags<G>& Fc,
                                             Frags<G>& Fn) {
    constexpr int NM = G::SUB * G::NB * G::MB, NR = G::SUB * (G::MB + G::NB), NG = G::LPS;
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (FULL) wait_vmcnt<(kStages - 2) * G::LPS>();
    else wait_stages<G::LPS>(min(kStages - 2, max(nk - 2 - kt, 0)));
    wait_lgkmcnt0();
    sync_point();
    const bool more = FULL || kt + 1 < nk, refill = FULL || kt + kStages < nk;
    const char* src = ring[(J + 1) % kStages];
    char* const dst = ring[J];
    const bool tail = !FULL && !G::TN && (kt + kStages + 1) * G::BK > ld.len;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int m = NM * g / NG; m < NM * (g + 1) / NG; ++m) w.mfma(m, Fc);
      if (more) {
#pragma unroll
        for (int r = NR * g / NG; r < NR * (g + 1) / NG; ++r) w.read(r, src, Fn);
      }
      if (refill) {
        if (!tail) ld.template issue<false>(g, kt + kStages, dst);
        else if constexpr (!FULL && !G::TN) ld.template issue<true>(g, kt + kStages, dst);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!FULL) {
      if (more && (kt + 2) * G::BK > ld.len) mask_frags<G>(Fn, ld.len - (kt + 1) * G::BK, ld.ln);
    }
  }
};

// All stages of a tile (or of a TN segment): nk = ceil(len / BK) > 0.
template <class G>
__device__ __forceinline__ void run_stages(char* const (&ring)[kStages], const Loader<G>& ld,
                                           Wave<G>& w) {
  const int nk = (ld.len + G::BK - 1) / G::BK, whole = ld.len / G::BK;
  Frags<G> F0, F1;
  int kt = 0;
#define MOE_STEP(J, FULL, KT) \
  Step<G, J, FULL>::run(KT, nk, ring, ld, w, (J) % 2 ? F1 : F0, (J) % 2 ? F0 : F1)
  // Prologue and the whole stages in one branch, so that the compiler sees the same loads in
  // flight on every path into the loop.
  if (whole >= 2 * kStages) {
#pragma unroll
    for (int i = 0; i < kStages; ++i)
#pragma unroll
      for (int j = 0; j < G::LPS; ++j) ld.template issue<false>(j, i, ring[i]);
    wait_vmcnt<(kStages - 1) * G::LPS>();
    sync_point();
#pragma unroll
    for (int r = 0; r < G::SUB * (G::MB + G::NB); ++r) w.read(r, ring[0], F0);
    for (; kt + 2 * kStages <= whole; kt += kStages) {
      MOE_STEP(0, true, kt);
      MOE_STEP(1, true, kt + 1);
      MOE_STEP(2, true, kt + 2);
      MOE_STEP(3, true, kt + 3);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      if (i < nk) ld.issue_stage(i, ring[i]);
    wait_stages<G::LPS>(min(kStages, nk) - 1);
    sync_point();
#pragma unroll
    for (int r = 0; r < G::SUB * (G::MB + G::NB); ++r) w.read(r, ring[0], F0);
    if (ld.len < G::BK) mask_frags<G>(F0, ld.len, ld.ln);
  }
  // at most 2 * kStages left
  if (kt < nk) { MOE_STEP(0, false, kt); }
  if (kt + 1 < nk) { MOE_STEP(1, false, kt + 1); }
  if (kt + 2 < nk) { MOE_STEP(2, false, kt + 2); }
  if (kt + 3 < nk) { MOE_STEP(3, false, kt + 3); }
  if (kt + 4 < nk) { MOE_STEP(0, false, kt + 4); }
  if (kt + 5 < nk) { MOE_STEP(1, false, kt + 5); }
  if (kt + 6 < nk) { MOE_STEP(2, false, kt + 6); }
  if (kt + 7 < nk) { MOE_STEP(3, false, kt + 7); }
#undef MOE_STEP
}

// A workgroup's tile: group e, its rows [r0, r1), output tile (mt, nt) of it.
struct TileAt {
  int e, r0, r1, mt, nt;
};

constexpr int kXcds = 8;
constexpr int kColBlock = 4;  // columns of tiles walked together

// Tile `slot` of XCD `xcd`'s share; false past its end. The tiles of all groups are listed
// group after group and each XCD takes a contiguous eighth of the list; within a group,
// blocks of kColBlock tile columns, rows outer and the block's columns inner, so that the
// tiles an XCD runs together share rows of a and columns of b in its L2.
template <class G>
__device__ __forceinline__ bool locate(const MatmulArgs& a, int64_t bid, TileAt& t) {
  const int lane = threadIdx.x & 63;
  const int NT = (int)((a.N + G::BN - 1) / G::BN);
  int start, end;
  group_bounds(a.offsets, a.E, (int)a.R, start, end);
  const int mts = G::TN ? (lane < a.E ? (int)((a.K + G::BM - 1) / G::BM) : 0) : (end - start + G::BM - 1) / G::BM;
  int64_t incl = (int64_t)mts * NT;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
  const int64_t total = __shfl(incl, 63);
  const int xcd = (int)(bid % kXcds);
  const int64_t lo = total * xcd / kXcds, hi = total * (xcd + 1) / kXcds;
  const int64_t i = lo + bid / kXcds;
  if (i >= hi) return false;
  const uint64_t past = __ballot(incl > i);
  t.e = __ffsll((unsigned long long)past) - 1;
  const int m = __shfl(mts, t.e);
  const int in = (int)(i - (__shfl(incl, t.e) - (int64_t)m * NT));
  t.r0 = __shfl(start, t.e);
  t.r1 = __shfl(end, t.e);
  const int blk = in / (m * kColBlock), cols = min(kColBlock, NT - blk * kColBlock);
  const int at = in - blk * m * kColBlock;
  t.mt = at / cols;
  t.nt = blk * kColBlock + at % cols;
  return true;
}

__device__ __forceinline__ int64_t gathered(const int32_t* g, int64_t r, int64_t rows) {
  return g ? min(max((int64_t)g[r], (int64_t)0), rows - 1) : r;
}

template <class G, typename TO>
__global__ __launch_bounds__(256, 1) void matmul_bf16_kernel(MatmulArgs a) {
  // (an array of its own for each stage: the compiler then sees that the reads of one stage
  // do not wait for the loads into another)
  __shared__ __attribute__((aligned(1024))) char s0[G::STAGE], s1[G::STAGE], s2[G::STAGE], s3[G::STAGE];
  __shared__ int tab[G::TN ? 2 * kTable : 1];
  char* const ring[kStages] = {s0, s1, s2, s3};
  TileAt t;
  if (!locate<G>(a, blockIdx.x, t)) return;
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.r0 = __builtin_amdgcn_readfirstlane(t.r0);
  t.r1 = __builtin_amdgcn_readfirstlane(t.r1);
  t.mt = __builtin_amdgcn_readfirstlane(t.mt);
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / G::WGN, wn = wave % G::WGN;
  const int K = (int)a.K, N = (int)a.N;
  const int m0 = t.mt * G::BM + (G::TN ? 0 : t.r0), n0 = t.nt * G::BN;
  const int mend = G::TN ? K : t.r1;
  const bf16* A = static_cast<const bf16*>(a.a);
  const bf16* B = static_cast<const bf16*>(a.b);

  Wave<G> w;
#pragma unroll
  for (int i = 0; i < G::MB; ++i) w.a_at[i] = G::A::frag(wm * G::WM + i * 32, ln);
#pragma unroll
  for (int i = 0; i < G::NB; ++i) w.b_at[i] = G::B::frag(wn * G::WN + i * 32, ln);
#pragma unroll
  for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
      for (int r = 0; r < 16; ++r) w.acc[nb][mb][r] = 0.f;

  Loader<G> ld;
  ld.wave = wave;
  ld.ln = ln;
  if constexpr (G::TN) {
    ld.step_a = K;
    ld.step_b = N;
    ld.ta = tab;
    ld.tb = tab + kTable;
#pragma unroll
    for (int j = 0; j < G::A::PW; ++j) ld.pa[j] = A + min(m0 + G::A::chunk(j, wave, ln) * 8, K - 8);
#pragma unroll
    for (int j = 0; j < G::B::PW; ++j) ld.pb[j] = B + min(n0 + G::B::chunk(j, wave, ln) * 8, N - 8);
    for (int r = t.r0; r < t.r1; r += kTable) {
      __syncthreads();  // the last segment's table is no longer read
      ld.len = min(kTable, t.r1 - r);
      const int fill = (ld.len + G::BK - 1) / G::BK * G::BK;
      for (int i = threadIdx.x; i < fill; i += 256) {
        const int64_t at = r + min(i, ld.len - 1);
        tab[i] = (int)gathered(a.gather_a, at, a.rows_a);
        tab[kTable + i] = (int)gathered(a.gather_b, at, a.rows_b);
      }
      __syncthreads();
      run_stages<G>(ring, ld, w);
    }
  } else {
    const bf16* Be = B + (size_t)t.e * K * N;
    ld.len = K;
    ld.step_a = G::BK;
#pragma unroll
    for (int j = 0; j < G::A::PW; ++j)
      ld.pa[j] = A + (size_t)gathered(a.gather_a, min(m0 + G::A::row(j, wave, ln), t.r1 - 1), a.rows_a) * K +
                 G::A::chunk(j, wave, ln) * 8;
    if constexpr (G::FORM == MOE_MATMUL_NT) {
      ld.step_b = G::BK;
#pragma unroll
      for (int j = 0; j < G::B::PW; ++j)
        ld.pb[j] = Be + (size_t)min(n0 + G::B::row(j, wave, ln), N - 1) * K + G::B::chunk(j, wave, ln) * 8;
    } else {
      ld.step_b = (size_t)G::BK * N;
#pragma unroll
      for (int j = 0; j < G::B::PW; ++j)
        ld.pb[j] = Be + (size_t)G::B::row(j, wave, ln) * N + min(n0 + G::B::chunk(j, wave, ln) * 8, N - 8);
    }
    run_stages<G>(ring, ld, w);
  }

  // acc[nb][mb][4 q + i]: row m = lane % 32 of block mb, column 8 q + 4 (lane / 32) + i of
  // block nb
  TO* out = static_cast<TO*>(a.out) + (G::TN ? (size_t)t.e * K * N : 0);
#pragma unroll
  for (int mb = 0; mb < G::MB; ++mb) {
    const int m = m0 + wm * G::WM + mb * 32 + (ln & 31);
    if (m >= mend) continue;
    TO* row = out + (size_t)m * N;
#pragma unroll
    for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn * G::WN + nb * 32 + 8 * q + 4 * (ln >> 5);
        if (n >= N) continue;  // (N is a multiple of 8)
        f32x4 v = {w.acc[nb][mb][4 * q], w.acc[nb][mb][4 * q + 1], w.acc[nb][mb][4 * q + 2],
                   w.acc[nb][mb][4 * q + 3]};
        if constexpr (sizeof(TO) == 2) {
          *reinterpret_cast<bf16x4*>(row + n) = __builtin_convertvector(v, bf16x4);
        } else {
          if (a.accumulate) v += *reinterpret_cast<const f32x4*>(row + n);
          *reinterpret_cast<f32x4*>(row + n) = v;
        }
      }
  }
}

// ---- fp32 ------------------------------------------------------------------------------
// One workgroup per 64 x 64 tile of the output, 16 of the summed axis at a time through LDS.
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

template <class G, typename TO>
hipError_t launch_bf16(const MatmulArgs& a, hipStream_t s) {
  const int64_t nt = (a.N + G::BN - 1) / G::BN;
  // an upper bound of the tiles, and a multiple of the XCDs: every XCD's eighth (rounded up)
  const int64_t mt = G::TN ? a.E * ((a.K + G::BM - 1) / G::BM) : a.R / G::BM + a.E;
  const int64_t blocks = (mt * nt + kXcds - 1) / kXcds * kXcds;
  matmul_bf16_kernel<G, TO><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int FORM, typename TO>
hipError_t pick(const MatmulArgs& a, hipStream_t s) {
  if constexpr (FORM != MOE_MATMUL_TN) {
    if (a.R <= 32 * (int64_t)a.E) return launch_bf16<Geo<FORM, 32, 128, 64, 1>, TO>(a, s);
  }
  const int64_t mt = FORM == MOE_MATMUL_TN ? a.E * ((a.K + 255) / 256) : a.R / 256 + a.E;
  if (mt * ((a.N + 255) / 256) < 256) return launch_bf16<Geo<FORM, 128, 128, 32, 2>, TO>(a, s);
  return launch_bf16<Geo<FORM, 256, 256, 32, 2>, TO>(a, s);
}

template <typename TO>
hipError_t launch_forms(const MatmulArgs& a, hipStream_t s) {
  if (a.form == MOE_MATMUL_NN) return pick<MOE_MATMUL_NN, TO>(a, s);
  if (a.form == MOE_MATMUL_NT) return pick<MOE_MATMUL_NT, TO>(a, s);
  return pick<MOE_MATMUL_TN, TO>(a, s);
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
  return a.bf16_out ? launch_forms<bf16>(a, s) : launch_forms<float>(a, s);
}

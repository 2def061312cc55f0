// Products of rows grouped by expert, with ragged group sizes: NN (a b_e), NT (a b_e^T) and
// TN (the group's a^T b), fp32 sums.
//
// One workgroup of four waves per BM x BN tile of the output, v_mfma_f32_32x32x16_bf16 or
// v_mfma_f32_32x32x2_f32.
// The summed axis advances in stages of BK through a ring of four LDS buffers filled by
// direct global -> LDS loads. An operand is either K-contiguous in memory (a of NN and NT,
// b of NT), and its fragments are 16-byte LDS reads, or K-strided (b of NN, both of TN), and
// its fragments come out of LDS with transposing reads: no operand is transposed in memory.
// Stages are software-pipelined: while the MFMAs of one stage run from registers, the
// fragments of the next are read from LDS and the stage just consumed is refilled.
// What is out of range is never loaded: addresses are clamped to the last row, column or
// chunk, and the values of the summed axis past its end are zeroed in both operands'
// fragments (the last stage only), so that a non-finite value there reaches no sum.
//
// Bounds: the matrix cores where groups are long (128 FLOP per byte of a 256 x 256 tile's
// operands and more), the weights' bytes where they are a few rows, and the output's bytes in
// TN with short sums, whose stores go out between two tiles' loads and are waited for with
// them. Measured, bf16, gathered rows, where a copy reaches 5.1 TB/s and a large square
// product 1197 TFLOP/s: 32768 skewed rows of 8 groups, K 4096, N 14336: NT 3.2 ms (1200
// TFLOP/s), NN 3.03 ms (1268), TN 3.3 ms (1163); 8192 rows of 8, K 1024, N 4096: NN 83 us
// (822 TFLOP/s, 57 us at those rates); 32764 rows of 64, 2048 x 1408: TN with fp32 results 300
// us (629 TFLOP/s and 2.9 TB/s at once; 168 us for the slower of the two alone); 16 rows of 8,
// K 4096, N 14336: NN 152-159 us (5.9-6.2 TB/s). fp32, 8192 rows of 8, K 1024, N 4096: NN 562 us
// (122 TFLOP/s, a large square product 134).
#include <math.h>

#include <type_traits>

#include "matmul_tile.h"
#include "train_common.h"
#include "train_kernels.h"

#include "moe.h"

namespace {

// One operand's stage in LDS: X rows (its output axis) by BK of the summed axis.
//   K-contiguous (KS false): [X][BK], 16-byte chunk c of a row stored at c ^ swz(row).
//   K-strided (KS true): [BK][X], 16-byte slot s of a row stored at s ^ swz(row).
// Both swizzles make the fragment reads free of bank conflicts. A direct load instruction
// moves 64 lanes x 16 bytes into 1 KB of LDS, lane l into slot l.
template <typename T, bool KS_, int X_, int BK_, int NW>
struct Operand {
  static constexpr bool KS = KS_;
  static constexpr int X = X_, BK = BK_, EB = sizeof(T), EPC = 16 / EB;  // elements per chunk
  static constexpr int BYTES = X * BK * EB;
  static constexpr int PW = BYTES / 1024 / NW;         // loads per wave and stage
  static constexpr int ROW = (KS ? X : BK) * EB;       // bytes per LDS row
  static constexpr int SLOTS = ROW / 16;               // chunks per LDS row
  static constexpr int RPI = 1024 / ROW;               // LDS rows per load instruction
  static_assert(PW >= 1 && BYTES % (1024 * NW) == 0, "whole loads per wave");
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (KS) return ((0xCA60 >> (4 * (row & 3))) & 15) % SLOTS;
    else if constexpr (SLOTS == 4) return (row >> 2) & 3;
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
    if constexpr (!KS) {
      const int m = x0 + (ln & 31);
      return m * ROW + ((ln >> 5) ^ swz(m)) * 16;
    } else if constexpr (EB == 2) {
      const int g = ln >> 4, r = (ln & 15) >> 2, c = ln & 3;
      const int n = x0 + (g & 1) * 16 + 4 * c, k = (g >> 1) * 8 + r;
      return k * ROW + ((n >> 3) ^ swz(k)) * 16 + ((n >> 2) & 1) * 8;
    } else {
      return (ln >> 5) * 4 * ROW + (x0 + (ln & 31)) * 4;  // (rows 4 h + i, swizzled by i below)
    }
  }
  // The fragment of substep s, 16 bytes. bf16: k = 16 s + 8 h .. + 7 (h = lane / 32); fp32:
  // k = 8 s + 4 h .. + 3.
  static __device__ __forceinline__ u32x4 read(const char* st, int at, int s) {
    if constexpr (!KS) {
      return *reinterpret_cast<const u32x4*>(st + (at ^ (32 * s)));
    } else if constexpr (EB == 2) {
      const char* p = st + at + 16 * s * ROW;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ROW));
      return __builtin_bit_cast(u32x4, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    } else {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const uint32_t*>(st + (at ^ (swz(i) * 16)) + (8 * s + i) * ROW);
      return v;
    }
  }
};

// BM x BN tile, WGM x (4 / WGM) waves. STREAM: b's loads are non-temporal.
template <typename T, int FORM_, int BM_, int BN_, int BK_, int WGM, bool STREAM_ = false>
struct Geo {
  typedef T type;
  static constexpr bool STREAM = STREAM_;
  static constexpr int FORM = FORM_, BM = BM_, BN = BN_, BK = BK_;
  static constexpr bool TN = FORM == MOE_MATMUL_TN;
  static constexpr int EPC = 16 / sizeof(T);
  static constexpr int WGN = 4 / WGM, SUB = BK / (2 * EPC);
  static constexpr int RW = BK / 4;  // TN: rows of the summed axis that a wave loads per stage
  typedef Operand<T, TN, BM, BK, 4> A;
  typedef Operand<T, FORM != MOE_MATMUL_NT, BN, BK, 4> B;
  static constexpr int WM = BM / WGM, WN = BN / WGN, MB = WM / 32, NB = WN / 32;
  static constexpr int STAGE = A::BYTES + B::BYTES, LPS = A::PW + B::PW;
  // LDS of each wave for its output: 32 rows of its columns in bf16 (the 32-row tiles have
  // none left, and little to store)
  static constexpr int OUT_BYTES = BM >= 128 ? 32 * WN * 2 : 0;
};

// Sources of a tile's direct loads. NN, NT: one pointer per load, advancing by a fixed step
// per stage. TN: the rows are the summed axis, and each load takes its row's index (the
// gather's, or the row itself) from the turn's indices.
template <class G>
struct Loader {
  typedef typename G::type T;
  const T* pa[G::A::PW];
  const T* pb[G::B::PW];
  size_t step_a, step_b;  // elements per stage (TN: per row)
  int len, wave, ln;

};

// One operand's address of load j of stage kt (NN, NT). Stages may end past len where CLAMP:
// the last chunk (or row) is then read again. (Class templates: hipcc's host pass rejects
// later calls of these as function templates once they are instantiated from two callers.)
template <class G, class Op, bool CLAMP>
struct Source {
  typedef typename G::type T;
  static __device__ __forceinline__ const T* at(const Loader<G>& ld, const T* p, size_t step, int j, int kt) {
    const T* q = p + (size_t)kt * step;
    if constexpr (CLAMP) {
      const int l = G::BM == 256 ? here(ld.ln) : ld.ln;
      const int k = kt * G::BK + (Op::KS ? Op::row(j, ld.wave, l) : Op::chunk(j, ld.wave, l) * G::EPC);
      const int back = min(0, ld.len - (Op::KS ? 1 : G::EPC) - k);
      // (at most two ring turns back, of rows of at most 2^20 values)
      q += Op::KS ? back * (int)(step / G::BK) : back;
    }
    return q;
  }
};

// Load j (A's, then B's; a constant at every call) of stage kt into st; TN: of the rows that
// `turn` holds for ring place q.
template <class G, bool CLAMP>
struct Issue {
  typedef typename G::type T;
  static __device__ __forceinline__ void run(const Loader<G>& ld, int j, int kt, int turn, int q, char* st) {
    const bool is_a = j < G::A::PW;
    const int i = is_a ? j : j - G::A::PW;
    const T* p;
    if constexpr (G::TN) {
      // the rows of one load instruction are consecutive lanes of `turn`
      constexpr int RPI = G::A::RPI;
      static_assert(RPI * G::A::PW == G::RW && G::B::RPI == RPI && G::B::PW == G::A::PW, "rows per wave");
      const int l0 = (is_a ? 0 : 32) + q * G::RW + i * RPI, mine = ld.ln / (64 / RPI);
      int row = __builtin_amdgcn_readlane(turn, l0);
#pragma unroll
      for (int r = 1; r < RPI; ++r) {
        const int v = __builtin_amdgcn_readlane(turn, l0 + r);
        row = mine >= r ? v : row;
      }
      p = is_a ? ld.pa[i] + (int64_t)row * (int64_t)ld.step_a : ld.pb[i] + (int64_t)row * (int64_t)ld.step_b;
    } else {
      p = is_a ? Source<G, typename G::A, CLAMP>::at(ld, ld.pa[i], ld.step_a, i, kt)
               : Source<G, typename G::B, CLAMP>::at(ld, ld.pb[i], ld.step_b, i, kt);
    }
    char* to = is_a ? st + (ld.wave * G::A::PW + i) * 1024
                    : st + G::A::BYTES + (ld.wave * G::B::PW + i) * 1024;
    if (G::STREAM && !is_a) __builtin_amdgcn_global_load_lds(p, (lds_void*)to, 16, 0, 2);
    else __builtin_amdgcn_global_load_lds(p, (lds_void*)to, 16, 0, 0);
  }
};

template <class G>
struct Frags {
  u32x4 a[G::SUB][G::MB], b[G::SUB][G::NB];
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
  // one fragment of each operand (fp32: four instructions, two deep each)
  __device__ __forceinline__ void mfma(int i, const Frags<G>& F) {
    const int s = i / (G::NB * G::MB), nb = i / G::MB % G::NB, mb = i % G::MB;
    if constexpr (sizeof(typename G::type) == 2) {
      acc[nb][mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(bf16x8, F.b[s][nb]), __builtin_bit_cast(bf16x8, F.a[s][mb]), acc[nb][mb],
          0, 0, 0);
    } else {
      const f32x4 b = __builtin_bit_cast(f32x4, F.b[s][nb]), a = __builtin_bit_cast(f32x4, F.a[s][mb]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[nb][mb] = __builtin_amdgcn_mfma_f32_32x32x2f32(b[j], a[j], acc[nb][mb], 0, 0, 0);
    }
  }
};

// Zero the summed axis past `left` (values left from the stage's first on), in both operands.
template <class G>
__device__ __forceinline__ void mask_frags(Frags<G>& F, int left, int ln) {
#pragma unroll
  for (int s = 0; s < G::SUB; ++s) {
    const int v = left - G::EPC * (2 * s + (ln >> 5));  // of this lane's EPC
    u32x4 m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (G::EPC == 8) m[j] = v >= 2 * j + 2 ? ~0u : v == 2 * j + 1 ? 0xffffu : 0u;
      else m[j] = v > j ? ~0u : 0u;
    }
#pragma unroll
    for (int i = 0; i < G::MB; ++i) F.a[s][i] &= m;
#pragma unroll
    for (int i = 0; i < G::NB; ++i) F.b[s][i] &= m;
  }
}

// Stage kt (J = kt % kStages). On entry its fragments are in Fc and the loads of the next
// kStages - 1 stages are in flight. Wait for this wave's loads of the next stage and its own
// LDS reads of this one, then the barrier: after it the next stage is whole in LDS and this
// stage's buffer is free. Then the stage's MFMAs, with the reads of the next stage into Fn and
// the refill of this buffer (stage `rs` of ld) spread between them.
// Every step loads and reads the same amounts, so that the loads in flight are known at
// every wait (where paths join inside a turn, the compiler loses count and waits for all of
// them): past an item's last stage the refills are the next item's first stages, and an item
// is a whole number of ring turns, whose spare stages run on zeros.
template <class G>
struct Wait {
  static __device__ __forceinline__ void run() {
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<(kStages - 2) * G::LPS>();
    wait_lgkmcnt0();
    sync_point();
  }
};
template <class G, int J, bool CLAMP>
struct Step {
  static __device__ __forceinline__ void run(int rs, int turn, char* const (&ring)[kStages],
                                             const Loader<G>& ld, Wave<G>& w, Frags<G>& Fc,
                                             Frags<G>& Fn) {
    constexpr int NM = G::SUB * G::NB * G::MB, NR = G::SUB * (G::MB + G::NB), NG = G::LPS;
    const char* src = ring[(J + 1) % kStages];
    char* const dst = ring[J];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int m = NM * g / NG; m < NM * (g + 1) / NG; ++m) w.mfma(m, Fc);
#pragma unroll
      for (int r = NR * g / NG; r < NR * (g + 1) / NG; ++r) w.read(r, src, Fn);
      Issue<G, CLAMP>::run(ld, g, rs, turn, J, dst);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Fragments of the first stage of an item of length len, once read.
template <class G>
__device__ __forceinline__ void mask_first(Frags<G>& F, int len, int ln) {
  if (len < G::BK) mask_frags<G>(F, len, ln);
}

// A workgroup's work: output tile (mt, nt) of group e, whose rows are [r0, r1), over a part of
// the summed axis: NN, NT [k0, k0 + len); TN rows [r0, r1) are that part. `split`: which of
// the part sums it is (TN: -1 for a whole sum, which goes to out).
struct Item {
  int e, r0, r1, mt, nt, k0, len, split;
};

constexpr int kXcds = 8;
constexpr int kCus = 256;
constexpr int kColBlock = 4;  // columns of tiles walked together
// The XCD's share of the tiles, lo .. hi of a list.
// NN, NT (every tile has the same work): the tiles of all groups group after group, of which
// each XCD takes a contiguous eighth.
// TN (a tile's work goes with its group's rows): the XCD takes an eighth of every group's
// tiles, the groups by falling length, so that all XCDs have the same work and the long
// tiles come first; `list` deals them in alternating order.
// Within a group, blocks of kColBlock tile columns, rows outer and the block's columns
// inner, so that the tiles an XCD runs together share rows of a and columns of b in its L2.
struct Groups {  // lane i: the i-th group of the list
  int e, start, end, first, incl;  // first: the share's first tile in the group; incl: tiles so far
  int parts, slot;  // TN: parts of the group's sum, and the first one's place among all part sums
};

// TN: in how many parts a group's sum is taken, so that none of them is much longer than a CU's
// share of the work, and the place of the group's first part sum (lane e: group e).
constexpr int kMaxParts = 32;
__device__ __forceinline__ void group_parts(const MatmulArgs& a, int len, int& parts, int& slot) {
  const int lane = threadIdx.x & 63;
  parts = 1;
  if (a.part_rows && len > a.part_rows)
    parts = (int)min(((int64_t)len + a.part_rows - 1) / a.part_rows, (int64_t)kMaxParts);
  const int mine = parts > 1 ? parts : 0;
  slot = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(slot, o);
    if (lane >= o) slot += v;
  }
  slot -= mine;
}

template <class G>
__device__ __forceinline__ void make_groups(const MatmulArgs& a, int xcd, Groups& g, int& lo, int& hi) {
  const int lane = threadIdx.x & 63;
  const int NT = (int)((a.N + G::BN - 1) / G::BN);
  int start, end;
  group_bounds(a.offsets, a.E, (int)a.R, start, end);
  g = Groups{lane, start, end, 0, 0, 1, 0};
  int tiles;  // (with splits: each part is a tile of its own)
  if constexpr (G::TN) {
    int parts, slot;
    group_parts(a, end - start, parts, slot);
    const int len = lane < a.E ? (end - start) / parts : -1;
    int rank = 0;
    for (int j0 = 0; j0 < a.E; j0 += 8)
#pragma unroll
      for (int j = j0; j < j0 + 8; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < lane);
      }
    if (lane >= a.E) rank = lane;
    g.e = __builtin_amdgcn_ds_permute(4 * rank, lane);
    g.start = __builtin_amdgcn_ds_permute(4 * rank, start);
    g.end = __builtin_amdgcn_ds_permute(4 * rank, end);
    g.parts = __builtin_amdgcn_ds_permute(4 * rank, parts);
    g.slot = __builtin_amdgcn_ds_permute(4 * rank, slot);
    const int64_t n = lane < a.E ? (a.K + G::BM - 1) / G::BM * NT * g.parts : 0;
    const int x = (xcd + lane) % kXcds;  // (a group of few tiles: another XCD's for each)
    g.first = (int)(n * x / kXcds);
    tiles = (int)(n * (x + 1) / kXcds) - g.first;
  } else {
    tiles = (end - start + G::BM - 1) / G::BM * NT * a.splits;
  }
  g.incl = tiles;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(g.incl, o);
    if (lane >= o) g.incl += v;
  }
  const int64_t all = __builtin_amdgcn_readlane(g.incl, 63);
  lo = G::TN ? 0 : (int)(all * xcd / kXcds);
  hi = G::TN ? (int)all : (int)(all * (xcd + 1) / kXcds);
}

template <class G>
__device__ __forceinline__ Item locate(const MatmulArgs& a, const Groups& g, int i) {
  Item t;
  const int NT = (int)((a.N + G::BN - 1) / G::BN);
  const int at_group = __ffsll((unsigned long long)__ballot(g.incl > i)) - 1;
  t.e = __builtin_amdgcn_readlane(g.e, at_group);
  t.r0 = __builtin_amdgcn_readlane(g.start, at_group);
  t.r1 = __builtin_amdgcn_readlane(g.end, at_group);
  const int m = G::TN ? (int)((a.K + G::BM - 1) / G::BM) : (t.r1 - t.r0 + G::BM - 1) / G::BM;
  const int before = at_group ? __builtin_amdgcn_readlane(g.incl, at_group - 1) : 0;
  const int part = i - before + __builtin_amdgcn_readlane(g.first, at_group);
  // TN: a part's tiles one after another (they share its rows), else a tile's parts
  const int parts = G::TN ? __builtin_amdgcn_readlane(g.parts, at_group) : a.splits;
  const int in = G::TN ? part % (m * NT) : part / parts;
  int split = G::TN ? part / (m * NT) : part - in * parts;
  const int blk = in / (m * kColBlock), cols = min(kColBlock, NT - blk * kColBlock);
  const int at = in - blk * m * kColBlock;
  t.mt = at / cols;
  t.nt = blk * kColBlock + at % cols;
  t.k0 = 0;
  t.len = G::TN ? t.r1 - t.r0 : (int)a.K;
  if (parts > 1) {  // whole stages per part; the last ones may be empty
    const int per = ((t.len + G::BK - 1) / G::BK + parts - 1) / parts * G::BK;
    t.k0 = min(split * per, t.len);
    t.len = min(per, t.len - t.k0);
    if constexpr (G::TN) {
      t.r0 += t.k0;
      t.r1 = t.r0 + t.len;
      split += __builtin_amdgcn_readlane(g.slot, at_group);
    }
  } else if (G::TN) {
    split = -1;
  }
  t.split = split;
  return t;
}

// TN: rows of the problem that a wave loads in a ring turn (four stages) of a group: RW of each
// stage's BK rows, so lane l < 4 RW stands for a's row of stage l / RW, place l % RW, and lane
// 32 + l for b's. Rows past the group's end give its last one again.
template <class G>
__device__ __forceinline__ int turn_row(const Item& t, int turn, int wave, int lane) {
  static_assert(!G::TN || kStages * G::RW <= 32, "a turn's rows in half a wave");
  const int l = (lane & 31) % (kStages * G::RW);
  const int64_t at = (int64_t)t.r0 + (int64_t)turn * (kStages * G::BK) + l / G::RW * G::BK +
                     wave * G::RW + l % G::RW;
  return (int)max(min(at, (int64_t)t.r1 - 1), (int64_t)0);
}
// Their gathered indices, fetched ahead and taken (clamped) a turn later. The load is always
// issued (without a gather, of any word): under a test the compiler would copy its value, and
// so wait for it, and for everything in flight, right away.
template <class G>
__device__ __forceinline__ int fetch_turn(const MatmulArgs& a, const Item& t, int turn, int wave, int lane) {
  if constexpr (!G::TN) return 0;
  const int32_t* g = lane < 32 ? a.gather_a : a.gather_b;
  const int32_t* p = g ? g + turn_row<G>(t, turn, wave, lane) : a.offsets;
  return *p;
}
template <class G>
__device__ __forceinline__ int take_turn(const MatmulArgs& a, const Item& t, int turn, int fetched, int wave,
                                         int lane) {
  if constexpr (!G::TN) return 0;
  const int64_t rows = lane < 32 ? a.rows_a : a.rows_b;
  const bool gathers = (lane < 32 ? a.gather_a : a.gather_b) != nullptr;
  const int g = (int)min(max((int64_t)fetched, (int64_t)0), rows - 1);
  return here(gathers ? g : turn_row<G>(t, turn, wave, lane));
}

// What a tile's loads take from memory, raw: NN, NT the gathered rows of a of this lane's
// loads, TN the row indices of the first turn.
template <class G>
struct Ahead {
  int rows[G::TN ? 1 : G::A::PW], turn;
  static __device__ __forceinline__ int row(const Item& t, int j, int wave, int ln) {
    return min(t.r0 + t.mt * G::BM + G::A::row(j, wave, ln), t.r1 - 1);
  }
  __device__ __forceinline__ void fetch(const MatmulArgs& a, const Item& t, int wave, int lane) {
    turn = fetch_turn<G>(a, t, 0, wave, lane);
    if constexpr (!G::TN) {
      const int ln = here(lane);
#pragma unroll
      for (int j = 0; j < G::A::PW; ++j) {
        const int32_t* p = a.gather_a ? a.gather_a + row(t, j, wave, ln) : a.offsets;
        rows[j] = *p;
      }
    }
  }
};

// The item's sources, in `ld`.
template <class G>
__device__ __forceinline__ void make_loader(const MatmulArgs& a, const Item& t, int wave, int lane,
                                            const Ahead<G>& ahead, Loader<G>& ld) {
  const int K = (int)a.K, N = (int)a.N, n0 = t.nt * G::BN;
  typedef typename G::type T;
  constexpr int C = G::EPC;
  const T* A = static_cast<const T*>(a.a);
  const T* B = static_cast<const T*>(a.b);
  const int ln = here(lane);
  ld.wave = wave;
  ld.ln = lane;
  if constexpr (G::TN) {
    const int m0 = t.mt * G::BM;
    ld.len = t.len;
    ld.step_a = K;
    ld.step_b = N;
#pragma unroll
    for (int j = 0; j < G::A::PW; ++j) ld.pa[j] = A + min(m0 + G::A::chunk(j, wave, ln) * C, K - C);
#pragma unroll
    for (int j = 0; j < G::B::PW; ++j) ld.pb[j] = B + min(n0 + G::B::chunk(j, wave, ln) * C, N - C);
  } else {
    const T* Be = B + (size_t)t.e * K * N;
    ld.len = t.len;
    ld.step_a = G::BK;
#pragma unroll
    for (int j = 0; j < G::A::PW; ++j) {
      const int64_t g = min(max((int64_t)ahead.rows[j], (int64_t)0), a.rows_a - 1);
      const int64_t r = a.gather_a ? g : Ahead<G>::row(t, j, wave, ln);
      ld.pa[j] = A + (size_t)r * K + t.k0 + G::A::chunk(j, wave, ln) * C;
    }
    if constexpr (G::FORM == MOE_MATMUL_NT) {
      ld.step_b = G::BK;
#pragma unroll
      for (int j = 0; j < G::B::PW; ++j)
        ld.pb[j] = Be + (size_t)min(n0 + G::B::row(j, wave, ln), N - 1) * K + t.k0 + G::B::chunk(j, wave, ln) * C;
    } else {
      ld.step_b = (size_t)G::BK * N;
#pragma unroll
      for (int j = 0; j < G::B::PW; ++j)
        ld.pb[j] = Be + (size_t)(t.k0 + G::B::row(j, wave, ln)) * N + min(n0 + G::B::chunk(j, wave, ln) * C, N - C);
    }
  }
}

// Output. acc[nb][mb][4 q + i] is row lane % 32 of block mb, column 8 q + 4 (lane / 32) + i of
// block nb: stored from there, an instruction would touch 32 rows with 8 or 16 bytes each,
// and the writes, not their bytes, would bound the tile's end. The 128- and 256-row tiles
// pass 32 rows at a time through a piece of LDS of the wave's own (16-byte chunk c of a row
// at c ^ (row % chunks)) and store whole row segments.
// ADD: to out's values (a part sum: to zeros). Each pass's are loaded a pass ahead, and loads
// and stores outside the tile's rows and columns go out of a buffer's range instead of being
// left out: without branches the waits for the loads do not include the stores before them
// (TN, 32768 rows of 64 groups, 2048 x 1408: 712 -> 407 us, 281 stored; NT, K 1408, N 2048: 418 -> 310).
template <class G, typename TO, bool ADD>
__device__ __forceinline__ void store_tile(const MatmulArgs& a, const Item& t, int wm, int wn, int lane,
                                           char* buf, const Wave<G>& w) {
  const int ln = here(lane);
  const int K = (int)a.K, N = (int)a.N;
  const int m0 = t.mt * G::BM + (G::TN ? 0 : t.r0) + wm * G::WM, mend = G::TN ? K : t.r1;
  const int n0 = t.nt * G::BN + wn * G::WN;
  const bool part = G::TN && t.split >= 0;
  TO* out = static_cast<TO*>(a.out) + (G::TN ? (size_t)t.e * K * N : (size_t)t.split * a.split_stride);
  if constexpr (G::TN && sizeof(TO) == 4) {
    if (part) out = a.parts + (size_t)t.split * K * N;
  }
  auto vec = [&](int mb, int nb, int q) {
    return f32x4{w.acc[nb][mb][4 * q], w.acc[nb][mb][4 * q + 1], w.acc[nb][mb][4 * q + 2],
                 w.acc[nb][mb][4 * q + 3]};
  };
  if constexpr (G::OUT_BYTES == 0) {
#pragma unroll
    for (int mb = 0; mb < G::MB; ++mb) {
      const int m = m0 + mb * 32 + (ln & 31);
      if (m >= mend) continue;
#pragma unroll
      for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + nb * 32 + 8 * q + 4 * (ln >> 5);
          if (n >= N) continue;  // (N is a multiple of 4)
          TO* p = out + (size_t)m * N + n;
          f32x4 v = vec(mb, nb, q);
          if constexpr (sizeof(TO) == 2) {
            *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
          } else {
            if constexpr (ADD) v += *reinterpret_cast<const f32x4*>(p);
            *reinterpret_cast<f32x4*>(p) = v;
          }
        }
    }
  } else {
    // The values are put there in fp32 by the 256-row tiles, whose accumulators go into LDS
    // as they are (converting them first takes registers those tiles do not have: the
    // spills' reloads wait for every load and store in flight), in TO by the 128-row ones.
    typedef typename std::conditional<G::BM == 256, float, TO>::type TL;
    constexpr int SEG = G::OUT_BYTES / 32, CHUNKS = SEG / 16;        // of a row, per pass
    constexpr int COLS = SEG / (int)sizeof(TL), BLOCKS = COLS / 32;  // columns, 32-column blocks
    constexpr int N16 = 16 / (int)sizeof(TO), PER = COLS / N16;      // a lane's columns; lanes per row
    constexpr int RPS = 64 / PER;                                    // rows per store instruction
    constexpr int PASSES = G::MB * (G::NB / BLOCKS);
    // (from the wave's corner of the tile: at most 256 rows of 2^20 values)
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(out + (size_t)m0 * N + n0, 0, 0x7fffffff, 0x00020000);
    auto place = [&](int pass, int i) {  // byte offset of this lane's chunk of store i
      const int row = pass / (G::NB / BLOCKS) * 32 + i * RPS + ln / PER;
      const int col = pass % (G::NB / BLOCKS) * COLS + ln % PER * N16;
      return m0 + row < mend && n0 + col < N ? (row * N + col) * (int)sizeof(TO) : (int)0x80000000;
    };
    u32x4 old[ADD ? 2 : 1][32 / RPS];
    auto fetch = [&](int pass) {
#pragma unroll
      for (int i = 0; i < 32 / RPS; ++i)
        old[ADD ? pass % 2 : 0][i] =
            __builtin_amdgcn_raw_buffer_load_b128(rsrc, part ? (int)0x80000000 : place(pass, i), 0, 0);
    };
    if constexpr (ADD) fetch(0);
#pragma unroll
    for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
      for (int nb0 = 0; nb0 < G::NB; nb0 += BLOCKS) {
        __builtin_amdgcn_sched_barrier(0);  // (one pass's registers at a time)
        const int r = ln & 31, pass = mb * (G::NB / BLOCKS) + nb0 / BLOCKS;
        if constexpr (ADD) {
          if (pass + 1 < PASSES) fetch(pass + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int nb = 0; nb < BLOCKS; ++nb)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at = (nb * 32 + 8 * q + 4 * (ln >> 5)) * (int)sizeof(TL);
            char* p = buf + r * SEG + (((at >> 4) ^ (r % CHUNKS)) << 4) + (at & 15);
            const f32x4 v = vec(mb, nb0 + nb, q);
            if constexpr (sizeof(TL) == 2) *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
            else *reinterpret_cast<f32x4*>(p) = v;
          }
#pragma unroll
        for (int i = 0; i < 32 / RPS; ++i) {
          const int row = i * RPS + ln / PER, c = ln % PER;
          const int m = m0 + mb * 32 + row, n = n0 + nb0 * 32 + c * N16;
          auto chunk = [&](int k) {
            return *reinterpret_cast<const u32x4*>(buf + row * SEG + ((k ^ (row % CHUNKS)) << 4));
          };
          u32x4 v;
          if constexpr (sizeof(TL) == sizeof(TO)) {
            v = chunk(c);
          } else {
            const bf16x4 lo = __builtin_convertvector(__builtin_bit_cast(f32x4, chunk(2 * c)), bf16x4);
            const bf16x4 hi = __builtin_convertvector(__builtin_bit_cast(f32x4, chunk(2 * c + 1)), bf16x4);
            v = __builtin_bit_cast(u32x4, bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
          }
          if constexpr (ADD) {
            v = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, v) + __builtin_bit_cast(f32x4, old[pass % 2][i]));
            __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, place(pass, i), 0, 2);  // (2: non-temporal)
          } else {
            if (m >= mend || n >= N) continue;  // (N is a multiple of a chunk)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + (size_t)m * N + n));
          }
        }
      }
  }
}

// Workgroups take their XCD's tiles in strides of the XCD's workgroups, as one stream of
// stages: the last ring turn of an item loads the first one of the next.
template <class G, typename TO, bool ADD>
__global__ __launch_bounds__(256, 1) void grouped_matmul_kernel(MatmulArgs a) {
  // (an array of its own for each stage: the compiler then sees that the reads of one stage
  // do not wait for the loads into another)
  __shared__ __attribute__((aligned(1024))) char s0[G::STAGE], s1[G::STAGE], s2[G::STAGE], s3[G::STAGE];
  __shared__ __attribute__((aligned(1024))) char outs[G::OUT_BYTES ? 4 * G::OUT_BYTES : 16];
  char* const ring[kStages] = {s0, s1, s2, s3};
  const int ln = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / G::WGN, wn = wave % G::WGN;
  const int slots = gridDim.x / kXcds;
  Groups groups;
  int lo, hi;
  make_groups<G>(a, blockIdx.x % kXcds, groups, lo, hi);
  // this workgroup's tiles: one of every `slots`; TN: in alternating order, so that who had
  // the longest of one round has the shortest of the next
  const int slot = blockIdx.x / kXcds;
  int round = 0;
  auto place = [&](int r) { return lo + r * slots + (G::TN && r % 2 ? slots - 1 - slot : slot); };
  const int i = place(0);
  if (i >= hi) return;

  Wave<G> w;
#pragma unroll
  for (int j = 0; j < G::MB; ++j) w.a_at[j] = G::A::frag(wm * G::WM + j * 32, ln);
#pragma unroll
  for (int j = 0; j < G::NB; ++j) w.b_at[j] = G::B::frag(wn * G::WN + j * 32, ln);
  // What the loads of a tile need to be told by memory (NN, NT: the rows of a; TN: the row
  // indices of its first turn) is fetched two tiles ahead: a whole turn, with its waits, then
  // lies between the fetch and the use, whatever the tiles' lengths.
  Loader<G> ld;
  Ahead<G> one, two;
  Item t = locate<G>(a, groups, i);
  one.fetch(a, t, wave, ln);
  make_loader<G>(a, t, wave, ln, one, ld);
  Frags<G> F0, F1;
  // TN: row indices of the turn whose loads come next
  int turn = fetch_turn<G>(a, t, 1, wave, ln);
  {
    const int now = take_turn<G>(a, t, 0, one.turn, wave, ln);
    one.fetch(a, place(1) < hi ? locate<G>(a, groups, place(1)) : t, wave, ln);
#pragma unroll
    for (int q = 0; q < kStages; ++q)
#pragma unroll
      for (int j = 0; j < G::LPS; ++j) Issue<G, true>::run(ld, j, q, now, q, ring[q]);
  }
  wait_vmcnt<(kStages - 1) * G::LPS>();
  sync_point();
#pragma unroll
  for (int r = 0; r < G::SUB * (G::MB + G::NB); ++r) w.read(r, ring[0], F0);

  for (;;) {
#pragma unroll
    for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
      for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
        for (int r = 0; r < 16; ++r) w.acc[nb][mb][r] = 0.f;
    const Item cur = t;
    const int len = ld.len, nk = (len + G::BK - 1) / G::BK, whole = len / G::BK;
    const int end = max((nk + kStages - 1) / kStages, 1) * kStages;  // whole ring turns
    const bool more = place(++round) < hi;
    if (more) t = locate<G>(a, groups, place(round));
    two.fetch(a, place(round + 1) < hi ? locate<G>(a, groups, place(round + 1)) : t, wave, ln);

    mask_first<G>(F0, len, ln);
    int kt = 0;
#define MOE_STEP(J, CLAMP, RS) \
  Wait<G>::run();              \
  Step<G, J, CLAMP>::run(RS, now, ring, ld, w, (J) % 2 ? F1 : F0, (J) % 2 ? F0 : F1)
    for (; kt + 2 * kStages <= whole && kt + kStages < end; kt += kStages) {
      const int now = take_turn<G>(a, cur, kt / kStages + 1, turn, wave, ln);
      turn = fetch_turn<G>(a, cur, kt / kStages + 2, wave, ln);
      MOE_STEP(0, false, kt + 4);
      MOE_STEP(1, false, kt + 5);
      MOE_STEP(2, false, kt + 6);
      MOE_STEP(3, false, kt + 7);
    }
    if (kt + kStages < end) {  // the refills end past len
      const int now = take_turn<G>(a, cur, kt / kStages + 1, turn, wave, ln);
      MOE_STEP(0, true, kt + 4);
      MOE_STEP(1, true, kt + 5);
      MOE_STEP(2, true, kt + 6);
      MOE_STEP(3, true, kt + 7);
      kt += kStages;
      if ((kt + 1) * G::BK > len) mask_frags<G>(F0, len - kt * G::BK, ln);
    }
    // the last turn: the next item's first stages (without one, this item's, never used)
    const int now = take_turn<G>(a, t, 0, one.turn, wave, ln);
    if (more) make_loader<G>(a, t, wave, ln, one, ld);
    turn = fetch_turn<G>(a, t, 1, wave, ln);
    const int left = len - kt * G::BK;
    MOE_STEP(0, true, 0);
    if (left < 2 * G::BK) mask_frags<G>(F1, left - G::BK, ln);
    MOE_STEP(1, true, 1);
    if (left < 3 * G::BK) mask_frags<G>(F0, left - 2 * G::BK, ln);
    MOE_STEP(2, true, 2);
    if (left < 4 * G::BK) mask_frags<G>(F1, left - 3 * G::BK, ln);
    MOE_STEP(3, true, 3);
#undef MOE_STEP
    if (G::TN && sizeof(TO) == 2 && cur.split >= 0)
      store_tile<G, float, false>(a, cur, wm, wn, ln, outs + wave * G::OUT_BYTES, w);
    else
      store_tile<G, TO, ADD>(a, cur, wm, wn, ln, outs + wave * G::OUT_BYTES, w);
    if (!more) break;
    one = two;
  }
  wait_vmcnt<0>();  // the loads that nobody reads have landed before the LDS is given back
}

// Parts' sums, in order, into out. NN, NT: from the first group's start to the last one's end (only
// these rows have sums); TN: of the groups that have parts, a group per grid row.
template <typename TO>
__global__ __launch_bounds__(256) void join_parts_kernel(MatmulArgs a, const float* __restrict__ sums) {
  TO* out = static_cast<TO*>(a.out);
  int parts = a.splits, start, end;
  int64_t from = 0, n = a.split_stride;
  const int last = group_bounds(a.offsets, a.E, (int)a.R, start, end);
  if (a.form == MOE_MATMUL_TN) {
    int all, slot;
    group_parts(a, end - start, all, slot);
    parts = __builtin_amdgcn_readlane(all, blockIdx.y);
    if (parts < 2) return;
    sums += (size_t)__builtin_amdgcn_readlane(slot, blockIdx.y) * a.split_stride;
    out += (size_t)blockIdx.y * a.split_stride;
  } else {
    from = (int64_t)__builtin_amdgcn_readlane(start, 0) * a.N;
    n = (int64_t)last * a.N;
  }
  for (int64_t i = from + ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    f32x4 v = *reinterpret_cast<const f32x4*>(sums + i);
#pragma unroll 4
    for (int p = 1; p < parts; ++p) v += *reinterpret_cast<const f32x4*>(sums + p * a.split_stride + i);
    if constexpr (sizeof(TO) == 2) {
      *reinterpret_cast<bf16x4*>(out + i) = __builtin_convertvector(v, bf16x4);
    } else {
      if (a.accumulate) v = *reinterpret_cast<const f32x4*>(out + i) + v;
      *reinterpret_cast<f32x4*>(out + i) = v;
    }
  }
}

// Tile of a product, and in how many parts its summed axis is taken. The tiles' count is
// bounded from the sizes alone (the groups' sizes are on the device): one part tile per group
// that can have rows.
struct Plan {
  int bm;
  int splits;           // NN, NT: parts of every sum
  int64_t part_rows;    // TN: rows of a part, 0: no parts
  int64_t part_sums;    // TN: the most part sums there can be
};
int64_t tiles_of(const MatmulArgs& a, int bm, int bn) {
  const int64_t nt = (a.N + bn - 1) / bn;
  if (a.form == MOE_MATMUL_TN) return a.E * ((a.K + bm - 1) / bm) * nt;
  return (a.R / bm + (a.R < a.E ? a.R : a.E)) * nt;
}
Plan plan_of(const MatmulArgs& a) {
  const bool tn = a.form == MOE_MATMUL_TN;
  Plan p{128, 1, 0, 0};
  // 32 rows: a row tile's other rows are work for nothing, or there are too few 128-row tiles
  // to fill the chip (us with 128 rows -> 32: fp32, 512 rows of 8 groups, K 128, 12.9 -> 7.3;
  // bf16, 300 rows of 4 groups, K 512, N 1024, 8.3 -> 6.7; 8 rows a group, 64 groups, K 2048,
  // N 1408, 67.9 -> 63.4; 64 rows a group, 20.5 with 32 against 15.8).
  const int64_t groups = a.R < a.E ? a.R : a.E;
  if (!tn && (a.R <= 32 * (int64_t)a.E || tiles_of(a, 128, 128) < 128)) p.bm = 32;
  // The rows of the longest group, as the host has to guess them: a skewed router gives it
  // about sqrt(E) times the mean (2.6 to 3.7 times of 8 groups, 5.6 to 10 of 64).
  const int64_t longest = (int64_t)((double)a.R / sqrt((double)a.E));
  // 256 rows: half the traffic through L2 of 128 rows, but one workgroup per CU. They pay once
  // the 128-row tiles (half of one lost per group) are more than are resident at once (us with
  // 128 -> 256 rows, 8192 rows of 8 groups, K 4096: N 4096 381 -> 292, N 1024 109 -> 79, N 512
  // 66 against 75); in NN and NT if the sum is long too (N 4096: K 1024 82 against 90, K 2048
  // 159 -> 151) and a group has rows enough (64 groups, K 2048, N 4096: 128 rows each 372 ->
  // 251, 64 rows 223 against 242); in TN, whose tiles have their group's rows' work, if a CU has
  // tiles enough to even out a long group (8192 rows of 8, even groups / one with 2.6 / with
  // 3.7 times the mean's rows: 1024 x 4096 97 -> 84, 97 -> 90, 95 against 105; 1024 x 2048 53
  // -> 51, 50 against 70, 58 against 90; 32764 rows of 64, 2048 x 1408 317 -> 294).
  const int64_t rows128 = a.R / 128 + groups / 2;
  const int64_t tiles128 = tn ? tiles_of(a, 128, 128) : rows128 * ((a.N + 127) / 128);
  const bool enough = tn ? a.R * (tiles_of(a, 256, 256) / a.E) / kCus * 3 / 2 >= longest
                         : a.K > 1024 && a.R >= 128 * (int64_t)a.E;
  if (p.bm == 128 && a.bf16_in && tiles128 > 2 * kCus && enough) p.bm = 256;
  if (p.bm == 256) return p;
  if (tn) {
    // So a group that has most of the rows keeps a few CUs busy long after the others: its sums
    // are taken in parts of little more than a CU's share of the rows, where a part stays long
    // enough to be worth its 64 KB of partial sums and the second launch. The device counts the
    // parts; the host leaves them out where the longest group should have none. 128-row tiles, us
    // without parts -> with, for even groups and one with 3.7 times the mean's rows: 32768 rows of
    // 8, 512 x 512 51 -> 42 and 155 -> 42; 512 x 1024 63 -> 54 and 156 -> 57; 1024 x 1024 88 -> 82
    // and 156 -> 97; 8192 rows of 8, 512 x 1024 21 -> 22 and 47 -> 26; fp32, 512 x 512 54 -> 53 and
    // 142 -> 60, 1024 x 1024 151 -> 147 and 277 -> 166. 16384 rows of one group, 104 x 200: 164 ->
    // 21. Left whole: bf16, 8192 rows, 1024 x 1024 (28 against 31 even, 36 against 41 with 2.6
    // times the mean's, 45 against 39 with 3.7).
    const int64_t tiles = tiles_of(a, 128, 128), share = a.R * (tiles / a.E) / kCus;
    const int bk = a.bf16_in ? 32 : 16;
    const int64_t least = (a.bf16_in ? 24 : 8) * bk, few = (a.bf16_in ? 80 : 40) * bk;
    int64_t rows = share + share / 4 < few ? share + share / 4 : few;
    // fp32, bound by the matrix units: all items (half a part more per group) are one round of
    // two workgroups per CU (us, against the bf16 rule: 32768 rows of 8 groups, 512 x 512 218 ->
    // 168; 20000 rows of one, 1024 x 512 277 -> 183; bf16, 32768 rows of 4, 512 x 1408 73 against 92).
    const int64_t round = a.bf16_in          ? share * 4 / 5
                          : tiles < 2 * kCus ? share * 2 * kCus / (4 * kCus - tiles)
                                             : share;
    if (rows < round) rows = round;
    if (rows < least) rows = least;
    if (longest <= rows || (a.bf16_in && tiles > kCus && share < 128 * bk)) return p;
    p.part_rows = rows;
    p.part_sums = a.R / rows + (groups < a.R / rows ? groups : a.R / rows);
    return p;
  }
  // NN, NT, few tiles and a long sum: parts of at least 16 stages, about one workgroup per CU.
  // 65 to 128 tiles are few where the matrix units are the bound (fp32, 16 rows, K 1024, N 2048:
  // 21.7 -> 17.0 us) or the sum is very long (NT, 4 rows, N 4096: K 14336 103 -> 82, K 10240 75
  // -> 57; K 4096 22.0 against 24.9). One row of 8 groups, K 14336, N 4096: 46 -> 38.
  const int64_t tiles = tiles_of(a, p.bm, 128);
  const int64_t stages = a.K / (p.bm == 32 ? (a.bf16_in ? 64 : 32) : (a.bf16_in ? 32 : 16));
  if (tiles <= (a.bf16_in && stages < 160 ? 64 : 128) && stages >= 32) {
    int64_t n = kCus / tiles;
    n = n < stages / 16 ? n : stages / 16;
    p.splits = (int)(n < 16 ? n : 16);
  }
  return p;
}

template <class G, typename TO>
hipError_t launch_tile(const MatmulArgs& a, hipStream_t s) {
  // at most as many workgroups as are resident together, a multiple of the XCDs
  constexpr int64_t resident = kCus * (G::BM == 256 ? 1 : 2);
  const int64_t tiles = tiles_of(a, G::BM, G::BN);
  const int64_t items = G::TN ? tiles + tiles / a.E * a.part_sums : tiles * a.splits;
  const int64_t blocks = (items + kXcds - 1) / kXcds * kXcds;
  const unsigned grid = (unsigned)(blocks < resident ? blocks : resident);
  if constexpr (sizeof(TO) == 4) {
    if (a.accumulate) {
      grouped_matmul_kernel<G, TO, true><<<grid, 256, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  grouped_matmul_kernel<G, TO, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

// Weights that are read once and do not fit the last-level cache: 32-row tiles, of the groups
// that R rows spread over E evenly leave with a row or more (us: NT, 16 rows of 8 groups, K 14336,
// N 4096, 147 -> 136; NN, 128 rows, K 4096, N 14336, 183 -> 164; what fits is better kept: NN, 2
// rows, 36 against 40).
template <typename T>
bool streams(const MatmulArgs& a) {
  constexpr double kLastLevel = 256e6;
  const double active = a.E * (1.0 - exp(-(double)a.R / a.E));
  return a.R <= 32 * (int64_t)a.E && active * (double)a.K * (double)a.N * sizeof(T) > kLastLevel;
}

template <typename T, int FORM, typename TO>
hipError_t launch_form(const MatmulArgs& a, int bm, hipStream_t s) {
  constexpr int BK = 64 / sizeof(T);  // 64 bytes
  if constexpr (FORM != MOE_MATMUL_TN) {
    if (bm == 32 && streams<T>(a)) return launch_tile<Geo<T, FORM, 32, 128, 2 * BK, 1, true>, TO>(a, s);
    if (bm == 32) return launch_tile<Geo<T, FORM, 32, 128, 2 * BK, 1>, TO>(a, s);
  }
  if constexpr (sizeof(T) == 2) {
    if (bm == 256) return launch_tile<Geo<T, FORM, 256, 256, BK, 2>, TO>(a, s);
  }
  return launch_tile<Geo<T, FORM, 128, 128, BK, 2>, TO>(a, s);
}

template <typename T, typename TO>
hipError_t launch_forms(const MatmulArgs& a, int bm, hipStream_t s) {
  if (a.form == MOE_MATMUL_NN) return launch_form<T, MOE_MATMUL_NN, TO>(a, bm, s);
  if (a.form == MOE_MATMUL_NT) return launch_form<T, MOE_MATMUL_NT, TO>(a, bm, s);
  return launch_form<T, MOE_MATMUL_TN, TO>(a, bm, s);
}

hipError_t launch_types(const MatmulArgs& a, int bm, hipStream_t s) {
  if (!a.bf16_in) return launch_forms<float, float>(a, bm, s);
  return a.bf16_out ? launch_forms<bf16, bf16>(a, bm, s) : launch_forms<bf16, float>(a, bm, s);
}

// Values of one part sum.
int64_t part_values(const MatmulArgs& a) { return (a.form == MOE_MATMUL_TN ? a.K : a.R) * a.N; }

}  // namespace

size_t grouped_matmul_workspace(const MatmulArgs& a) {
  const Plan p = plan_of(a);
  const int64_t sums = a.form == MOE_MATMUL_TN ? p.part_sums : p.splits > 1 ? p.splits : 0;
  return (size_t)sums * part_values(a) * sizeof(float);
}

hipError_t launch_grouped_matmul(const MatmulArgs& args, float* ws, hipStream_t s) {
  MatmulArgs a = args;
  const Plan p = plan_of(a);
  const bool tn = a.form == MOE_MATMUL_TN;
  a.splits = p.splits;
  a.split_stride = part_values(a);
  a.part_rows = p.part_rows;
  a.part_sums = p.part_sums;
  a.parts = ws;
  if (p.splits == 1 && !p.part_rows) return launch_types(a, p.bm, s);
  MatmulArgs part = a;
  if (!tn) {  // every sum is in parts
    part.out = ws;
    part.bf16_out = part.accumulate = 0;
  }
  const hipError_t e = launch_types(part, p.bm, s);
  if (e != hipSuccess) return e;
  // (TN: few workgroups per group, of which most leave at once where most groups are whole)
  const int64_t blocks = (a.split_stride / 4 + 255) / 256, most = 2048 / a.E;
  const dim3 grid(capped_grid(tn && blocks > most ? most : blocks), tn ? a.E : 1);
  if (a.bf16_out) join_parts_kernel<bf16><<<grid, 256, 0, s>>>(a, ws);
  else join_parts_kernel<float><<<grid, 256, 0, s>>>(a, ws);
  return hipGetLastError();
}

// What the tiles of the matrix products share: waits, and one operand's stage in LDS.
#pragma once

#include "common.h"

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kStages = 4;    // LDS ring

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkmcnt0() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
}
__device__ __forceinline__ void sync_point() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// The value, hidden from the compiler: what depends on it is computed where it is used, and
// not kept in registers (which the 256-row tiles do not have) from before the tile loop.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

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

}  // namespace

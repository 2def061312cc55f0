// Helpers of the training operators' kernels.
#pragma once

#include "common.h"

// 16 bytes of a row.
template <typename TI>
struct Chunk;
template <>
struct Chunk<bf16> {
  static constexpr int N = 8;
  typedef bf16x8 vec;
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  typedef f32x4 vec;
};

// Workgroups of a launch that covers n items in strides of its grid: a grid's work-items
// (256 threads per workgroup here) have to stay below 2^32, so that a row count may not
// become a grid size unchecked.
constexpr int64_t kMaxGrid = int64_t(1) << 20;
inline unsigned capped_grid(int64_t n) { return (unsigned)(n < kMaxGrid ? n : kMaxGrid); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Group bounds as every training operator takes them: bound e is the largest of 0 and
// offsets[0 .. e], and at most R, so that no table moves a row out of [0, R). Lane e < E of
// the calling wave (all 64 lanes active, E <= 64) gets group e's [start, end); lanes past E
// get empty groups at the last bound. Returns the last bound.
__device__ __forceinline__ int group_bounds(const int32_t* __restrict__ offsets, int E, int R,
                                            int& start, int& end) {
  const int lane = threadIdx.x & 63;
  int m = max(0, offsets[lane < E ? lane : E]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(m, o);
    if (lane >= o) m = max(m, v);
  }
  start = min(m, R);
  const int next = __shfl_down(start, 1);
  const int last = min(max(__shfl(m, E - 1), offsets[E]), R);
  end = lane >= E - 1 ? last : next;
  if (lane >= E) start = last;
  return last;
}

// w4a16_lanes.h -- a wave's lanes together: order-preserving keys, maxima and sums
// over the wave, and the choice of a token's experts from them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace w4a16_internal {

constexpr int kRtMaxExperts = 1024;

// Order-preserving bits: a < b as numbers iff key(a) < key(b) as unsigned.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double f) {
  const uint64_t b = __builtin_bit_cast(uint64_t, f);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// The number a key stands for.
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __builtin_bit_cast(double, k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}

// v of another lane: CTRL as in dpp_f32, for any 4- or 8-byte type; 0 where the
// pattern does not reach (ROWS: the rows written).
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_of(T v) {
  if constexpr (sizeof(T) == 4) {
    const int b = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, b, CTRL, ROWS, 0xF, false));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
  }
}

// v of lane `src` (uniform) in every lane.
template <typename T>
__device__ __forceinline__ T lane_of(T v, int src) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), src));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), src);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), src);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
  }
}

// Maximum over the wave, in every lane: within quads, half rows and rows of 16
// lanes, then from row to row into lane 63. A lane a step does not reach meets
// 0, so keys only.
template <typename T>
__device__ __forceinline__ T wave_max_of(T v) {
  auto step = [](T a, T b) { return b > a ? b : a; };
  v = step(v, dpp_of<0xB1, 0xF>(v));
  v = step(v, dpp_of<0x4E, 0xF>(v));
  v = step(v, dpp_of<0x141, 0xF>(v));
  v = step(v, dpp_of<0x140, 0xF>(v));
  v = step(v, dpp_of<0x142, 0xA>(v));  // row_bcast 15: rows 1 and 3
  v = step(v, dpp_of<0x143, 0xC>(v));  // row_bcast 31: rows 2 and 3
  return lane_of(v, 63);
}
// Sum over the wave, in every lane, in the order of wave_max_of.
template <typename T>
__device__ __forceinline__ T wave_sum_of(T v) {
  v += dpp_of<0xB1, 0xF>(v);
  v += dpp_of<0x4E, 0xF>(v);
  v += dpp_of<0x141, 0xF>(v);
  v += dpp_of<0x140, 0xF>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// The i-th expert of a lane. Choice by value takes consecutive ones, so that
// groups are whole lanes; choice by logit takes every 64th, so that the order
// of (i, lane) is that of the experts and equal keys need no second look.
template <int P, bool WIDE>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return WIDE ? lane * P + i : i * 64 + lane;
}

// The top_k largest keys (0: never), one after the other, the lowest expert of
// equal ones first: lane j gets the j-th choice, -1 where nothing is left.
template <int P, bool WIDE, typename Key>
__device__ __forceinline__ int take(Key (&key)[P], int top_k, int lane) {
  int id = -1;
  for (int j = 0; j < top_k; ++j) {
    Key best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < P; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    const Key top = wave_max_of(best);
    if (top == 0) break;
    const uint32_t back = best == top ? kRtMaxExperts - expert_of<P, WIDE>(lane, bi) : 0;
    const int e = kRtMaxExperts - static_cast<int>(wave_max_of(back));
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (expert_of<P, WIDE>(lane, i) == e) key[i] = 0;
  }
  return id;
}

}  // namespace w4a16_internal

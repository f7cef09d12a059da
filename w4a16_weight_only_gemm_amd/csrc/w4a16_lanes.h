// w4a16_lanes.h -- a wave's lanes together: order-preserving keys, maxima and sums
// over the wave.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace w4a16_internal {

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

}  // namespace w4a16_internal

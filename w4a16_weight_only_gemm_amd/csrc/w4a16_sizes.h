// w4a16_sizes.h -- sizes that kernels form in 32 bits, without HIP, so that a host
// test can hold them to 64-bit arithmetic.
#pragma once

#include <cstdint>

namespace w4a16_internal {

// Bytes of a packed matrix of `blocks` column blocks (16 columns of K codes, half a
// byte each), below 4 GB. Halved before it is multiplied: N x K is past 2^32 from 2 GiB on.
constexpr uint32_t packed_matrix_bytes(int blocks, int K) {
  return static_cast<uint32_t>(blocks) * 8u * static_cast<uint32_t>(K);
}

// The g-th group of a wave's unit u of `per` groups, the last one again where K ends inside
// the unit: what a scalar offset past the end of a buffer reads is not the range check's to
// decide.
constexpr int unit_group(int u, int per, int g, int groups) {
  return u * per + g < groups ? u * per + g : groups - 1;
}

}  // namespace w4a16_internal

// w4a16_layer_launch.h -- internal interface of the operators between a layer's
// products (public side: include/w4a16_layer.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/w4a16_layer.h"
#include "w4a16_epilogue.h"
#include "w4a16_launch.h"

namespace w4a16_internal {

// Checked by the caller: a shape w4a16_gemm runs, for gated activations N % 32
// == 0. hipErrorNotSupported: a grid of more than 2^32 threads.
hipError_t launch_epilogue(const GemmArgs& a, const Epilogue& ep, hipStream_t stream);

// Checked by the caller: the header's ranges.
hipError_t launch_norm(const w4a16_norm_args& a, int T, int N, hipStream_t stream);

// ---- a mixture-of-experts layer for a few tokens (w4a16_moe_layer.hip) ----
struct MoeLayerArgs {
  w4a16_moe_layer_args layer;
  const uint16_t* x;    // bf16 [T][H]
  const int* live;      // [T] or null
  const uint16_t* base; // bf16 [T][H] or null
  uint16_t* out;        // bf16 [T][H]
  int* ids;             // [T][top_k]
  float* weights;       // [T][top_k]
  char* workspace;
  int T;
};
size_t moe_layer_workspace_bytes(int T, int E, int top_k, int H, int I);
// Checked by the caller: 1 <= T <= W4A16_MOE_LAYER_MAX_TOKENS and the header's
// ranges.
hipError_t launch_moe_layer(const MoeLayerArgs& a, hipStream_t stream);

}  // namespace w4a16_internal

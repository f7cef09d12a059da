// w4a16_moe_launch.h -- internal interface of the mixture-of-experts and W8A8
// kernels (public side: include/w4a16_moe.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace w4a16_internal {

// ---- routing (w4a16_moe.hip) ----
struct RouteArgs {
  const void* logits;  // f32 or bf16 [T][E]
  const float* bias;   // [E] or null
  int* ids;            // [T][top_k]
  float* weights;      // [T][top_k]
  int* offsets;        // [E + 1]
  int* rows;           // [T * top_k]
  void* workspace;
  uint8_t* counts;     // workspace: [chunks][E rounded up to 4] slots per expert
  int* sums;           // workspace: [chunks + 1][E] of the chunks before
  int T, E, top_k;
  int sigmoid, bf16, groups, groups_kept, group_top, renormalize;
  float scale;
  // filled in by launch_route
  int per;             // experts per group
  uint32_t per_inverse;  // floor(e / per) = high half of e * per_inverse
  int group_lanes;     // lanes that look at a group, a power of two
  int group_whole;     // a group's experts are exactly those its lanes hold
  int chunk;           // tokens per workgroup
  int chunks;
};
// Workspace of T tokens (0: the one-launch form runs).
size_t route_workspace_bytes(int T, int E);
// Checked by the caller: T >= 0 and the fields' ranges.
hipError_t launch_route(RouteArgs a, hipStream_t stream);

// ---- weighted sum back into token order (w4a16_moe.hip) ----
struct CombineArgs {
  const uint16_t* y;     // bf16 [T * top_k][N]
  const int* ids;        // [T][top_k]
  const float* weights;  // [T][top_k]
  const uint16_t* base;  // bf16 [T][N] or null
  uint16_t* out;         // bf16 [T][N]
  int T, top_k, N;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);

// ---- experts' products (w4a16_experts.hip) ----
struct ExpertsArgs {
  const uint16_t* x;        // bf16 [ceil(slots / x_div)][K]
  const uint32_t* qweight;  // experts' packed weights, one after another
  const uint16_t* scales;
  uint16_t* y;              // bf16 [slots][N], or [slots][N / 2] with SwiGLU
  const int* rows;          // [slots]
  const int* offsets;       // [E + 1]
  int slots, E, x_div, N, K, group, swiglu;
};
// Checked by the caller: slots >= 1, shapes as the header says, x and one
// expert's weights below 4 GB.
hipError_t launch_experts(const ExpertsArgs& a, hipStream_t stream);

// ---- W8A8 (w8a8.hip) ----
struct W8A8Args {
  const uint8_t* xq;       // int8 codes [M][K], 16-blocks in MFMA step order
  const float* sx;         // [M]
  const uint8_t* qweight;  // [ceil(N/16)][ceil(K/64)][64][16]
  const float* sw;         // [N]
  uint16_t* y;             // bf16 [M][N]
  int M, N, K;
};
hipError_t launch_w8a8(const W8A8Args& a, hipStream_t stream);

}  // namespace w4a16_internal

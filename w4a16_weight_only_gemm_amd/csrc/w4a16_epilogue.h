// w4a16_epilogue.h -- what w4a16_gemm_epilogue does to a finished fp32 sum: bias,
// activation, scale, residual.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/w4a16_layer.h"
#include "w4a16_device.h"

namespace w4a16_internal {

struct Epilogue {
  const uint16_t* bias;      // bf16 [N] or null
  const uint16_t* residual;  // bf16 [M][columns of y] or null; may be y
  float scale;
  int act;  // W4A16_ACT_*
};

// Kinds of kernel: sums as they are, one value per sum, one per pair of sums.
constexpr int kEpiNone = 0, kEpiPlain = 1, kEpiGated = 2;

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t b) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16);
}

__device__ __forceinline__ float silu(float v) { return v / (1.f + __expf(-v)); }

// (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)): no cancellation for u far below 0.
__device__ __forceinline__ float gelu_tanh(float v) {
  const float u = 0.7978845608028654f * __builtin_fmaf(0.044715f * v * v, v, v);
  return v / (1.f + __expf(-2.f * u));
}

// (1 + erf(v / sqrt 2)) / 2 = erfc(-v / sqrt 2) / 2, for the same reason.
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * erfcf(-0.7071067811865476f * v); }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {  // the same for every thread
    case W4A16_ACT_SILU: return silu(v);
    case W4A16_ACT_GELU: return gelu(v);
    case W4A16_ACT_GELU_TANH: return gelu_tanh(v);
    case W4A16_ACT_RELU: return v < 0.f ? 0.f : v;
    default: return v;
  }
}

__device__ __forceinline__ float with_bias(const Epilogue& ep, float v, int column) {
  return ep.bias ? v + bf16_bits_to_f32(to_global(ep.bias)[column]) : v;
}

// The activated value of column n's sum, not yet scaled.
__device__ __forceinline__ float epilogue_value(const Epilogue& ep, float v, int n) {
  return activate(with_bias(ep, v, n), ep.act);
}

// The same of the gate's and the up's sum of column n; ups start at column n_out.
__device__ __forceinline__ float epilogue_gated(const Epilogue& ep, float gate, float up, int n,
                                                int n_out) {
  gate = with_bias(ep, gate, n);
  up = with_bias(ep, up, n_out + n);
  return (ep.act == W4A16_ACT_SWIGLU ? silu(gate) : gelu_tanh(gate)) * up;
}

// Scaled and added to the residual, whose element is at `at`.
__device__ __forceinline__ float epilogue_residual(const Epilogue& ep, float v, size_t at) {
  if (!ep.residual) return ep.scale * v;
  return __builtin_fmaf(ep.scale, v, bf16_bits_to_f32(to_global(ep.residual)[at]));
}

}  // namespace w4a16_internal

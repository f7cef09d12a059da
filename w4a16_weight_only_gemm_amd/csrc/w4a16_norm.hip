// w4a16_norm.hip -- the norms behind and before a block with its gate, its scale
// and the residual sum between them (w4a16_norm).
//
//     u = post(y),  r = residual + scale * gate * u,  v = norm(r)
//
// Every row is read once into registers, eight columns to a 16-byte piece, and
// stays there in fp32 through both norms; the means are taken of the registers (of
// the deviations from the mean, in a second pass over them, for layer norms), and
// r and v are rounded once, on their way out. A row belongs to 16, 32 or 64 lanes
// of a wave (DPP sums, no LDS) or to the waves of a workgroup (one barrier a sum).
// What bounds it: HBM for many rows; for few, the launch and the chain of a load,
// the sums and a store.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "w4a16_device.h"
#include "w4a16_epilogue.h"
#include "w4a16_layer_launch.h"

namespace w4a16_internal {
namespace {

constexpr int kNormMaxWaves = 16;

struct NormArgs {
  w4a16_norm_args a;
  int T, N;
};

struct Piece {
  float v[8];
};

__device__ __forceinline__ Piece bf16_piece(u32x4 d) {
  Piece p;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = d[j / 2];
    p.v[j] = __builtin_bit_cast(float, j % 2 ? w & 0xFFFF0000u : w << 16);
  }
  return p;
}

__device__ __forceinline__ u32x4 to_bf16(const Piece& p) {
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = f32_to_bf16_bits(p.v[2 * j]) | static_cast<uint32_t>(f32_to_bf16_bits(p.v[2 * j + 1])) << 16;
  return o;
}

// Eight floats of a row, or the first `left` of them, from any address of a float.
typedef float f32_quad __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ Piece load_f32(gptr<const float> x, int left) {
  Piece p;
  if (left >= 8) {
    const f32x4 lo = *reinterpret_cast<gptr<const f32_quad>>(x);
    const f32x4 hi = *reinterpret_cast<gptr<const f32_quad>>(x + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) p.v[j] = j < 4 ? lo[j % 4] : hi[j % 4];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p.v[j] = j < left ? x[j] : 0.f;
  }
  return p;
}
__device__ __forceinline__ void store_f32(gptr<float> x, const Piece& p, int left) {
  if (left >= 8) {
    *reinterpret_cast<gptr<f32_quad>>(x) = f32x4{p.v[0], p.v[1], p.v[2], p.v[3]};
    *reinterpret_cast<gptr<f32_quad>>(x + 4) = f32x4{p.v[4], p.v[5], p.v[6], p.v[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < left) x[j] = p.v[j];
  }
}

// Joins a value over the L lanes of a row within a wave, in every one of them: a
// butterfly whose steps add (or compare) two values in either order, so all get the
// same bits.
template <int L, typename F>
__device__ __forceinline__ float lanes_join(float v, F f) {
  v = f(v, dpp_f32<0xB1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp_f32<0x4E>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp_f32<0x141>(v));  // row_half_mirror
  v = f(v, dpp_f32<0x140>(v));  // row_mirror
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16));
  if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}

// The same over a whole row. BLOCK: of the workgroup's waves, in the order of the
// waves; consecutive calls use the two halves of `parts` in turn, so one barrier a
// call is enough.
template <int L, bool BLOCK>
struct RowJoin {
  float* parts;  // [2][kNormMaxWaves]
  int waves, turn;
  template <typename F>
  __device__ __forceinline__ float operator()(float v, F f) {
    v = lanes_join<L>(v, f);
    if constexpr (BLOCK) {
      float* p = parts + turn * kNormMaxWaves;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
      __syncthreads();
      v = p[0];
      for (int w = 1; w < waves; ++w) v = f(v, p[w]);
    }
    return v;
  }
};

// P: pieces per thread. A row's pieces go round its threads, so that a wave's loads
// are contiguous.
template <int P, int L, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 64 * kNormMaxWaves : 256) void norm_kernel(const NormArgs args) {
  const w4a16_norm_args& a = args.a;
  const int N = args.N;
  __shared__ float parts[2 * kNormMaxWaves];
  RowJoin<L, BLOCK> join{parts, static_cast<int>(blockDim.x) / 64, 0};
  auto sum = [&](float v) { return join(v, [](float x, float y) { return x + y; }); };
  const int per = BLOCK ? static_cast<int>(blockDim.x) : L;  // threads of a row
  const int mine = BLOCK ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % L;
  const long long row = BLOCK ? static_cast<long long>(blockIdx.x)
                              : static_cast<long long>(blockIdx.x) * (256 / L) + threadIdx.x / L;
  if (!BLOCK && row >= args.T) return;  // whole rows of lanes; no barrier follows
  const float n = static_cast<float>(N);  // sums are divided: a constant row's mean is its value
  const bool layer = a.kind == W4A16_NORM_LAYER;
  const float one = a.unit_offset ? 1.f : 0.f;
  auto left_of = [&](int p) { return N - 8 * (mine + p * per); };
  auto at_of = [&](int p) { return 8 * (mine + p * per); };
  auto vector = [&](const void* ptr, int p) {  // bf16 [N]
    return bf16_piece(load_piece(to_global(static_cast<const uint16_t*>(ptr)) + at_of(p), left_of(p)));
  };
  auto bf16_row = [&](const void* ptr, long long r, int p) {
    return bf16_piece(load_piece(to_global(static_cast<const uint16_t*>(ptr)) + r * N + at_of(p), left_of(p)));
  };

  Piece v[P];
  // (v - mean) / sqrt(mean square + eps) * weight + bias, in place; columns past N
  // hold zeros and stay out of the sums
  auto normalise = [&](const void* weight, const void* bias) {
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[p].v[j];
      const float mean = sum(s) / n;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[p].v[j] = j < left_of(p) ? v[p].v[j] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fmaf(v[p].v[j], v[p].v[j], s);
    const float r = 1.f / sqrtf(sum(s) / n + a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (left_of(p) <= 0) continue;
      Piece w, b;
      if (weight) w = vector(weight, p);
      if (bias) b = vector(bias, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x = v[p].v[j] * r;
        if (weight) x *= w.v[j] + one;
        if (bias) x += j < left_of(p) ? b.v[j] : 0.f;
        v[p].v[j] = x;
      }
    }
  };

#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (left_of(p) > 0 && a.y) {
      v[p] = bf16_row(a.y, row, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p].v[j] = 0.f;
    }
  }
  if (a.y) {
    if (a.post_norm) normalise(a.post_weight, a.post_bias);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (left_of(p) <= 0) continue;
      if (a.gate) {
        const Piece g = bf16_row(a.gate, row / a.gate_rows, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[p].v[j] *= g.v[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p].v[j] *= a.scale;
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (left_of(p) <= 0) continue;
    const size_t at = static_cast<size_t>(row) * N + at_of(p);
    const bool wide = a.residual_type == W4A16_RESIDUAL_F32;
    if (a.residual) {
      const Piece r = wide ? load_f32(to_global(static_cast<const float*>(a.residual)) + at, left_of(p))
                           : bf16_row(a.residual, row, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p].v[j] += r.v[j];
    }
    if (a.residual_out) {
      if (wide)
        store_f32(to_global(static_cast<float*>(a.residual_out)) + at, v[p], left_of(p));
      else
        store_piece(to_global(static_cast<uint16_t*>(a.residual_out)) + at, to_bf16(v[p]), left_of(p));
    }
  }
  if (!a.x && !a.xq) return;
  normalise(a.weight, a.bias);
  if (a.x) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (left_of(p) > 0)
        store_piece(to_global(static_cast<uint16_t*>(a.x)) + static_cast<size_t>(row) * N + at_of(p),
                    to_bf16(v[p]), left_of(p));
    return;
  }
  // The codes and scale of w4a8_quantize, of values that were not rounded before.
  float big = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(v[p].v[j]));
  big = join(big, [](float x, float y) { return fmaxf(x, y); });
  const float inv = big > 0.f ? 127.f / big : 0.f;
  if (mine == 0) to_global(a.sx)[row] = big / 127.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (left_of(p) <= 0) continue;
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float q = __builtin_rintf(v[p].v[j] * inv);
      q = q > 127.f ? 127.f : q;
      q = q < -127.f ? -127.f : q;
      c[j] = static_cast<uint32_t>(static_cast<int>(q)) & 0xFFu;
    }
    // half a 16-block: byte j holds offset 0,4,1,5,2,6,3,7
    const u32x2 o = {c[0] | c[4] << 8 | c[1] << 16 | c[5] << 24, c[2] | c[6] << 8 | c[3] << 16 | c[7] << 24};
    *reinterpret_cast<gptr<u32x2>>(to_global(static_cast<uint8_t*>(a.xq)) + static_cast<size_t>(row) * N +
                                   at_of(p)) = o;
  }
}

template <int P, int L, bool BLOCK>
hipError_t launch_norm_t(const NormArgs& args, int threads, hipStream_t stream) {
  const long long blocks = BLOCK ? args.T : (static_cast<long long>(args.T) + 256 / L - 1) / (256 / L);
  if (blocks * threads > 0xFFFFFFFFLL) return hipErrorNotSupported;
  NormArgs copy = args;
  void* kargs[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(&norm_kernel<P, L, BLOCK>),
                         dim3(static_cast<unsigned>(blocks)), dim3(threads), kargs, 0, stream);
}

template <int P>
hipError_t launch_norm_block(const NormArgs& args, int pieces, hipStream_t stream) {
  const int waves = (pieces + 64 * P - 1) / (64 * P);
  return launch_norm_t<P, 64, true>(args, 64 * waves, stream);
}

}  // namespace

hipError_t launch_norm(const w4a16_norm_args& a, int T, int N, hipStream_t stream) {
  const NormArgs args = {a, T, N};
  const int pieces = (N + 7) / 8;
  if (pieces <= 16) return launch_norm_t<1, 16, false>(args, 256, stream);
  if (pieces <= 32) return launch_norm_t<1, 32, false>(args, 256, stream);
  if (pieces <= 64) return launch_norm_t<1, 64, false>(args, 256, stream);
  if (pieces <= 64 * kNormMaxWaves) return launch_norm_block<1>(args, pieces, stream);
  if (pieces <= 2 * 64 * kNormMaxWaves) return launch_norm_block<2>(args, pieces, stream);
  if (pieces <= 4 * 64 * kNormMaxWaves) return launch_norm_block<4>(args, pieces, stream);
  return launch_norm_block<8>(args, pieces, stream);
}

}  // namespace w4a16_internal

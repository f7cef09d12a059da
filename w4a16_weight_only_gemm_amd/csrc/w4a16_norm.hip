// w4a16_norm.hip -- the norms behind and before a block with its gate, its scale
// and the residual sum between them (w4a16_norm).
//
//     u = post(y),  r = residual + scale * gate * u,  v = norm(r)
//
// Every row is read once into registers, eight columns to a 16-byte piece, and
// stays there in fp32 through both norms; the means are taken of the registers (of
// the deviations from the mean, in a second pass over them, for layer norms; after
// two more where the mean's rounding counts among them), and r and v are rounded
// once, on their way out. A row belongs to 16, 32 or 64 lanes of a wave (DPP sums, no
// LDS) or to the waves of a workgroup (one barrier a sum).
// What bounds it: HBM for many long rows (4095 of 5120, fp32 residual: 52.4 us, 252 MB);
// otherwise the launch and a chain of loads, sums and a store: every operand's pieces are
// asked for behind its own condition and waited for one after the other, 14 such waits in
// the form of 2048 rows of 2741 with gate and layer norms on both sides (17 us).
#include <hip/hip_runtime.h>

#include <cfloat>
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

// Where a thread's p-th piece of a row lies. The last piece of a row whose length is no
// multiple of 8 is read as the row's last 8 columns and moved down by those that are not
// its own, so that no load is a loop over columns.
struct Span {
  int at;     // first column read
  int shift;  // columns read in front of the piece
  int left;   // columns of the piece, 8 and more: all; 0 and less: there is none
};

__device__ __forceinline__ u32x4 moved_down(u32x4 v, int shift) {
  if (shift & 4) v = u32x4{v[2], v[3], 0u, 0u};
  if (shift & 2) v = u32x4{v[1], v[2], v[3], 0u};
  if (shift & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return v;
}

// A piece as loaded, zeros where there is none. Unaligned addresses as in store_piece.
typedef uint32_t half_piece __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32_quad __attribute__((ext_vector_type(4), aligned(4)));
template <bool TAIL>
__device__ __forceinline__ u32x4 load_bf16(gptr<const uint16_t> row, const Span& s) {
  u32x4 v = *reinterpret_cast<gptr<const half_piece>>(row + s.at);
  if constexpr (TAIL) v = moved_down(v, s.shift);
  if (s.left <= 0) v = u32x4{0u, 0u, 0u, 0u};
  return v;
}
template <bool TAIL>
__device__ __forceinline__ Piece load_f32(gptr<const float> row, const Span& s) {
  const f32x4 lo = *reinterpret_cast<gptr<const f32_quad>>(row + s.at);
  const f32x4 hi = *reinterpret_cast<gptr<const f32_quad>>(row + s.at + 4);
  Piece p;
#pragma unroll
  for (int j = 0; j < 8; ++j) p.v[j] = j < 4 ? lo[j % 4] : hi[j % 4];
  if constexpr (TAIL) {
#pragma unroll
    for (int by = 4; by; by /= 2)
      if (s.shift & by) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p.v[j] = j + by < 8 ? p.v[j + by] : 0.f;
      }
  }
  if (s.left <= 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p.v[j] = 0.f;
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
// are contiguous. TAIL: N is no multiple of 8 (and at least 8).
// Only y is asked for in front of the first sum. Asking for everything there costs
// registers, and waves that would hide the waits more cheaply: 2048 rows of 2741, layer
// norms on both sides and a gate 22.1 against 17.3 us (two pieces a thread; one piece,
// which needs 33 to 39 registers, and loads together within a step were not tried).
template <int P, int L, bool BLOCK, bool TAIL>
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
  const float n = static_cast<float>(N);
  const bool layer = a.kind == W4A16_NORM_LAYER;
  const float one = a.unit_offset ? 1.f : 0.f;
  const bool wide = a.residual_type == W4A16_RESIDUAL_F32;
  Span span[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int at = 8 * (mine + p * per);
    span[p].at = min(at, N - 8);
    span[p].shift = min(at - span[p].at, 7);
    span[p].left = N - at;
  }
  auto bf16_row = [&](const void* ptr, long long r, int p) {
    return load_bf16<TAIL>(to_global(static_cast<const uint16_t*>(ptr)) + r * N, span[p]);
  };
  auto first_of = [&](int p) { return span[p].at + span[p].shift; };  // where there is a piece

  const u32x4 none = {0u, 0u, 0u, 0u};
  const bool next = a.x || a.xq;

  Piece v[P];
  // (v - mean) / sqrt(mean square + eps) * weight + bias, in place; columns past N
  // hold zeros and stay out of the sums
  auto mean_of = [&] {
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[p].v[j];
    return sum(s) / n;
  };
  auto mean_square = [&](float by) {
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[p].v[j] * by;
        s = __builtin_fmaf(x, x, s);
      }
    return sum(s) / n;
  };
  auto subtract = [&](float m) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      int left = span[p].left;
      // compared here: masks of all columns, made once for every use, fill the registers
      asm volatile("" : "+v"(left) : :);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p].v[j] = (TAIL ? j < left : left > 0) ? v[p].v[j] - m : 0.f;
    }
  };
  auto normalise = [&](const void* w, const void* b) {
    float mean = 0.f;
    if (layer) {
      mean = mean_of();
      // A sum past fp32 has a value of 2^112 or more. Either all are equal, or two are 2^88
      // or more apart and the mean square is past fp32: zeros both times, NaN for what is
      // not finite.
      if (!(fabsf(mean) <= FLT_MAX)) {
        mean = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[p].v[j] -= v[p].v[j];
      }
      subtract(mean);
    }
    float square = mean_square(1.f);
    // Rows for which that is not it, a condition that all threads of a row share. Loops, so
    // that they take no registers from the others.
    // The sum of a row rounds by up to some 90 half steps of its mean, which count among
    // deviations that are small against it: beyond 64 times their root mean square they
    // are taken from the fp32 number next to the mean, which is the value itself in a row
    // of equal ones, and then from their own mean.
    // Squares whose sum is past fp32 are summed again of numbers times 2^-96: one is 2^56
    // or more, so what that flushes to 0 does not count. A mean square that is past fp32
    // itself stays infinite and makes zeros, of a deviation past fp32 too.
    if (!(mean * mean * 0x1p-12f <= square && square <= FLT_MAX)) {
      if (layer) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[p].v[j] = fabsf(v[p].v[j]) > FLT_MAX ? copysignf(FLT_MAX, v[p].v[j]) : v[p].v[j];
#pragma unroll 1
        for (int round = 0; round < 2; ++round) {
          float m = mean_of();
          if (!(fabsf(m) <= FLT_MAX)) m = 0.f;  // so is the mean square then
          subtract(round == 0 ? (mean + m) - mean : m);
        }
      }
      float by = 1.f, back = 1.f;
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
        square = mean_square(by) * back * back;
        if (square <= FLT_MAX) break;
        by = 0x1p-96f;
        back = 0x1p96f;
      }
    }
    const float r = 1.f / sqrtf(square + a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const Piece wp = bf16_piece(w ? bf16_row(w, 0, p) : none), bp = bf16_piece(b ? bf16_row(b, 0, p) : none);
      if (span[p].left <= 0) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x = v[p].v[j] * r;
        if (w) x *= wp.v[j] + one;
        if (b) x += bp.v[j];  // 0 past N
        v[p].v[j] = x;
      }
    }
  };

#pragma unroll
  for (int p = 0; p < P; ++p) v[p] = bf16_piece(a.y ? bf16_row(a.y, row, p) : none);
  if (a.y) {
    if (a.post_norm) normalise(a.post_weight, a.post_bias);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const Piece g = bf16_piece(a.gate ? bf16_row(a.gate, row / a.gate_rows, p) : none);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p].v[j] = (a.gate ? v[p].v[j] * g.v[j] : v[p].v[j]) * a.scale;
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (a.residual) {
      const Piece res = wide ? load_f32<TAIL>(to_global(static_cast<const float*>(a.residual)) + row * N, span[p])
                             : bf16_piece(bf16_row(a.residual, row, p));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p].v[j] += res.v[j];
    }
    if (a.residual_out && span[p].left > 0) {
      const size_t at = static_cast<size_t>(row) * N + first_of(p);
      if (wide)
        store_f32(to_global(static_cast<float*>(a.residual_out)) + at, v[p], span[p].left);
      else
        store_piece(to_global(static_cast<uint16_t*>(a.residual_out)) + at, to_bf16(v[p]), span[p].left);
    }
  }
  if (!next) return;
  normalise(a.weight, a.bias);
  if (a.x) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (span[p].left > 0)
        store_piece(to_global(static_cast<uint16_t*>(a.x)) + static_cast<size_t>(row) * N + first_of(p),
                    to_bf16(v[p]), span[p].left);
    return;
  }
  // The codes and scale of w4a8_quantize, of values that were not rounded before. 127 /
  // max is past fp32 for a row below 2^-121, which is raised by a power of two first.
  float big = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(v[p].v[j]));
  big = join(big, [](float x, float y) { return fmaxf(x, y); });
  const float raise = big < 0x1p-100f ? 0x1p64f : 1.f;
  const float inv = big > 0.f ? 127.f / (big * raise) : 0.f;
  if (mine == 0) to_global(a.sx)[row] = big / 127.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (span[p].left <= 0) continue;
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float q = __builtin_rintf(v[p].v[j] * raise * inv);
      q = q > 127.f ? 127.f : q;
      q = q < -127.f ? -127.f : q;
      c[j] = static_cast<uint32_t>(static_cast<int>(q)) & 0xFFu;
    }
    // half a 16-block: byte j holds offset 0,4,1,5,2,6,3,7
    const u32x2 o = {c[0] | c[4] << 8 | c[1] << 16 | c[5] << 24, c[2] | c[6] << 8 | c[3] << 16 | c[7] << 24};
    *reinterpret_cast<gptr<u32x2>>(to_global(static_cast<uint8_t*>(a.xq)) + static_cast<size_t>(row) * N +
                                   first_of(p)) = o;
  }
}

// Rows of fewer than 8 columns: a thread a row.
__global__ __launch_bounds__(64) void norm_short_kernel(const NormArgs args) {
  const w4a16_norm_args& a = args.a;
  const int N = args.N;
  const long long row = static_cast<long long>(blockIdx.x) * 64 + threadIdx.x;
  if (row >= args.T) return;
  const float n = static_cast<float>(N);
  const bool wide = a.residual_type == W4A16_RESIDUAL_F32;
  auto bf16_at = [](const void* p, long long i) { return bf16_bits_to_f32(to_global(static_cast<const uint16_t*>(p))[i]); };
  float v[7];
  auto normalise = [&](const void* w, const void* b) {
    // In 64 bits: sums of at most 7 values, and of their squares, are exact there but for
    // their last half steps, and none overflows.
    double mean = 0.0, s = 0.0;
    if (a.kind == W4A16_NORM_LAYER) {
      for (int j = 0; j < 7; ++j) mean += j < N ? v[j] : 0.f;
      mean /= n;
    }
    for (int j = 0; j < 7; ++j) s += j < N ? (v[j] - mean) * (v[j] - mean) : 0.0;
    const float r = 1.f / sqrtf(static_cast<float>(s / n) + a.eps);
    for (int j = 0; j < 7; ++j) {
      if (j >= N) continue;
      v[j] = static_cast<float>((v[j] - mean) * r);
      if (w) v[j] *= bf16_at(w, j) + (a.unit_offset ? 1.f : 0.f);
      if (b) v[j] += bf16_at(b, j);
    }
  };
  for (int j = 0; j < 7; ++j) v[j] = a.y && j < N ? bf16_at(a.y, row * N + j) : 0.f;
  if (a.y && a.post_norm) normalise(a.post_weight, a.post_bias);
  for (int j = 0; j < 7; ++j) {
    if (j >= N) continue;
    if (a.y) v[j] = (a.gate ? v[j] * bf16_at(a.gate, row / a.gate_rows * N + j) : v[j]) * a.scale;
    if (a.residual)
      v[j] += wide ? to_global(static_cast<const float*>(a.residual))[row * N + j] : bf16_at(a.residual, row * N + j);
    if (a.residual_out) {
      if (wide)
        to_global(static_cast<float*>(a.residual_out))[row * N + j] = v[j];
      else
        to_global(static_cast<uint16_t*>(a.residual_out))[row * N + j] = f32_to_bf16_bits(v[j]);
    }
  }
  if (!a.x) return;  // codes need 16 columns
  normalise(a.weight, a.bias);
  for (int j = 0; j < 7; ++j)
    if (j < N) to_global(static_cast<uint16_t*>(a.x))[row * N + j] = f32_to_bf16_bits(v[j]);
}

template <int P, int L, bool BLOCK>
hipError_t launch_norm_t(const NormArgs& args, int threads, hipStream_t stream) {
  const long long blocks = BLOCK ? args.T : (static_cast<long long>(args.T) + 256 / L - 1) / (256 / L);
  if (blocks * threads > 0xFFFFFFFFLL) return hipErrorNotSupported;
  NormArgs copy = args;
  void* kargs[] = {&copy};
  const void* fn = args.N % 8 != 0 ? reinterpret_cast<const void*>(&norm_kernel<P, L, BLOCK, true>)
                                   : reinterpret_cast<const void*>(&norm_kernel<P, L, BLOCK, false>);
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(threads), kargs, 0, stream);
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
  if (N < 8) {
    NormArgs copy = args;
    void* kargs[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void*>(&norm_short_kernel), dim3((T - 1) / 64 + 1), dim3(64), kargs, 0,
                           stream);
  }
  if (pieces <= 16) return launch_norm_t<1, 16, false>(args, 256, stream);
  if (pieces <= 32) return launch_norm_t<1, 32, false>(args, 256, stream);
  if (pieces <= 64) return launch_norm_t<1, 64, false>(args, 256, stream);
  // Two pieces a thread halve the waves that a sum has to meet; with few rows, which do
  // not fill the card, one a thread is sooner done (us, one / two / four): 64 rows of 5120
  // with post norm and codes 11.3 / 12.1 / 13.9, 500 of 4096 7.1 / 7.6 / 10.6; 2048 of
  // 2741 with layer norms 20.1 / 17.4 / 22.1, 4000 of 4096 with post norm 32.6 / 29.9 / 35.7.
  if (args.T < 1024 && pieces <= 64 * kNormMaxWaves) return launch_norm_block<1>(args, pieces, stream);
  if (pieces <= 2 * 64 * kNormMaxWaves) return launch_norm_block<2>(args, pieces, stream);
  // (1000 rows of 17408: 35.5 us with three, 46.3 with four)
  if (pieces <= 3 * 64 * kNormMaxWaves) return launch_norm_block<3>(args, pieces, stream);
  if (pieces <= 4 * 64 * kNormMaxWaves) return launch_norm_block<4>(args, pieces, stream);
  // rows past 32768, which this form's 64 values fill the registers with: 7 of a thread's 128
  // lie in scratch memory, 33 with odd lengths (500 rows of 65536: 72 us, of 65535: 104)
  return launch_norm_block<8>(args, pieces, stream);
}

}  // namespace w4a16_internal

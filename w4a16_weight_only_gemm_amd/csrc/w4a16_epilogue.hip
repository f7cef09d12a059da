// w4a16_epilogue.hip -- the product of w4a16_gemm with bias, activation, scale and
// residual in its epilogue.
//
//     y = residual + scale * act(x W + bias),  gated: residual + scale * act(g) * u
//
// The product is w4a16_gemm's, by the same two kernels and the same rule between
// them (w4a16_plain.h, w4a16_tile.h), and so is what bounds it; the sums are never
// rounded before the epilogue, and y is written once. Gated, a workgroup owns the
// same columns of the gate half and of the up half, so both sums of a value meet
// in it and only N / 2 columns are written.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "w4a16_device.h"
#include "w4a16_epilogue.h"
#include "w4a16_launch.h"
#include "w4a16_layer_launch.h"
#include "w4a16_plain.h"
#include "w4a16_tile.h"

namespace w4a16_internal {
namespace {

// ------------------------------------------------------------- many rows

// Columns of y of one tile, and the row stride (floats) of the finished values in
// LDS, padded so that the rows of a register's lanes start in different banks.
template <int EPI>
struct EpTile {
  static constexpr int Cols = EPI == kEpiGated ? kLgWaves * 16 : kLgBlocks * 16;
  static constexpr int Stride = Cols + 4;
};

// One workgroup per MB x 16 rows by 256 columns (gated: 128 of each half) over the
// whole K range, loads issued D k-tiles ahead.
template <int GS, int MB, int D, int EPI>
__global__ __launch_bounds__(kLgThreads, 1) void tile_epilogue_kernel(const GemmArgs a, const Epilogue ep,
                                                                      int MT, int NT) {
  using C = LgCfg<GS, MB>;
  constexpr bool GATED = EPI == kEpiGated;
  constexpr int Cols = EpTile<EPI>::Cols, Stride = EpTile<EPI>::Stride;
  extern __shared__ __attribute__((aligned(16))) unsigned char ep_lds[];
  const int tile = xcd_grouped(blockIdx.x, MT * NT);
  const int mt = tile % MT, nt = tile / MT, m0 = mt * C::Rows;
  TileEngine<GS, MB> e;
  e.setup(ep_lds, a.x, a.qweight, a.scales, a.M, a.N, a.K, m0, nt);
  if constexpr (GATED) {
    // a wave's two blocks are the gate and the up block of 16 columns
    e.blk[0] = min(nt * kLgWaves + e.wave, e.NCB / 2 - 1);
    e.blk[1] = e.blk[0] + e.NCB / 2;
  }
  Acc<MB> acc;
  zero(acc);
  const int kt = (e.G + C::T - 1) / C::T;
  if constexpr (D == 1)
    e.kloop_spread(acc, 0, kt);  // 1024 rows, 5120 x 34816, gated: 371 us, with kloop 390
  else
    e.template kloop_deep<D>(acc, 0, kt);

  // Through LDS (free behind the k-loop's last barrier) to whole 16-byte pieces of
  // rows: the registers hold one column of four rows per lane.
  const int n_out = GATED ? a.N / 2 : a.N, col0 = nt * Cols;
  float* const vals = reinterpret_cast<float*>(ep_lds);
  const int jgrp = e.lane >> 4, c16 = e.lane & 15;
#pragma unroll
  for (int nb = 0; nb < (GATED ? 1 : kLgNB); ++nb) {
    const int col = (GATED ? e.wave : e.wave * kLgNB + nb) * 16 + c16;
    const int n = min(col0 + col, n_out - 1);  // past the last column: not stored
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        vals[(mb * 16 + 4 * jgrp + r) * Stride + col] =
            GATED ? epilogue_gated(ep, acc.v[mb][0][r], acc.v[mb][1][r], n, n_out)
                  : epilogue_value(ep, acc.v[mb][nb][r], n);
  }
  __syncthreads();
  gptr<uint16_t> yg = to_global(a.y);
  const gptr<const uint16_t> res = to_global(ep.residual);
  for (int i = threadIdx.x; i < C::Rows * (Cols / 8); i += kLgThreads) {
    const int r = i / (Cols / 8), col = i % (Cols / 8) * 8;
    const int left = n_out - (col0 + col);
    if (m0 + r >= a.M || left <= 0) continue;
    const size_t at = static_cast<size_t>(m0 + r) * n_out + col0 + col;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(vals + r * Stride + col);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(vals + r * Stride + col + 4);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = ep.scale * (j < 4 ? lo[j % 4] : hi[j % 4]);
    if (ep.residual) {
      const u32x4 d = load_piece(res + at, left);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = d[j / 2];
        const float rv = __builtin_bit_cast(float, j % 2 ? w & 0xFFFF0000u : w << 16);
        v[j] = __builtin_fmaf(ep.scale, j < 4 ? lo[j % 4] : hi[j % 4], rv);
      }
    }
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = f32_to_bf16_bits(v[2 * j]) | static_cast<uint32_t>(f32_to_bf16_bits(v[2 * j + 1])) << 16;
    store_piece(yg + at, o, left);
  }
}

template <int GS, int MB, int D, int EPI>
hipError_t launch_tile_epilogue_t(const GemmArgs& a, const Epilogue& ep, hipStream_t stream) {
  using C = LgCfg<GS, MB>;
  constexpr size_t Out = static_cast<size_t>(C::Rows) * EpTile<EPI>::Stride * 4;
  constexpr size_t Lds = C::Lds > Out ? C::Lds : Out;
  const int NCB = (a.N + 15) / 16;
  int NT = EPI == kEpiGated ? (NCB / 2 + kLgWaves - 1) / kLgWaves : (NCB + kLgBlocks - 1) / kLgBlocks;
  const int n_out = EPI == kEpiGated ? a.N / 2 : a.N;
  const void* fn = reinterpret_cast<const void*>(&tile_epilogue_kernel<GS, MB, D, EPI>);
  hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Lds));
  if (e != hipSuccess) return e;
  // Buffer offsets are 32-bit: each launch covers at most `rows` rows of x.
  long long rows = (0xFFFFFFFFLL - 16) / (2LL * a.K);
  rows -= rows % C::Rows;
  if (rows < C::Rows) return hipErrorNotSupported;
  const long long most = a.M < rows ? a.M : rows;
  if ((most + C::Rows - 1) / C::Rows * NT * kLgThreads > 0xFFFFFFFFLL) return hipErrorNotSupported;
  for (long long r0 = 0; r0 < a.M; r0 += rows) {
    GemmArgs part = a;
    Epilogue pe = ep;
    part.M = static_cast<int>(a.M - r0 < rows ? a.M - r0 : rows);
    part.x = a.x + r0 * a.K;
    part.y = a.y + r0 * n_out;
    if (pe.residual) pe.residual += r0 * n_out;
    int MT = (part.M + C::Rows - 1) / C::Rows;
    void* kargs[] = {&part, &pe, &MT, &NT};
    e = hipLaunchKernel(fn, dim3(static_cast<unsigned>(MT * NT)), dim3(kLgThreads), kargs, Lds, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Loads ahead as in w4a16_gemm's tiles.
template <int GS, int EPI>
hipError_t launch_tile_epilogue_g(const GemmArgs& a, const Epilogue& ep, int rows, hipStream_t stream) {
  switch (rows) {
    case 32: return launch_tile_epilogue_t<GS, 2, 3, EPI>(a, ep, stream);
    case 64: return launch_tile_epilogue_t<GS, 4, 3, EPI>(a, ep, stream);
    default: return launch_tile_epilogue_t<GS, 8, 1, EPI>(a, ep, stream);
  }
}

// --------------------------------------------------------------- few rows

// The form for a gated product: w4a16_gemm's where its column blocks come in pairs,
// else one that has pairs. For the 4-wave forms of wide N that is 6 blocks while that
// gives every compute unit a workgroup, else 2 (us of 2, 4 and 6 blocks at 5120 x 34816: 1
// row 24.0, 21.8, 20.8, 16 rows 29.1, 27.4, 23.7; at 2560 x 17408: 1 row 8.1, 9.9, 10.5, 16
// rows 10.2, 10.4, 10.7).
int gated_form(int M, int N, int K, int group) {
  const int f = plain_form(M, N, K, group);
  const size_t staged = static_cast<size_t>(M < 16 ? M : 16) * (static_cast<size_t>(K) + 8) * 2 +
                        static_cast<size_t>(K / group) * 64 + 16 * 2 * 1024;
  switch (f) {
    case kOne16Staged: return staged <= kPlainLdsLimit ? kDeepStaged : kTwo16;
    case kOne16: return kTwo16;
    case kXs1x3w4: case kXs1x5w4: return N / 32 / 3 >= kModelCUs ? kXs1x6w4 : kXs1x2w4;
    case kXs1x5: return kXs1x4;
    case kXs2x3: case kXs2x5: case kXs2x5w4: return kXs2x4;
    default: return f;
  }
}

template <int GS>
hipError_t launch_epilogue_g(const GemmArgs& a, const Epilogue& ep, bool gated, hipStream_t stream) {
  if constexpr (GS <= 128) {
    // The 4-wave form of 2 x 5 blocks has no twin in pairs as good as the tiles (2 x 4 blocks
    // at 24 rows, 5120 x 34816: 36.2 us, tiles 32.1), which end at weights of 4 GB.
    const bool tiles = choose_path(a.M, a.N, a.K, GS) == W4A16_PATH_LARGE ||
                       (gated && a.M <= kPlainMaxRows && plain_form(a.M, a.N, a.K, GS) == kXs2x5w4);
    if (tiles && large_runs(a.N, a.K, GS)) {
      int rows = 128;
      tile_estimate_us(a.M, a.N, a.K, GS, &rows);
      return gated ? launch_tile_epilogue_g<GS, kEpiGated>(a, ep, rows, stream)
                   : launch_tile_epilogue_g<GS, kEpiPlain>(a, ep, rows, stream);
    }
  }
  if (a.M > kPlainMaxRows) return hipErrorNotSupported;
  return gated ? launch_plain_form<GS, kEpiGated>(gated_form(a.M, a.N, a.K, GS), a, ep, stream)
               : launch_plain_form<GS, kEpiPlain>(plain_form(a.M, a.N, a.K, GS), a, ep, stream);
}

}  // namespace

hipError_t launch_epilogue(const GemmArgs& a, const Epilogue& ep, hipStream_t stream) {
  const bool gated = ep.act == W4A16_ACT_SWIGLU || ep.act == W4A16_ACT_GEGLU;
  switch (a.group) {
    case 32: return launch_epilogue_g<32>(a, ep, gated, stream);
    case 64: return launch_epilogue_g<64>(a, ep, gated, stream);
    case 128: return launch_epilogue_g<128>(a, ep, gated, stream);
    case 256: return launch_epilogue_g<256>(a, ep, gated, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w4a16_internal

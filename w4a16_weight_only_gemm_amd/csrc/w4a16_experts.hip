// w4a16_experts.hip -- the experts' W4A16 products over the rows routed to them.
//
// Expert e multiplies the n_e = offsets[e + 1] - offsets[e] rows listed for it
// by its own packed weights. How many rows each expert has is known on the
// device only, so the grid covers the most row tiles the slots can make
// (floor(slots / tile) + min(slots, experts)), and every workgroup finds its
// expert, row tile and column tile from the offsets: a wave sums the experts'
// row-tile counts (a few per lane, one prefix sum over the lanes) and looks up
// its own index. Workgroups past the last tile exit. One launch, no host
// round trip, no workspace.
//
// The tiles of an expert follow each other, its row tiles fastest: workgroups
// that share a column tile's weights run at the same time on one XCD and find
// them in its L2.
//
//  * few rows per expert (decode): experts_small_kernel, 16 or 32 rows x a few
//    16-column blocks per workgroup, whose waves split K and are summed
//    through LDS; every weight byte of an expert is read from HBM once. Bound
//    by HBM.
//  * many rows: experts_tile_kernel, the R x 256 MFMA tile engine of the dense
//    product with its rows gathered. Bound by MFMA.
//
// With SwiGLU a workgroup owns the same columns of the gate half and of the
// up half (its column blocks come in such pairs), so the activation is formed
// on the fp32 sums and only N / 2 columns are written.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "w4a16_device.h"
#include "w4a16_moe_launch.h"
#include "w4a16_tile.h"

namespace w4a16_internal {
namespace {

// A workgroup's place: expert (or -1), first list entry and number of rows of
// its row tile, the row tile within the expert and the expert's row tiles.
struct Place {
  int expert, tile, tiles, begin, count;
};

// Expert and row tile of unit `u` of all experts' (row tile, column tile)
// units, NT column tiles each; TM rows per row tile. Offsets out of range are
// clamped, so that a bad list cannot lead outside the buffers. `total` is the
// number of units.
template <int TM>
struct TileMap {
  int per, lane, excl, sum, total_tiles;
  const int* off;
  int E, slots;

  __device__ __forceinline__ int clamp(int v) const { return v < 0 ? 0 : v > slots ? slots : v; }
  __device__ __forceinline__ void setup(const int* offsets, int E_, int slots_) {
    off = offsets;
    E = E_;
    slots = slots_;
    lane = threadIdx.x & 63;
    per = (E + 63) / 64;
    sum = 0;
    int lo = clamp(off[min(lane * per, E)]);
    for (int i = 0; i < per; ++i) {
      const int hi = clamp(off[min(lane * per + i + 1, E)]);
      sum += hi > lo ? (hi - lo + TM - 1) / TM : 0;
      lo = hi;
    }
    int s = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(s, o);
      if (lane >= o) s += v;
    }
    excl = s - sum;
    total_tiles = __builtin_amdgcn_readlane(s, 63);
  }
  // The place of unit u < total_tiles * NT, and its column tile.
  __device__ __forceinline__ Place find(int u, int NT, int& nt) const {
    const int rt = u / NT;
    const uint64_t owner = __ballot(rt >= excl && rt < excl + sum);
    const int src = __builtin_ctzll(owner);
    int first = excl, e = 0, lo = clamp(off[min(lane * per, E)]), begin = 0, n = 0, tiles = 0, at = 0;
    for (int i = 0; i < per; ++i) {
      const int hi = clamp(off[min(lane * per + i + 1, E)]);
      const int t = hi > lo ? (hi - lo + TM - 1) / TM : 0;
      if (rt >= first && rt < first + t) {
        e = lane * per + i;
        begin = lo;
        n = hi - lo;
        tiles = t;
        at = first;
      }
      first += t;
      lo = hi;
    }
    Place p;
    p.expert = __builtin_amdgcn_readlane(e, src);
    p.tiles = __builtin_amdgcn_readlane(tiles, src);
    const int eb = __builtin_amdgcn_readlane(begin, src);
    const int en = __builtin_amdgcn_readlane(n, src);
    // the expert's units in order: row tiles fastest
    const int local = u - __builtin_amdgcn_readlane(at, src) * NT;
    nt = local / p.tiles;
    p.tile = local - nt * p.tiles;
    p.begin = eb + p.tile * TM;
    p.count = min(en - p.tile * TM, TM);
    return p;
  }
};

__device__ __forceinline__ float swiglu(float gate, float up) {
  return gate / (1.f + __expf(-gate)) * up;
}

// --------------------------------------------------------------- few rows

template <int GS, int MB, int NB>
struct ExStage {
  uint32_t w[NB][GS / 32];
  uint32_t s2[NB];
  u32x4 x[MB][GS / 32];
};

// MB x 16 rows by NB column blocks; the WAVES waves split the groups of K.
// XS (group 128): activation rows are loaded coalesced, 16 lanes per 256-byte
// row piece, and turned into the MFMA operand arrangement through a
// wave-private LDS area (lg_slot: free of bank conflicts).
template <int GS, int MB, int NB, int WAVES, int P, bool XS, bool ACT>
__global__ __launch_bounds__(64 * WAVES) void experts_small_kernel(const ExpertsArgs a, int NT) {
  constexpr int WPL = GS / 32;
  constexpr int TM = 16 * MB;
  static_assert(!XS || GS == 128, "coalesced staging: group 128");
  static_assert(!ACT || NB % 2 == 0, "gate and up blocks in pairs");
  TileMap<TM> map;
  map.setup(a.offsets, a.E, a.slots);
  const int total = map.total_tiles * NT;
  if (static_cast<int>(blockIdx.x) >= total) return;
  int nt;
  const Place pl = map.find(xcd_grouped(blockIdx.x, total), NT, nt);

  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int c16 = lane & 15, lg = lane >> 4;
  const int K = a.K, G = K / GS, NCB = (a.N + 15) / 16;
  const int g0 = static_cast<int>(static_cast<long long>(G) * wave / WAVES);
  const int g1 = static_cast<int>(static_cast<long long>(G) * (wave + 1) / WAVES);

  extern __shared__ __attribute__((aligned(16))) uint32_t ex_lds[];
  __shared__ int slot_of[TM];  // output row of each tile row, -1: none
  float* const red = reinterpret_cast<float*>(ex_lds);
  constexpr int kXsWaveBytes = XS ? MB * 16 * 256 : 0;
  unsigned char* const xs_lds = reinterpret_cast<unsigned char*>(ex_lds) +
                                static_cast<size_t>(WAVES) * MB * NB * 1024 + wave * kXsWaveBytes;
  if (static_cast<int>(threadIdx.x) < TM) {
    const int r = threadIdx.x;
    int s = r < pl.count ? a.rows[pl.begin + r] : -1;
    if (s < 0 || s >= a.slots) s = -1;
    slot_of[r] = s;
  }

  // column block of nb: with ACT the first half are gate blocks, the second
  // the up blocks of the same columns; past the last: clamped, not stored
  const uint32_t* qw = a.qweight + static_cast<size_t>(pl.expert) * NCB * G * 64 * WPL;
  const uint16_t* sp = a.scales + static_cast<size_t>(pl.expert) * NCB * G * 16;
  gptr<const uint32_t> wbase[NB];
  gptr<const uint32_t> sbase[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    int b;
    if constexpr (ACT)
      b = min(nt * (NB / 2) + nb % (NB / 2), NCB / 2 - 1) + (nb >= NB / 2 ? NCB / 2 : 0);
    else
      b = min(nt * NB + nb, NCB - 1);
    wbase[nb] = to_global(qw) + static_cast<size_t>(b) * G * 64 * WPL + lane * WPL;
    sbase[nb] = reinterpret_cast<gptr<const uint32_t>>(to_global(sp) + static_cast<size_t>(b) * G * 16 +
                                                       (c16 & ~1));
  }
  // activation row of tile row r: rows past the last repeat it
  auto row_ptr = [&](int r) {
    int s = a.rows[pl.begin + min(r, pl.count - 1)];
    if (s < 0 || s >= a.slots) s = 0;
    return to_global(a.x) + static_cast<size_t>(s / a.x_div) * K;
  };
  constexpr int XR = XS ? 4 : 1;
  gptr<const uint16_t> xrow[MB * XR];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int i = 0; i < XR; ++i)
      xrow[mb * XR + i] = XS ? row_ptr(16 * mb + 4 * i + lg) + 8 * c16
                             : row_ptr(16 * mb + c16) + lg * WPL * 8;

  auto load_stage = [&](ExStage<GS, MB, NB>& st, int grp) {
    grp = min(grp, g1 - 1);  // past the wave's last group: re-read it (unused)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const gptr<const uint32_t> wp = wbase[nb] + static_cast<size_t>(grp) * 64 * WPL;
      if constexpr (WPL >= 4) {
#pragma unroll
        for (int h = 0; h < WPL / 4; ++h) {
          const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<gptr<const u32x4>>(wp) + h);
#pragma unroll
          for (int q = 0; q < 4; ++q) st.w[nb][4 * h + q] = v[q];
        }
      } else {
#pragma unroll
        for (int t = 0; t < WPL; ++t) st.w[nb][t] = __builtin_nontemporal_load(wp + t);
      }
      st.s2[nb] = sbase[nb][static_cast<size_t>(grp) * 8];
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < WPL; ++i) {
        if constexpr (XS)
          st.x[mb][i] = *reinterpret_cast<gptr<const u32x4>>(xrow[mb * 4 + i] + static_cast<size_t>(grp) * GS);
        else
          st.x[mb][i] = *reinterpret_cast<gptr<const u32x4>>(xrow[mb] + static_cast<size_t>(grp) * GS + 8 * i);
      }
  };

  f32x4 yacc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) yacc[mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (g1 > g0) {
    ExStage<GS, MB, NB> stage[P];
#pragma unroll
    for (int p = 0; p < P; ++p) load_stage(stage[p], g0 + p);
    const bf16x8 bias = bias_operand();
    for (int c = g0; c < g1; c += P) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int grp = c + p;
        if (grp < g1) {
          ExStage<GS, MB, NB>& st = stage[p];
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            bf16x8 xa[WPL];
            if constexpr (XS) {
              unsigned char* area = xs_lds + mb * 16 * 256;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = 4 * i + lg;
                *reinterpret_cast<u32x4*>(area + row * 256 + lg_slot(c16, row) * 16) = st.x[mb][i];
              }
#pragma unroll
              for (int t = 0; t < WPL; ++t)
                xa[t] = *reinterpret_cast<const bf16x8*>(area + c16 * 256 + lg_slot(lg * WPL + t, c16) * 16);
            } else {
#pragma unroll
              for (int t = 0; t < WPL; ++t) xa[t] = act_frag(st.x[mb][t]);
            }
            f32x4 accb = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < WPL; ++t) accb = mfma16(xa[t], bias, accb);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              f32x4 acc = accb;
#pragma unroll
              for (int t = 0; t < WPL; ++t) acc = mfma16(xa[t], dequant_biased(st.w[nb][t]), acc);
              const float s = fp16_bits_to_f32(static_cast<uint16_t>(st.s2[nb] >> (16 * (c16 & 1))));
#pragma unroll
              for (int r = 0; r < 4; ++r) yacc[mb][nb][r] = __builtin_fmaf(s, acc[r], yacc[mb][nb][r]);
            }
          }
          load_stage(st, grp + P);
        }
      }
    }
  }

  // Sum over the waves in wave order: register r of (mb, nb) of lane l from
  // wave w at red[((w * MB + mb) * NB + nb) * 4 + r][l]; lane l holds rows
  // 4 (l / 16) + r of column l % 16 of its block.
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[(((wave * MB + mb) * NB + nb) * 4 + r) * 64 + lane] = yacc[mb][nb][r];
  __syncthreads();
  constexpr int NBO = ACT ? NB / 2 : NB;  // stored column blocks
  const int out_cols = ACT ? a.N / 2 : a.N;
  auto total_of = [&](int mb, int nb, int r, int l) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += red[(((w * MB + mb) * NB + nb) * 4 + r) * 64 + l];
    return sum;
  };
  for (int e = threadIdx.x; e < MB * NBO * 256; e += 64 * WAVES) {
    const int l = e & 63, r = (e >> 6) & 3, blk = e >> 8;
    const int mb = blk / NBO, nb = blk - mb * NBO;
    const int m = 16 * mb + 4 * (l >> 4) + r;
    const int n = (nt * NBO + nb) * 16 + (l & 15);
    const int s = slot_of[m];
    if (s < 0 || n >= out_cols) continue;
    float v = total_of(mb, nb, r, l);
    if constexpr (ACT) v = swiglu(v, total_of(mb, nb + NBO, r, l));
    to_global(a.y)[static_cast<size_t>(s) * out_cols + n] = f32_to_bf16_bits(v);
  }
}

template <int GS, int MB, int NB, int WAVES, int P, bool ACT>
hipError_t launch_small_t(const ExpertsArgs& a, hipStream_t stream) {
  constexpr bool XS = GS == 128;
  constexpr int TM = 16 * MB;
  const int NCB = (a.N + 15) / 16;
  int NT = ACT ? (NCB / 2 + NB / 2 - 1) / (NB / 2) : (NCB + NB - 1) / NB;
  const long long row_tiles = a.slots / TM + (a.slots < a.E ? a.slots : a.E);
  const long long blocks = row_tiles * NT;
  if (blocks * 64 * WAVES > 0xFFFFFFFFLL) return hipErrorInvalidValue;
  size_t lds = static_cast<size_t>(WAVES) * MB * NB * 1024;
  if (XS) lds += static_cast<size_t>(WAVES) * MB * 16 * 256;
  const void* fn = reinterpret_cast<const void*>(&experts_small_kernel<GS, MB, NB, WAVES, P, XS, ACT>);
  if (lds > 48 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  ExpertsArgs args = a;
  void* kargs[] = {&args, &NT};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(64 * WAVES), kargs, lds, stream);
}

// -------------------------------------------------------------- many rows

template <int GS, int MB, int D, bool ACT>
__global__ __launch_bounds__(kLgThreads, 1) void experts_tile_kernel(const ExpertsArgs a, int NT) {
  using C = LgCfg<GS, MB>;
  extern __shared__ __attribute__((aligned(16))) unsigned char ex_tile_lds[];
  __shared__ int slot_of[C::Rows];
  TileMap<C::Rows> map;
  map.setup(a.offsets, a.E, a.slots);
  const int total = map.total_tiles * NT;
  if (static_cast<int>(blockIdx.x) >= total) return;
  int nt;
  const Place pl = map.find(xcd_grouped(blockIdx.x, total), NT, nt);
  const int NCB = (a.N + 15) / 16, G = a.K / GS;
  if (static_cast<int>(threadIdx.x) < C::Rows) {
    const int r = threadIdx.x;
    int s = r < pl.count ? a.rows[pl.begin + r] : -1;
    if (s < 0 || s >= a.slots) s = -1;
    slot_of[r] = s;
  }
  __syncthreads();
  const int wave = uniform(threadIdx.x >> 6);
  // ACT: a wave's two blocks are the gate and the up block of 16 columns
  const int col_blk = ACT ? nt * kLgWaves + wave : nt * kLgBlocks + 2 * wave;
  const int blk0 = ACT ? min(col_blk, NCB / 2 - 1) : col_blk;
  const int blk1 = ACT ? blk0 + NCB / 2 : col_blk + 1;
  const size_t words = static_cast<size_t>(NCB) * 16 * a.K / 8;
  const long long x_rows = (static_cast<long long>(a.slots) + a.x_div - 1) / a.x_div;
  using Engine = TileEngine<GS, MB, true>;
  Engine e;
  e.setup_gathered(ex_tile_lds, a.x, static_cast<uint32_t>(x_rows * a.K * 2),
                   a.qweight + pl.expert * words, a.scales + static_cast<size_t>(pl.expert) * NCB * G * 16,
                   a.N, a.K, blk0, blk1, [&](int r) {
                     const int s = slot_of[r];
                     return s < 0 ? Engine::kNoRow
                                  : static_cast<uint32_t>(s / a.x_div) * static_cast<uint32_t>(a.K) * 2u;
                   });
  Acc<MB> acc;
  zero(acc);
  const int kt = (G + C::T - 1) / C::T;
  if constexpr (D == 1)
    e.kloop(acc, 0, kt);
  else
    e.template kloop_deep<D>(acc, 0, kt);
  gptr<uint16_t> yg = to_global(a.y);
  const int lane = threadIdx.x & 63, jgrp = lane >> 4;
  const int out_cols = ACT ? a.N / 2 : a.N;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int s = slot_of[mb * 16 + 4 * jgrp + r];
      if (s < 0) continue;
      const size_t at = static_cast<size_t>(s) * out_cols;
      if constexpr (ACT) {
        const int col = col_blk * 16 + (lane & 15);
        if (col < out_cols) yg[at + col] = f32_to_bf16_bits(swiglu(acc.v[mb][0][r], acc.v[mb][1][r]));
      } else {
#pragma unroll
        for (int nb = 0; nb < kLgNB; ++nb) {
          const int col = (col_blk + nb) * 16 + (lane & 15);
          if (col < out_cols) yg[at + col] = f32_to_bf16_bits(acc.v[mb][nb][r]);
        }
      }
    }
}

template <int GS, int MB, int D, bool ACT>
hipError_t launch_tile_t(const ExpertsArgs& a, hipStream_t stream) {
  using C = LgCfg<GS, MB>;
  const int NCB = (a.N + 15) / 16;
  int NT = ACT ? (NCB / 2 + kLgWaves - 1) / kLgWaves : (NCB + kLgBlocks - 1) / kLgBlocks;
  const long long row_tiles = a.slots / C::Rows + (a.slots < a.E ? a.slots : a.E);
  const long long blocks = row_tiles * NT;
  if (blocks * kLgThreads > 0xFFFFFFFFLL) return hipErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&experts_tile_kernel<GS, MB, D, ACT>);
  const hipError_t e =
      hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::Lds));
  if (e != hipSuccess) return e;
  ExpertsArgs args = a;
  void* kargs[] = {&args, &NT};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kLgThreads), kargs, C::Lds, stream);
}

// Few rows per expert on average: the small kernel; many: the tile engine
// (group 32, 64 or 128).
template <int GS, bool ACT>
hipError_t launch_experts_t(const ExpertsArgs& a, hipStream_t stream) {
  const int mean = a.slots / a.E;
  if constexpr (GS <= 128) {
    if (mean >= 96) return launch_tile_t<GS, 8, 1, ACT>(a, stream);
    if (mean >= 48) return launch_tile_t<GS, 4, 2, ACT>(a, stream);
  }
  if (mean >= 12) return launch_small_t<GS, 2, 2, 8, 1, ACT>(a, stream);
  return launch_small_t<GS, 1, 2, 8, 1, ACT>(a, stream);
}

}  // namespace

hipError_t launch_experts(const ExpertsArgs& a, hipStream_t stream) {
  switch (a.group) {
    case 32: return a.swiglu ? launch_experts_t<32, true>(a, stream) : launch_experts_t<32, false>(a, stream);
    case 64: return a.swiglu ? launch_experts_t<64, true>(a, stream) : launch_experts_t<64, false>(a, stream);
    case 128: return a.swiglu ? launch_experts_t<128, true>(a, stream) : launch_experts_t<128, false>(a, stream);
    case 256: return a.swiglu ? launch_experts_t<256, true>(a, stream) : launch_experts_t<256, false>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w4a16_internal

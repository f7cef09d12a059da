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
//  * few active experts (decode of few streams) or a deep K: experts_small_kernel,
//    16 rows x a few 16-column blocks per workgroup, whose waves split K and
//    are summed through LDS. Bound by HBM, and at one token by the chain of
//    dependent loads in front of it (offsets, then rows, then activations; the
//    first weights need only the offsets and start beside it).
//  * otherwise experts_tile_kernel, the R x 256 MFMA tile engine of the dense
//    product with its rows gathered: 32-row tiles, bound by HBM while the
//    experts have few rows each (4.6 TB/s at 37 tokens of 8 experts out of
//    128, of which 93 have rows), 128-row tiles, bound by LDS reads and MFMA, when they have many.
//
// With SwiGLU a workgroup owns the same columns of the gate half and of the
// up half (its column blocks come in such pairs), so the activation is formed
// on the fp32 sums and only N / 2 columns are written.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "w4a16_device.h"
#include "w4a16_launch.h"
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
// clamped, so that a bad list cannot lead outside the buffers; and the tiles are
// counted up to the grid's (`most`, at most 2^24: 64 lanes' counts fit an int),
// since offsets that do not ascend can list the slots E / 2 times over.
template <int TM>
struct TileMap {
  static constexpr int kHeld = 4;  // experts per lane held in registers
  int per, lane, excl, sum, total_tiles;
  int edge[kHeld + 1];             // the lane's experts' offsets, up to kHeld experts
  const int* off;
  int E, slots;

  __device__ __forceinline__ int load(int i) const {
    const int v = off[min(i, E)];
    return v < 0 ? 0 : v > slots ? slots : v;
  }
  static __device__ __forceinline__ int tiles_of(int lo, int hi) { return hi > lo ? (hi - lo + TM - 1) / TM : 0; }
  // Calls f(expert, lo, hi) for the lane's experts.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (per <= kHeld) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i < per) f(lane * per + i, edge[i], edge[i + 1]);
    } else {
      int lo = load(lane * per);
      for (int i = 0; i < per; ++i) {
        const int hi = load(lane * per + i + 1);
        f(lane * per + i, lo, hi);
        lo = hi;
      }
    }
  }
  __device__ __forceinline__ void setup(const int* offsets, int E_, int slots_, int most) {
    off = offsets;
    E = E_;
    slots = slots_;
    lane = threadIdx.x & 63;
    per = (E + 63) / 64;
    if (per <= kHeld) {  // all loads at once
#pragma unroll
      for (int i = 0; i <= kHeld; ++i) edge[i] = load(lane * per + min(i, per));
    }
    sum = 0;
    each([&](int, int lo, int hi) { sum += tiles_of(lo, hi); });
    sum = min(sum, most);
    int s = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(s, o);
      if (lane >= o) s += v;
    }
    excl = s - sum;
    total_tiles = min(__builtin_amdgcn_readlane(s, 63), most);
  }
  // The place of unit u < total_tiles * NT, and its column tile.
  __device__ __forceinline__ Place find(int u, int NT, int& nt) const {
    const int rt = u / NT;
    const uint64_t owner = __ballot(rt >= excl && rt < excl + sum);
    const int src = __builtin_ctzll(owner);
    int first = excl, e = 0, begin = 0, n = 0, tiles = 1, at = 0;
    each([&](int expert, int lo, int hi) {
      const int t = tiles_of(lo, hi);
      if (rt >= first && rt < first + t) {
        e = expert;
        begin = lo;
        n = hi - lo;
        tiles = t;
        at = first;
      }
      first += t;
    });
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

// MB x 16 rows by NB column blocks; the WAVES waves split the groups of K.
// XS (group 128): activation rows are loaded coalesced, 16 lanes per 256-byte
// row piece, and turned into the MFMA operand arrangement through a
// wave-private LDS area (lg_slot: free of bank conflicts).
template <int GS, int MB, int NB, int WAVES, int P4, int P16, bool XS, bool ACT>
__global__ __launch_bounds__(64 * WAVES) void experts_small_kernel(const ExpertsArgs a, int NT, int row_tiles) {
  constexpr int WPL = GS / 32;
  constexpr int TM = 16 * MB;
  static_assert(!XS || GS == 128, "coalesced staging: group 128");
  static_assert(!ACT || NB % 2 == 0, "gate and up blocks in pairs");
  TileMap<TM> map;
  map.setup(a.offsets, a.E, a.slots, row_tiles);
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
  f32x4 yacc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) yacc[mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

  // XI (with XS): load instructions per row block, 4 rows each. Tiles of at
  // most 4 rows take one; the operand rows behind them are left as they are in
  // LDS, and their results are not stored.
  auto stream = [&](auto xi_, auto p_) {
    constexpr int XI = xi_.value, P = p_.value;
    struct Stage {
      uint32_t w[NB][WPL];
      uint32_t s2[NB];
      u32x4 x[MB][XS ? XI : WPL];
    };
    auto load_weights = [&](Stage& st, int grp) {
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
    };
    // The weights need the expert only: the first groups' are on their way
    // before the rows are known.
    Stage stage[P];
#pragma unroll
    for (int p = 0; p < P; ++p) load_weights(stage[p], g0 + p);
    __builtin_amdgcn_sched_barrier(0);
    // activation row of tile row r: rows past the last repeat it
    auto row_ptr = [&](int r) {
      int s = a.rows[pl.begin + min(r, pl.count - 1)];
      if (s < 0 || s >= a.slots) s = 0;
      return to_global(a.x) + static_cast<size_t>(s / a.x_div) * K;
    };
    constexpr int XR = XS ? XI : 1;
    gptr<const uint16_t> xrow[MB * XR];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < XR; ++i)
        xrow[mb * XR + i] = XS ? row_ptr(16 * mb + 4 * i + lg) + 8 * c16
                               : row_ptr(16 * mb + c16) + lg * WPL * 8;
    auto load_rows = [&](Stage& st, int grp) {
      grp = min(grp, g1 - 1);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < (XS ? XI : WPL); ++i) {
          const gptr<const uint16_t> xp = XS ? xrow[mb * XR + i] : xrow[mb] + 8 * i;
          st.x[mb][i] = *reinterpret_cast<gptr<const u32x4>>(xp + static_cast<size_t>(grp) * GS);
        }
    };
#pragma unroll
    for (int p = 0; p < P; ++p) load_rows(stage[p], g0 + p);
    const bf16x8 bias = bias_operand();
    for (int c = g0; c < g1; c += P) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int grp = c + p;
        if (grp < g1) {
          Stage& st = stage[p];
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            bf16x8 xa[WPL];
            if constexpr (XS) {
              unsigned char* area = xs_lds + mb * 16 * 256;
#pragma unroll
              for (int i = 0; i < XI; ++i) {
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
          load_weights(st, grp + P);
          load_rows(st, grp + P);
        }
      }
    }
  };
  if (g1 > g0) {
    if constexpr (XS && MB == 1) {
      if (pl.count <= 4)
        stream(std::integral_constant<int, 1>{}, std::integral_constant<int, P4>{});
      else
        stream(std::integral_constant<int, 4>{}, std::integral_constant<int, P16>{});
    } else {
      // groups of 32 and 64: more of them ahead, as they are smaller (784 x
      // 4352, group 32, 1 token of 8 experts: 16.7 -> 11.6 us)
      constexpr int kAhead = GS == 32 ? 8 : GS == 64 ? 4 : P16;
      stream(std::integral_constant<int, 4>{}, std::integral_constant<int, kAhead>{});
    }
  }
  if (static_cast<int>(threadIdx.x) < TM) {
    const int r = threadIdx.x;
    int s = r < pl.count ? a.rows[pl.begin + r] : -1;
    if (s < 0 || s >= a.slots) s = -1;
    slot_of[r] = s;
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

template <int GS, int MB, int NB, int WAVES, int P4, int P16, bool ACT>
hipError_t launch_small_t(const ExpertsArgs& a, hipStream_t stream) {
  constexpr bool XS = GS == 128;
  constexpr int TM = 16 * MB;
  const int NCB = (a.N + 15) / 16;
  int NT = ACT ? (NCB / 2 + NB / 2 - 1) / (NB / 2) : (NCB + NB - 1) / NB;
  int row_tiles = a.slots / TM + (a.slots < a.E ? a.slots : a.E);
  const long long blocks = static_cast<long long>(row_tiles) * NT;
  if (blocks * 64 * WAVES > 0xFFFFFFFFLL) return hipErrorNotSupported;
  size_t lds = static_cast<size_t>(WAVES) * MB * NB * 1024;
  if (XS) lds += static_cast<size_t>(WAVES) * MB * 16 * 256;
  const void* fn = reinterpret_cast<const void*>(&experts_small_kernel<GS, MB, NB, WAVES, P4, P16, XS, ACT>);
  if (lds >= 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  ExpertsArgs args = a;
  void* kargs[] = {&args, &NT, &row_tiles};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(64 * WAVES), kargs, lds, stream);
}

// -------------------------------------------------------------- many rows

// Output columns of a tile and their LDS row stride in the epilogue (padded
// against bank conflicts).
template <bool ACT>
struct ExTile {
  static constexpr int Cols = ACT ? kLgWaves * 16 : kLgBlocks * 16;
  static constexpr int Stride = Cols * 2 + 16;
};

// One row tile with MB x 16 row blocks of the tile engine, D k-tiles ahead;
// slot_of names the output row of each tile row. ONCE: the expert's only tile.
template <int GS, int MB, int D, bool ACT, bool ONCE = false>
__device__ __forceinline__ void expert_tile(const ExpertsArgs& a, unsigned char* lds, const int* slot_of,
                                            const Place& pl, int nt) {
  using C = LgCfg<GS, MB>;
  const int NCB = (a.N + 15) / 16, G = a.K / GS;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  // ACT: a wave's two blocks are the gate and the up block of 16 columns
  const int blk0 = ACT ? min(nt * kLgWaves + wave, NCB / 2 - 1) : nt * kLgBlocks + 2 * wave;
  const int blk1 = ACT ? blk0 + NCB / 2 : blk0 + 1;
  const size_t words = static_cast<size_t>(NCB) * 16 * a.K / 8;
  const long long x_rows = (static_cast<long long>(a.slots) + a.x_div - 1) / a.x_div;
  using Engine = TileEngine<GS, MB, true, ONCE>;
  Engine e;
  e.setup_gathered(lds, a.x, static_cast<uint32_t>(x_rows * a.K * 2),
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
    e.kloop_spread(acc, 0, kt);
  else
    e.template kloop_deep<D>(acc, 0, kt);

  // Through LDS (free behind the k-loop's last barrier) to whole 16-byte
  // pieces of rows: the registers hold one column of four rows per lane
  // (32-byte runs otherwise).
  constexpr int Cols = ExTile<ACT>::Cols, Stride = ExTile<ACT>::Stride;
  const int jgrp = lane >> 4;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint16_t* row = reinterpret_cast<uint16_t*>(lds + (mb * 16 + 4 * jgrp + r) * Stride);
      if constexpr (ACT) {
        row[wave * 16 + (lane & 15)] = f32_to_bf16_bits(swiglu(acc.v[mb][0][r], acc.v[mb][1][r]));
      } else {
#pragma unroll
        for (int nb = 0; nb < kLgNB; ++nb)
          row[(wave * kLgNB + nb) * 16 + (lane & 15)] = f32_to_bf16_bits(acc.v[mb][nb][r]);
      }
    }
  __syncthreads();
  const int out_cols = ACT ? a.N / 2 : a.N, col0 = nt * Cols;
  gptr<uint16_t> yg = to_global(a.y);
  for (int i = threadIdx.x; i < MB * 16 * (Cols / 8); i += kLgThreads) {
    const int r = i / (Cols / 8), col = i % (Cols / 8) * 8;
    const int s = slot_of[r], left = out_cols - (col0 + col);
    if (s < 0 || left <= 0) continue;
    const u32x4 v = *reinterpret_cast<const u32x4*>(lds + r * Stride + col * 2);
    store_piece(yg + static_cast<size_t>(s) * out_cols + col0 + col, v, left);
  }
}

// MB: the most row blocks of a tile; the last tile of an expert takes the
// smallest of 2, 4, 8 row blocks that hold its rows.
template <int GS, int MB, bool ACT>
__global__ __launch_bounds__(kLgThreads, 1) void experts_tile_kernel(const ExpertsArgs a, int NT, int row_tiles) {
  constexpr int Rows = MB * 16;
  extern __shared__ __attribute__((aligned(16))) unsigned char ex_tile_lds[];
  __shared__ int slot_of[Rows];
  TileMap<Rows> map;
  map.setup(a.offsets, a.E, a.slots, row_tiles);
  const int total = map.total_tiles * NT;
  if (static_cast<int>(blockIdx.x) >= total) return;
  int nt;
  const Place pl = map.find(xcd_grouped(blockIdx.x, total), NT, nt);
  if (static_cast<int>(threadIdx.x) < Rows) {
    const int r = threadIdx.x;
    int s = r < pl.count ? a.rows[pl.begin + r] : -1;
    if (s < 0 || s >= a.slots) s = -1;
    slot_of[r] = s;
  }
  __syncthreads();
  if (MB > 2 && pl.count > 64)
    expert_tile<GS, MB, MB == 8 ? 1 : 2, ACT>(a, ex_tile_lds, slot_of, pl, nt);
  else if (MB > 2 && pl.count > 32)
    expert_tile<GS, MB == 2 ? 2 : 4, 2, ACT>(a, ex_tile_lds, slot_of, pl, nt);
  else if (MB == 2 && pl.tiles == 1)
    expert_tile<GS, 2, 2, ACT, true>(a, ex_tile_lds, slot_of, pl, nt);
  else
    expert_tile<GS, 2, 2, ACT>(a, ex_tile_lds, slot_of, pl, nt);
}

template <int GS, int MB, bool ACT>
hipError_t launch_tile_t(const ExpertsArgs& a, hipStream_t stream) {
  constexpr int Rows = MB * 16;
  constexpr size_t Out = static_cast<size_t>(Rows) * ExTile<ACT>::Stride;
  constexpr size_t Lds = LgCfg<GS, MB>::Lds > Out ? LgCfg<GS, MB>::Lds : Out;
  const int NCB = (a.N + 15) / 16;
  int NT = ACT ? (NCB / 2 + kLgWaves - 1) / kLgWaves : (NCB + kLgBlocks - 1) / kLgBlocks;
  int row_tiles = a.slots / Rows + (a.slots < a.E ? a.slots : a.E);
  const long long blocks = static_cast<long long>(row_tiles) * NT;
  if (blocks * kLgThreads > 0xFFFFFFFFLL) return hipErrorNotSupported;
  const void* fn = reinterpret_cast<const void*>(&experts_tile_kernel<GS, MB, ACT>);
  if (Lds > 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Lds));
    if (e != hipSuccess) return e;
  }
  ExpertsArgs args = a;
  void* kargs[] = {&args, &NT, &row_tiles};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kLgThreads), kargs, Lds, stream);
}

// The form, from what the host knows: slots, experts, N and K (how the slots
// spread over the experts is known on the device only; any form is right for
// any spread). Modelled on even spreads, in microseconds, and fitted to N x K =
// 2048 x 5120, 1536 x 2048, 8192 x 4096 (SwiGLU), 5120 x 1024 and 2048 x 768 at
// group 128 with 8, 32 and 128 experts, 1 to 2048 tokens of 8 experts each:
//   few rows (4 waves, 32 columns):  3 + workgroups (0.003 + 2e-6 K), a fifth
//     more from 2 rows per expert on (tiles past 4 rows)
//   32-row tiles: 3 + k-tiles max(0.7, 0.3 + 0.0025 workgroups)
// For instance (us, few rows against 32-row tiles, 128 experts): 2048 x 5120 at
// 1 token 11.2 / 31.9, at 16 86 / 84, at 64 140 / 113; 5120 x 1024 at 1 token
// 12.0 / 10.5, at 64 136 / 68. While there is at most one workgroup per compute
// unit, few rows takes 64 columns and 8 waves (2048 x 5120 at 1 token: 11.0
// against 11.7). With 8 waves a compute unit has enough on the way with one
// group per wave: 1, 2, 3 and 5 ahead 11.0, 11.1, 12.1, 13.5; 1536 x 2048 6.8,
// 7.3, 8.0, 8.7. With 4 waves 1, 2, 4 and 6 ahead: 12.2, 11.5, 11.7, 13.1; 2048 x
// 5120 at 4 tokens 35.1, 33.3, 33.0, 37.0.
// 128-row tiles from 100 rows per expert on with two workgroups per compute
// unit or more (32-row against 128-row: 2048 x 5120, 128 experts, mean 64: 246
// / 292, 128: 437 / 438, 256: 915 / 810; 8 experts of 256 rows: 55 / 74).
// Over 180 shapes (the five N x K, 8, 32 and 128 experts, 1 to 2048 tokens, even
// spread, weights from HBM) the form taken needs 1.02 times the fastest in the
// mean and 1.35 at worst (2048 x 768, 16 tokens of 8 experts: 8.9 against 6.6).
// 128-row tiles are ahead below that bound in places: 8 experts of 512 rows 104 /
// 83, group 32, 1344 x 2688, 40 experts of 200 rows 145 / 120.
// Group 256 has no tile engine; 16 rows a workgroup, from 12 rows per expert on
// 32, which reads the weights half as often but is behind where measured (16 rows
// each, 16 rows x 64 columns against 32 x 32: 2048 x 5120 347 / 394, 5120 x 1024
// 238 / 385).
template <int GS, bool ACT>
hipError_t launch_experts_t(const ExpertsArgs& a, hipStream_t stream) {
  const double mean = static_cast<double>(a.slots) / a.E;
  const double active = a.E * (1.0 - std::pow(1.0 - 1.0 / a.E, a.slots));
  const double blocks = (a.N + 15) / 16;
  if constexpr (GS <= 128) {
    const double kt = (a.K + kLgKT - 1) / kLgKT;
    const double cols = std::ceil(blocks / kLgBlocks);  // 256-column tiles
    const double rows16 = active + a.slots / 16, rows32 = active + a.slots / 32;
    const double small = 3.0 + rows16 * std::ceil(blocks / 2) * (0.003 + 2e-6 * a.K) * (mean > 2 ? 1.2 : 1.0);
    const double load = 0.3 + 0.0025 * rows32 * cols;
    const double tile = 3.0 + kt * (load > 0.7 ? load : 0.7);
    if (tile <= small) {
      if (mean >= 100 && a.slots / 128.0 * cols >= 2 * kModelCUs) return launch_tile_t<GS, 8, ACT>(a, stream);
      return launch_tile_t<GS, 2, ACT>(a, stream);
    }
  } else {
    if (mean >= 12) return launch_small_t<GS, 2, 2, 8, 1, 1, ACT>(a, stream);
  }
  if (active * std::ceil(blocks / 4) <= kModelCUs) return launch_small_t<GS, 1, 4, 8, 1, 1, ACT>(a, stream);
  return launch_small_t<GS, 1, 2, 4, 4, 1, ACT>(a, stream);
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

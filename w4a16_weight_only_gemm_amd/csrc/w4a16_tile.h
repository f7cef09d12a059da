// w4a16_tile.h -- the MFMA tile engine of the W4A16 kernels for many rows: an
// R x 256 output tile (R = 32, 64 or 128) per workgroup of 8 waves, activations
// staged through LDS, packed weights straight into registers. Used by the dense
// kernels (w4a16_large.hip, which describes the scheme) and by the experts'
// products (w4a16_experts.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "w4a16_device.h"

namespace w4a16_internal {

inline constexpr int kLgWaves = 8;                   // all along N
inline constexpr int kLgNB = 2;                      // 16-column blocks per wave
inline constexpr int kLgBlocks = kLgWaves * kLgNB;   // 16 column blocks = 256 columns
inline constexpr int kLgThreads = kLgWaves * 64;
inline constexpr int kLgKT = 128;                    // k per k-tile
inline constexpr int kLgPieces = kLgKT / 8;          // 16-byte pieces per row per k-tile
inline constexpr int kLgRowBytes = kLgKT * 2;
inline constexpr int kLgRowStep = kLgThreads / kLgPieces;  // 32 rows staged per pass

// Tile geometry and LDS layout for group size GS and MB 16-row blocks.
template <int GS, int MB>
struct LgCfg {
  static_assert(MB == 2 || MB == 4 || MB == 8, "32, 64 or 128 rows per tile");
  static constexpr int Rows = MB * 16;
  static constexpr int Loads = Rows * kLgPieces / kLgThreads;  // pieces staged per thread
  static constexpr int ABytes = Rows * kLgRowBytes;
  static constexpr int T = kLgKT / GS;        // groups per k-tile
  static constexpr int WPL = GS / 32;         // MFMA steps (words per lane) per group
  static constexpr int LPG = GS / 8;          // staging lanes per group
  static constexpr int SBytes = T * Rows * 4;
  static constexpr int BufBytes = ABytes + SBytes;
  static constexpr size_t Lds = 2 * static_cast<size_t>(BufBytes);
  static constexpr int Regs = MB * kLgNB * 4;  // accumulator floats per lane
};


template <int GS, int MB>
struct StageRegs {
  u32x4 d[LgCfg<GS, MB>::Loads];
};

template <int GS>
struct BRegs {
  uint32_t w[kLgNB][kLgKT / 32];    // 4 words per block per k-tile
  uint32_t s[kLgNB][kLgKT / GS];    // scale pairs (fp16 x 2) per group
};

template <int MB>
struct Acc {
  f32x4 v[MB][kLgNB];
};

template <int MB>
__device__ __forceinline__ void zero(Acc<MB>& a) {
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < kLgNB; ++nb) a.v[mb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// ------------------------------------------------------------------ tile engine
//
// One workgroup's view of one output tile: rows m0 .. m0 + Rows - 1, column
// blocks 16 nt .. 16 nt + 15 (wave w owns blocks 16 nt + 2w, 16 nt + 2w + 1).
// kloop() accumulates k-tiles [k0, k1) into acc; every wave of the workgroup
// must call it with the same arguments (it holds workgroup barriers).
//
// GATHER: the tile's rows are rows of x in any order (the rows routed to one
// expert): setup_gathered takes each thread's byte offsets of the rows it
// stages, and the two column blocks of every wave, instead of setup's
// contiguous ones. The rest (kloop, kloop_deep, compute) is the same.
// ONCE: no other workgroup reads the weights, so they pass the caches by
// (non-temporal; experts' products, 8 rows each of 128 experts, N = 2048, K =
// 5120: 126 -> 116 us).
template <int GS, int MB, bool GATHER = false, bool ONCE = false>
struct TileEngine {
  using C = LgCfg<GS, MB>;
  unsigned char* lds;
  int tid, lane, wave;
  int M, N, K, G, NCB, m0, nt;
  const uint16_t* xrow0;
  uint32_t xbytes;
  __amdgpu_buffer_rsrc_t rq, rs;
  int blk[kLgNB];
  uint32_t voff[GATHER ? C::Loads : 1];  // gathered rows: this thread's staging offsets

  __device__ __forceinline__ void setup(unsigned char* lds_, const uint16_t* x, const uint32_t* qw,
                                        const uint16_t* sp, int M_, int N_, int K_, int m0_,
                                        int nt_) {
    lds = lds_;
    tid = threadIdx.x;
    lane = tid & 63;
    wave = uniform(tid >> 6);
    M = M_;
    N = N_;
    K = K_;
    G = K / GS;
    NCB = (N + 15) / 16;
    m0 = m0_;
    nt = nt_;
    xbytes = static_cast<uint32_t>(M - m0) * static_cast<uint32_t>(K) * 2u;
    xrow0 = x + static_cast<size_t>(m0) * K;
    rq = make_rsrc(qw, static_cast<uint32_t>(NCB) * 16u * static_cast<uint32_t>(K) / 2u);
    rs = make_rsrc(sp, static_cast<uint32_t>(NCB) * 16u * static_cast<uint32_t>(G) * 2u);
#pragma unroll
    for (int nb = 0; nb < kLgNB; ++nb) {
      const int b = nt * kLgBlocks + wave * kLgNB + nb;
      blk[nb] = b < NCB ? b : NCB - 1;
    }
  }

  // The gathered form. x spans xbytes bytes (below 4 GB); row_off(r) is the byte
  // offset of the tile's row r in x, or kNoRow for one that reads as zero.
  static constexpr uint32_t kNoRow = 0xFFFFFE00u;
  template <typename RowOff>
  __device__ __forceinline__ void setup_gathered(unsigned char* lds_, const uint16_t* x,
                                                 uint32_t xbytes_, const uint32_t* qw,
                                                 const uint16_t* sp, int N_, int K_, int blk0,
                                                 int blk1, RowOff row_off) {
    lds = lds_;
    tid = threadIdx.x;
    lane = tid & 63;
    wave = uniform(tid >> 6);
    N = N_;
    K = K_;
    G = K / GS;
    NCB = (N + 15) / 16;
    xbytes = xbytes_;
    xrow0 = x;
    rq = make_rsrc(qw, static_cast<uint32_t>(NCB) * 16u * static_cast<uint32_t>(K) / 2u);
    rs = make_rsrc(sp, static_cast<uint32_t>(NCB) * 16u * static_cast<uint32_t>(G) * 2u);
    blk[0] = blk0 < NCB ? blk0 : NCB - 1;
    blk[1] = blk1 < NCB ? blk1 : NCB - 1;
    const int spiece = tid % kLgPieces, srow0 = tid / kLgPieces;
#pragma unroll
    for (int i = 0; i < C::Loads; ++i) {
      const uint32_t o = row_off(srow0 + i * kLgRowStep);
      voff[i] = o == kNoRow ? kNoRow : o + static_cast<uint32_t>(spiece) * 16u;
    }
  }

  // ---- activation staging: thread stages piece tid % 16 (8 values) of rows
  // tid / 16 + 32 i, through a buffer resource based at (row m0, k of the
  // k-tile) and ending at the end of x, so rows beyond M read as zero ----
  __device__ __forceinline__ void stage_load(StageRegs<GS, MB>& r, int t, int i0 = 0,
                                             int i1 = C::Loads) const {
    const __amdgpu_buffer_rsrc_t rx =
        make_rsrc(xrow0 + t * kLgKT, xbytes - static_cast<uint32_t>(t) * (kLgKT * 2));
    const int spiece = tid % kLgPieces, srow0 = tid / kLgPieces;
#pragma unroll
    for (int i = 0; i < C::Loads; ++i) {
      if (i < i0 || i >= i1) continue;
      uint32_t off;
      if constexpr (GATHER)
        off = voff[i];
      else
        off = (static_cast<uint32_t>(srow0 + i * kLgRowStep) * K + spiece * 8) * 2u;
      r.d[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0);
    }
  }
  __device__ __forceinline__ void stage_store(const StageRegs<GS, MB>& r, int buf) const {
    unsigned char* base = lds + buf * C::BufBytes;
    float* sums = reinterpret_cast<float*>(base + C::ABytes);
    const int spiece = tid % kLgPieces, srow0 = tid / kLgPieces;
#pragma unroll
    for (int i = 0; i < C::Loads; ++i) {
      const int row = srow0 + i * kLgRowStep;
      const float s = group_lane_sum<C::LPG>(neg_bias_sum8(r.d[i]));
      sums[(spiece / C::LPG) * C::Rows + row] = s;  // every lane of the group: same value
      const int sl = lg_slot(spiece, row);
      *reinterpret_cast<u32x4*>(base + row * kLgRowBytes + sl * 16) = r.d[i];
    }
  }

  // ---- this wave's weights and scales of k-tile t ----
  __device__ __forceinline__ void load_b(BRegs<GS>& r, int t, int nb0 = 0, int nb1 = kLgNB) const {
    const uint32_t qlane = static_cast<uint32_t>(lane) * C::WPL * 4u;
    const uint32_t slane = static_cast<uint32_t>(lane & 14) * 2u;
    constexpr int kCache = ONCE ? 2 : 0;  // the instruction's nt bit
#pragma unroll
    for (int gi = 0; gi < C::T; ++gi) {
      int grp = t * C::T + gi;
      if (grp > G - 1) grp = G - 1;
#pragma unroll
      for (int nb = 0; nb < kLgNB; ++nb) {
        if (nb < nb0 || nb >= nb1) continue;
        const uint32_t tile_idx = static_cast<uint32_t>(blk[nb]) * G + grp;
        const int qoff = static_cast<int>(tile_idx * (64u * C::WPL * 4u));
        if constexpr (C::WPL == 4) {
          u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rq, qlane, qoff, kCache);
#pragma unroll
          for (int w = 0; w < 4; ++w) r.w[nb][gi * 4 + w] = v[w];
        } else if constexpr (C::WPL == 2) {
          u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rq, qlane, qoff, kCache);
          r.w[nb][gi * 2 + 0] = v[0];
          r.w[nb][gi * 2 + 1] = v[1];
        } else {
          r.w[nb][gi] = __builtin_amdgcn_raw_buffer_load_b32(rq, qlane, qoff, kCache);
        }
        r.s[nb][gi] =
            __builtin_amdgcn_raw_buffer_load_b32(rs, slane, static_cast<int>(tile_idx * 32u), 0);
      }
    }
  }

  // One k-tile: 4 MFMA steps of 32 k. Step st belongs to group st / WPL of the
  // k-tile; a group's accumulation starts from its -24 * row-sum tile and
  // ends with the scaled add into acc_out.
  // after(st) runs behind step st's MFMAs.
  template <typename F>
  __device__ __forceinline__ void compute(Acc<MB>& acc_out, const BRegs<GS>& b, int t, int buf,
                                          F after) const {
    const unsigned char* base = lds + buf * C::BufBytes;
    const float* sums = reinterpret_cast<const float*>(base + C::ABytes);
    const int arow = lane & 15, jgrp = lane >> 4;
    const int shalf = (lane & 1) * 16;
    f32x4 acc[kLgNB][MB];
    f32x4 bias[MB];
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      const int gi = st / C::WPL, w = st % C::WPL;
      if (C::T > 1 && t * C::T + gi >= G) break;  // ragged last k-tile (uniform)
      if (w == 0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
          bias[mb] = *reinterpret_cast<const f32x4*>(sums + gi * C::Rows + mb * 16 + 4 * jgrp);
      }
      const int piece = gi * C::LPG + jgrp * C::WPL + w;
      bf16x8 af[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
        af[mb] = *reinterpret_cast<const bf16x8*>(base + (arow + mb * 16) * kLgRowBytes +
                                                 lg_slot(piece, arow) * 16);
      // Both blocks' operands are dequantized first and the step's
      // 2 x MB MFMAs then issue as one uninterrupted run (the scheduling
      // fences keep the compiler from spreading them among the VALU work),
      // row block by row block so that each A fragment is done with after
      // two MFMAs: 3 to 4 % faster at 512 to 1024 rows, 6 % at 64.
      bf16x8 bq[kLgNB];
#pragma unroll
      for (int nb = 0; nb < kLgNB; ++nb) bq[nb] = dequant_biased(b.w[nb][st]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < kLgNB; ++nb)
          acc[nb][mb] = mfma16(af[mb], bq[nb], w == 0 ? bias[mb] : acc[nb][mb]);
      __builtin_amdgcn_sched_barrier(0);
      after(st);
      if (w == C::WPL - 1) {
#pragma unroll
        for (int nb = 0; nb < kLgNB; ++nb) {
          const float sc = fp16_bits_to_f32(static_cast<uint16_t>(b.s[nb][gi] >> shalf));
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) acc_out.v[mb][nb] += sc * acc[nb][mb];
        }
      }
    }
  }

  __device__ __forceinline__ void compute(Acc<MB>& acc_out, const BRegs<GS>& b, int t,
                                          int buf) const {
    compute(acc_out, b, t, buf, [](int) {});
  }

  // k-tiles [k0, k1): k-tile t computes from LDS buffer (t - k0) & 1 while
  // k-tile t + 1 is loaded into registers and then staged into the other
  // buffer. Weight registers alternate between two sets (no copies). Every
  // k-tile ends with a workgroup barrier, so the LDS buffers are free on
  // return.
  __device__ __forceinline__ void kloop(Acc<MB>& acc, int k0, int k1) const {
    StageRegs<GS, MB> sr;
    BRegs<GS> b0, b1;
    stage_load(sr, k0);
    load_b(b0, k0);
    stage_store(sr, 0);
    lds_barrier();
    auto iter = [&](int t, const BRegs<GS>& cur, BRegs<GS>& nxt) {
      const int tn = t + 1 < k1 ? t + 1 : t;   // the last iteration reloads (unused)
      const int buf = (t - k0) & 1;
      stage_load(sr, tn);
      load_b(nxt, tn);
      __builtin_amdgcn_sched_barrier(0);       // issue the loads before the math
      compute(acc, cur, t, buf);
      stage_store(sr, buf ^ 1);
      lds_barrier();
    };
    for (int t = k0; t < k1; t += 2) {
      iter(t, b0, b1);
      if (t + 1 >= k1) break;
      iter(t + 1, b1, b0);
    }
  }

  // kloop with the weights' loads behind the MFMA runs of the first two steps:
  // issued in one run with the activations', they queue up in front of the
  // address unit and hold back the MFMAs behind them (experts' products, 256
  // rows each of 128 experts, N = 2048, K = 5120: 842 -> 810 us).
  __device__ __forceinline__ void kloop_spread(Acc<MB>& acc, int k0, int k1) const {
    StageRegs<GS, MB> sr;
    BRegs<GS> b0, b1;
    stage_load(sr, k0);
    load_b(b0, k0);
    stage_store(sr, 0);
    lds_barrier();
    auto iter = [&](int t, const BRegs<GS>& cur, BRegs<GS>& nxt) {
      const int tn = t + 1 < k1 ? t + 1 : t;   // the last iteration reloads (unused)
      const int buf = (t - k0) & 1;
      stage_load(sr, tn);
      __builtin_amdgcn_sched_barrier(0);
      compute(acc, cur, t, buf, [&](int st) {
        if (st == 0) load_b(nxt, tn, 0, 1);
        if (st == 1) load_b(nxt, tn, 1, 2);
      });
      stage_store(sr, buf ^ 1);
      lds_barrier();
    };
    for (int t = k0; t < k1; t += 2) {
      iter(t, b0, b1);
      if (t + 1 >= k1) break;
      iter(t + 1, b1, b0);
    }
  }

  // k-tiles [k0, k1) with the loads of k-tile t + D issued before k-tile t
  // computes: D register sets of activation pieces and D + 1 of weights (the
  // LDS double buffer as in kloop). For workgroups that each own a whole K
  // range at tile counts near the number of compute units, where one
  // workgroup's k-tiles follow each other on load latency rather than on
  // arithmetic. The step is unrolled over D (D + 1) k-tiles so that every
  // register set has a fixed name (an indexed copy would wait for its loads).
  template <int D>
  __device__ __forceinline__ void kloop_deep(Acc<MB>& acc, int k0, int k1) const {
    constexpr int PER = D * (D + 1);  // a multiple of D, D + 1 and 2
    StageRegs<GS, MB> sr[D];
    BRegs<GS> b[D + 1];
#pragma unroll
    for (int j = 0; j < D; ++j) {
      const int t = k0 + j < k1 ? k0 + j : k1 - 1;  // past the end: reload (unused)
      stage_load(sr[j], t);
      load_b(b[j], t);
    }
    stage_store(sr[0], 0);
    lds_barrier();
    for (int t0 = k0; t0 < k1; t0 += PER) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        // k-tile t = t0 + j: its weights are b[j % (D + 1)], its activations
        // sit in LDS buffer j & 1; sr[j % D] and b[(j + D) % (D + 1)] are free
        const int t = t0 + j;
        if (t >= k1) break;
        const int tl = t + D < k1 ? t + D : k1 - 1;
        stage_load(sr[j % D], tl);
        load_b(b[(j + D) % (D + 1)], tl);
        __builtin_amdgcn_sched_barrier(0);  // issue the loads before the math
        compute(acc, b[j % (D + 1)], t, j & 1);
        stage_store(sr[(j + 1) % D], (j + 1) & 1);
        lds_barrier();
      }
    }
  }

  // bf16 (RNE) stores of the rows and columns that exist.
  __device__ __forceinline__ void store(const Acc<MB>& acc, uint16_t* y) const {
    gptr<uint16_t> yg = to_global(y);
    const int jgrp = lane >> 4;
#pragma unroll
    for (int nb = 0; nb < kLgNB; ++nb) {
      const int col = (nt * kLgBlocks + wave * kLgNB + nb) * 16 + (lane & 15);
      if (col >= N) continue;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = m0 + mb * 16 + 4 * jgrp + r;
          if (row < M) yg[static_cast<size_t>(row) * N + col] = f32_to_bf16_bits(acc.v[mb][nb][r]);
        }
      }
    }
  }
};

}  // namespace w4a16_internal

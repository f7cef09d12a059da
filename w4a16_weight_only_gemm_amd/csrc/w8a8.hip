// w8a8.hip -- 8-bit integer product: int8 activations with one scale per row,
// int8 weights with one scale per output column, v_mfma_i32_16x16x64_i8.
//
// The sum over k is exact in int32 whatever its order (K <= 131072 keeps it in
// range); one conversion to fp32, two fp32 products and one rounding to bf16
// follow. Both operands keep the codes of an aligned 16-block of k in the same
// order (w4a8_quantize's), so the operands meet as they lie.
//
//  * w8a8_small_kernel (few rows): MB x 16 rows by NB 16-column blocks per
//    workgroup, whose waves split K and are summed through LDS. Weights stream
//    as contiguous 1 KB tiles, one per wave and 64-deep step, each read from
//    HBM once. Bound by HBM.
//  * w8a8_tile_kernel (many rows): a workgroup owns a row x column tile; its
//    waves form WM x WN and each an MB x NB grid of 16 x 16 blocks. Both
//    operands are copied to LDS, one to three k-tiles ahead. Bound by the rate
//    of those copies and by MFMA.
//
// The last k step may be partial: its weight codes past K are zero, so the
// activation codes there may be anything; their addresses are clamped into the
// row.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "w4a16_device.h"
#include "w4a16_launch.h"
#include "w4a16_moe_launch.h"

namespace w4a16_internal {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// LDS slot of piece p of a 128-byte row: conflict-free for the staging writes
// (eight rows a wave) and the fragment reads (sixteen rows, one piece).
__device__ __forceinline__ int t8_slot(int piece, int row) {
  return piece ^ (row & 7) ^ ((row >> 3) & 1);
}

// --------------------------------------------------------------- few rows

// A wave works through pairs of steps (128 k). XS: it loads its rows' 128-byte
// pieces coalesced (8 lanes a row) and turns them into operands through a
// wave-private LDS area; read in operand order, a load's 16 consecutive lanes
// sit in 16 rows, 16 cache lines for 256 bytes.
// ONCE: a single row tile reads the weights.
template <int MB, int NB, int WAVES, bool XS, bool ONCE>
__global__ __launch_bounds__(64 * WAVES) void w8a8_small_kernel(const W8A8Args a, int MT) {
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int c16 = lane & 15, lg = lane >> 4;
  const int S = (a.K + 63) / 64, S2 = (S + 1) / 2, NCB = (a.N + 15) / 16;
  // row tiles of a column tile side by side on one XCD: its L2 serves the
  // others (5120 x 17408, M = 128: 59.7 -> 51.1 us)
  const int tile = xcd_grouped(blockIdx.x, gridDim.x);
  const int b0 = tile / MT * NB, m0 = tile % MT * 16 * MB;
  const int s0 = static_cast<int>(static_cast<long long>(S2) * wave / WAVES);
  const int s1 = static_cast<int>(static_cast<long long>(S2) * (wave + 1) / WAVES);
  extern __shared__ __attribute__((aligned(16))) int q8s_lds[];  // operands, then the waves' sums
  unsigned char* const area = reinterpret_cast<unsigned char*>(q8s_lds) + wave * (MB * 2048);

  gptr<const i32x4> wbase[NB];
  constexpr int XR = XS ? 2 * MB : MB;
  gptr<const uint8_t> xrow[XR];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)  // past the last block: clamped, not stored
    wbase[nb] = reinterpret_cast<gptr<const i32x4>>(
                    to_global(a.qweight) + static_cast<size_t>(min(b0 + nb, NCB - 1)) * S * 1024) + lane;
#pragma unroll
  for (int i = 0; i < XR; ++i) {  // past the last row: repeats it, not stored
    const int r = XS ? 8 * i + lane / 8 : 16 * i + c16;
    xrow[i] = to_global(a.xq) + static_cast<size_t>(min(m0 + r, a.M - 1)) * a.K;
  }

  struct Stage {
    i32x4 w[2][NB], x[2][MB];
  };
  auto load = [&](Stage& st, int s) {
    s = min(s, s1 - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {  // past the last step: re-read, not used
        const auto at = wbase[nb] + static_cast<size_t>(min(2 * s + h, S - 1)) * 64;
        // several row tiles read them: kept in L2 (5120 x 17408, M = 64, two row
        // tiles: 31.4 -> 29.2 us; one row, read once: 17.0 against 18.3)
        st.w[h][nb] = ONCE ? __builtin_nontemporal_load(at) : *at;
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int k = min(128 * s + (XS ? 16 * (lane & 7) : 64 * h + 16 * lg), a.K - 16);
        st.x[h][mb] = *reinterpret_cast<gptr<const i32x4>>(xrow[XS ? 2 * mb + h : mb] + k);
      }
  };
  i32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = i32x4{0, 0, 0, 0};
  auto compute = [&](const Stage& st, int c) {
    if constexpr (XS) {  // rows 16 mb + 8 h + lane / 8, piece lane % 8
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 8 * h + lane / 8;
          *reinterpret_cast<i32x4*>(area + (16 * mb + row) * 128 + t8_slot(lane & 7, row) * 16) = st.x[h][mb];
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * c + h >= S) break;  // uniform: the last pair may have one step
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        i32x4 xa = st.x[h][mb];
        if constexpr (XS)
          xa = *reinterpret_cast<const i32x4*>(area + (16 * mb + c16) * 128 + t8_slot(4 * h + lg, c16) * 16);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_i8(xa, st.w[h][nb], acc[mb][nb]);
      }
    }
  };
  if (s1 > s0) {
    // the next pair's loads are issued before a pair's math, into the other of
    // two register sets (past the last pair: re-read, not used)
    Stage st0, st1;
    load(st0, s0);
    for (int c = s0; c < s1; c += 2) {
      load(st1, c + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(st0, c);
      if (c + 1 < s1) {
        load(st0, c + 2);
        __builtin_amdgcn_sched_barrier(0);
        compute(st1, c + 1);
      }
    }
  }
  if constexpr (XS) __syncthreads();  // the operand areas are no longer read
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        q8s_lds[(((wave * MB + mb) * NB + nb) * 4 + r) * 64 + lane] = acc[mb][nb][r];
  __syncthreads();
  for (int e = threadIdx.x; e < MB * NB * 256; e += 64 * WAVES) {
    const int l = e & 63, r = (e >> 6) & 3, blk = e >> 8;
    const int mb = blk / NB, nb = blk - mb * NB;
    const int m = m0 + 16 * mb + 4 * (l >> 4) + r;
    const int n = (b0 + nb) * 16 + (l & 15);
    if (m >= a.M || n >= a.N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += q8s_lds[(((w * MB + mb) * NB + nb) * 4 + r) * 64 + l];
    to_global(a.y)[static_cast<size_t>(m) * a.N + n] =
        f32_to_bf16_bits(static_cast<float>(sum) * (a.sx[m] * a.sw[n]));
  }
}

template <int MB, int NB, int WAVES, bool XS>
hipError_t launch_small(const W8A8Args& a, hipStream_t stream) {
  const int NCB = (a.N + 15) / 16;
  const size_t lds = static_cast<size_t>(WAVES) * MB * 1024 * (XS && NB < 2 ? 2 : NB);
  int MT = (a.M + 16 * MB - 1) / (16 * MB);
  const long long blocks = static_cast<long long>((NCB + NB - 1) / NB) * MT;
  if (blocks * 64 * WAVES > 0xFFFFFFFFLL) return hipErrorNotSupported;
  // read in operand order there is one row tile
  const void* fn = MT == 1 ? reinterpret_cast<const void*>(&w8a8_small_kernel<MB, NB, WAVES, XS, true>)
                           : reinterpret_cast<const void*>(&w8a8_small_kernel<MB, NB, WAVES, XS, !XS>);
  if (lds >= 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  W8A8Args args = a;
  void* kargs[] = {&args, &MT};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(64 * WAVES), kargs, lds, stream);
}

// -------------------------------------------------------------- many rows

constexpr int kT8KT = 128;  // k per k-tile: two matrix-instruction steps

template <int WM, int WN, int MB, int NB, int BUFS>
struct T8Cfg {
  static constexpr int Waves = WM * WN;
  static constexpr int Threads = 64 * Waves;
  static constexpr int Rows = WM * MB * 16;
  static constexpr int Blocks = WN * NB;                       // 16-column blocks
  static constexpr int Pieces = Rows / 8 + Blocks * 2;         // 1 KB pieces of a k-tile
  static constexpr int Loads = (Pieces + Waves - 1) / Waves;   // per wave
  static constexpr int ABytes = Rows * kT8KT;
  static constexpr int BufBytes = ABytes + Blocks * 2048;
  static constexpr size_t Lds = BUFS * static_cast<size_t>(BufBytes);
  static_assert(Lds <= 160 * 1024, "the buffers fit");
};

typedef int rsrc4 __attribute__((ext_vector_type(4)));

// Buffer descriptor of [base, base + bytes); loads past the end do not fault.
__device__ __forceinline__ rsrc4 raw_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  rsrc4 r;
  r[0] = uniform(static_cast<int>(p));
  r[1] = uniform(static_cast<int>((p >> 32) & 0xFFFFu));
  r[2] = uniform(static_cast<int>(bytes));
  r[3] = 0x00020000;
  return r;
}

// One wave's copy of 64 x 16 bytes from r + voff (per lane) to LDS bytes
// lds .. lds + 1023 (lane l's at 16 l), without passing through registers.
// In inline assembly because the compiler, which cannot tell these LDS bytes
// from others, would wait for every such copy before the next LDS read; the
// loops that use it hold every wait themselves. M0 is named as written, of which
// the compiler warns, as it gives M0 to no value of its own.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(uint32_t lds, uint32_t voff, rsrc4 r) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(r)
      : "m0", "memory");
}
#pragma clang diagnostic pop

// Waits until at most N of the wave's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_vmem_but() {
  static_assert(N < 64, "the counter has six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// A workgroup's tile is (16 MB WM) rows x (16 NB WN) columns; k advances in
// k-tiles of 128. Both operands of a k-tile are copied to one of BUFS LDS
// buffers: activation rows of 128 bytes with their 16-byte pieces permuted by
// t8_slot on the way (the lanes read permuted addresses of the same cache
// lines), weight tiles as they lie. Per k-tile a wave reads 2 (MB + NB)
// operands for 2 MB NB matrix instructions, those of half a k-tile while the
// half before it multiplies. The one barrier per k-tile sits between the
// halves: behind it, every wave has read the current buffer, which is refilled
// with the k-tile BUFS further on, and the next buffer, whose copies were
// issued BUFS - 1 k-tiles earlier, is complete. A compute unit that holds one
// workgroup waits for its copies with two buffers; four instead of two: 7168 x
// 5120, M = 128, 64 x 64 tiles 26.1 -> 14.5 us, M = 512, 128 x 128 33.4 -> 26.2;
// three for 128 x 192: 5120 x 17408, M = 1024 114 -> 92 us, but 176 -> 198 at
// 34816 x 5120, M = 1024, where two workgroups of two buffers share one.
//
// Copies and operand reads are dealt out among the matrix instructions: issued
// in one run, the copies queue up in front of the address unit (16 cycles for
// each KB) and hold back the matrix instructions behind them. At M = 1024, N =
// 34816, K = 5120, 256 x 192 tiles: 188 -> 173 us (2,110 TOP/s; a library
// product of 8192^3 reaches 2,135 on the same card). There the matrix
// instructions alone take 117 us and with the operand reads 135: the copies'
// rate, about 20 bytes a cycle and compute unit, bounds the rest. Copies
// through registers were not faster (189 us).
template <int WM, int WN, int MB, int NB, int BUFS>
__global__ __launch_bounds__(64 * WM * WN, WM * WN / 4) void w8a8_tile_kernel(const W8A8Args a, int MT, int NT) {
  using C = T8Cfg<WM, WN, MB, NB, BUFS>;
  extern __shared__ __attribute__((aligned(16))) unsigned char t8_lds[];
  const int tile = xcd_grouped(blockIdx.x, MT * NT);
  const int mt = tile % MT, nt = tile / MT;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int c16 = lane & 15, lg = lane >> 4;
  const int m0 = mt * C::Rows;
  const int S = (a.K + 63) / 64, NCB = (a.N + 15) / 16, KT = (a.K + kT8KT - 1) / kT8KT;
  const int rows = min(a.M - m0, C::Rows);

  // Piece i of a wave is piece wave + Waves i of the k-tile (past the last:
  // the last again): 8 activation rows, or one block's weight tile of one
  // step. Rows and blocks past the last repeat it (their results are not
  // stored). What lies past the end of K is the next row's codes or zero, and
  // meets zero weights; weight tiles past the last step are not used.
  uint32_t off[C::Loads];
#pragma unroll
  for (int i = 0; i < C::Loads; ++i) {
    const int c = min(wave + C::Waves * i, C::Pieces - 1);
    if (c < C::Rows / 8) {
      const int row = c * 8 + lane / 8;
      off[i] = static_cast<uint32_t>(min(row, rows - 1)) * static_cast<uint32_t>(a.K) + t8_slot(lane & 7, row & 15) * 16;
    } else {
      const int b = c - C::Rows / 8;  // block b / 2, step b % 2
      off[i] = (static_cast<uint32_t>(min(nt * C::Blocks + b / 2, NCB - 1)) * S + b % 2) * 1024u + lane * 16u;
    }
  }
  const uint8_t* xbase = a.xq + static_cast<size_t>(m0) * a.K;
  const uint32_t xbytes = static_cast<uint32_t>(rows) * static_cast<uint32_t>(a.K);
  const uint32_t wbytes = static_cast<uint32_t>(NCB) * static_cast<uint32_t>(S) * 1024u;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) unsigned char*)t8_lds));
  // part g of G of k-tile t's copies, into buffer b
  auto copy = [&](int t, int b, int g, int G) {
    const rsrc4 rx = raw_rsrc(xbase + static_cast<size_t>(t) * kT8KT, xbytes - static_cast<uint32_t>(t) * kT8KT);
    const rsrc4 rw = raw_rsrc(a.qweight + static_cast<size_t>(t) * 2048, wbytes - static_cast<uint32_t>(t) * 2048u);
#pragma unroll
    for (int i = 0; i < C::Loads; ++i) {
      if (i * G / C::Loads != g) continue;
      const int c = min(wave + C::Waves * i, C::Pieces - 1);
      copy_to_lds(lds0 + b * C::BufBytes + c * 1024, off[i], c < C::Rows / 8 ? rx : rw);
    }
  };

  struct Half {
    i32x4 x[MB], w[NB];
  };
  const unsigned char* const xfrag = t8_lds + (wm * MB * 16 + c16) * kT8KT;
  const unsigned char* const wfrag = t8_lds + C::ABytes + wn * NB * 2048 + lane * 16;
  // part g of G of the operands of half s of k-tile t
  auto read = [&](Half& h, int t, int s, int g, int G) {
    const int buf = static_cast<unsigned>(t) % BUFS * C::BufBytes;
#pragma unroll
    for (int i = 0; i < MB + NB; ++i) {
      if (i * G / (MB + NB) != g) continue;
      if (i < NB)
        h.w[i] = *reinterpret_cast<const i32x4*>(wfrag + buf + i * 2048 + s * 1024);
      else
        h.x[i - NB] = *reinterpret_cast<const i32x4*>(xfrag + buf + (i - NB) * 16 * kT8KT + t8_slot(4 * s + lg, c16) * 16);
    }
  };
  i32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = i32x4{0, 0, 0, 0};
  auto multiply = [&](const Half& h, int mb) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_i8(h.w[nb], h.x[mb], acc[mb][nb]);
  };

  Half h0, h1;
#pragma unroll
  for (int i = 0; i < BUFS; ++i) copy(min(i, KT - 1), i, 0, 1);  // past the last: not read
  wait_vmem_but<(BUFS - 1) * C::Loads>();
  lds_barrier();
  read(h0, 0, 0, 0, 1);
  auto tile_of = [&](int t, auto refill) {
#pragma unroll
    for (int g = 0; g < MB; ++g) {
      read(h1, t, 1, g, MB);
      __builtin_amdgcn_sched_barrier(0);
      multiply(h0, g);
      __builtin_amdgcn_sched_barrier(0);
    }
    // k-tile t + 1 has landed, everywhere, and k-tile t has been read
    wait_vmem_but<refill ? (BUFS - 2) * C::Loads : 0>();
    lds_barrier();
#pragma unroll
    for (int g = 0; g < MB; ++g) {
      if constexpr (refill) copy(t + BUFS, static_cast<unsigned>(t) % BUFS, g, MB);
      read(h0, t + 1, 0, g, MB);         // past the last: not used
      __builtin_amdgcn_sched_barrier(0);
      if (2 * t + 1 < S) multiply(h1, g);  // else: the last k-tile has one step
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int t = 0;
  for (; t + BUFS < KT; ++t) tile_of(t, std::true_type{});
  for (; t < KT; ++t) tile_of(t, std::false_type{});

  // The accumulator of lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of
  // its block (the weights are the first operand), so four bf16 go to LDS at
  // once; one row block at a time passes through the wave's own part of LDS
  // and leaves as 16-byte stores of whole row pieces. (Two-byte stores from
  // the registers, 32 bytes of a row together, took 23 us of 211 at M = 1024,
  // N = 34816, K = 5120.)
  __syncthreads();
  constexpr int RowBytes = NB * 32, Stride = RowBytes + 16;  // padded against bank conflicts
  static_assert(C::Waves * 16 * Stride <= static_cast<int>(C::Lds), "the wave parts fit");
  unsigned char* const part = t8_lds + wave * (16 * Stride);
  const int n0 = (nt * C::Blocks + wn * NB) * 16;  // the wave's first column
  f32x4 cs[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int r = 0; r < 4; ++r) cs[nb][r] = to_global(a.sw)[min(n0 + nb * 16 + 4 * lg + r, a.N - 1)];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int row0 = m0 + (wm * MB + mb) * 16;
    const float rs = to_global(a.sx)[min(row0 + c16, a.M - 1)];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      u32x2 o;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float lo = static_cast<float>(acc[mb][nb][2 * q]) * (rs * cs[nb][2 * q]);
        const float hi = static_cast<float>(acc[mb][nb][2 * q + 1]) * (rs * cs[nb][2 * q + 1]);
        o[q] = f32_to_bf16_bits(lo) | static_cast<uint32_t>(f32_to_bf16_bits(hi)) << 16;
      }
      *reinterpret_cast<u32x2*>(part + c16 * Stride + nb * 32 + lg * 8) = o;
    }
    constexpr int Pieces = NB * 2;  // per row
#pragma unroll
    for (int i = 0; i < (16 * Pieces + 63) / 64; ++i) {
      const int e = i * 64 + lane, row = e / Pieces, col = e % Pieces * 8;
      if (e >= 16 * Pieces) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + row * Stride + col * 2);
      if (row0 + row < a.M && n0 + col < a.N)
        store_piece(to_global(a.y) + static_cast<size_t>(row0 + row) * a.N + n0 + col, v, a.N - (n0 + col));
    }
  }
}

template <int WM, int WN, int MB, int NB, int BUFS>
hipError_t launch_tile(const W8A8Args& a, hipStream_t stream) {
  using C = T8Cfg<WM, WN, MB, NB, BUFS>;
  const int NCB = (a.N + 15) / 16;
  int MT = static_cast<int>((static_cast<long long>(a.M) + C::Rows - 1) / C::Rows);
  int NT = (NCB + C::Blocks - 1) / C::Blocks;
  const long long blocks = static_cast<long long>(MT) * NT;
  if (blocks * C::Threads > 0xFFFFFFFFLL) return hipErrorNotSupported;
  const void* fn = reinterpret_cast<const void*>(&w8a8_tile_kernel<WM, WN, MB, NB, BUFS>);
  if (C::Lds >= 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::Lds));
    if (e != hipSuccess) return e;
  }
  W8A8Args args = a;
  void* kargs[] = {&args, &MT, &NT};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(C::Threads), kargs, C::Lds, stream);
}

// The forms, by modelled time. Few rows: a workgroup streams its 16 (rows +
// columns) x K operand bytes after 3 us, at about 45 GB/s where it alone reads
// its weights and 60 GB/s where other row tiles read them too (a fifth less from
// three workgroups per compute unit on), with a fixed cost per step as of eight
// columns; one round of workgroups follows the other, so the smallest rounds x
// columns) is best. Tiles: 3 us and a time per k-tile and round of workgroups;
// 128 x 128 and 128 x 192 hold more buffers while there is one round, and from
// two on two buffers, so that two workgroups share a compute unit. Measured on N
// x K = 7168 x 5120, 5120 x 6144, 34816 x 5120, 5120 x 17408, their eighths, 12000
// x 4096, 2756 x 10368, 21968 x 1408, 710 x 17408 and 1500 x 704 at M = 1 to 4096
// with every form (214 shapes): the one chosen takes 1.003 times the fastest
// measured in the mean and at most 1.13. For instance (us): 5120 x 17408, M = 64: 2 x 3 blocks
// 27.1, 2 x 4 31.3; M = 256: 64 x 128 55, 64 x 64 63, 128 x 128 72; 34816 x 5120, M
// = 64: 128 x 192 37, 64 x 128 50, 2 x 4 blocks 61; M = 512: 128 x 192 98, 256 x
// 192 103; M = 1024: 175, 155; 7168 x 5120, M = 2048: 128 x 192 with two buffers
// 82, with three 92. Forms of 2 x 1, 4 x 2, 4 x 3 and 4 x 4 blocks and of 64 x 192
// gained 1 % or less over these.
enum W8A8Form : int { kS1x1, kS1x2, kS2x2, kS2x3, kS2x4, kT64x64, kT64x128, kT128x128, kT128x128Shared, kT128x192, kT128x192Shared, kT256x192 };
constexpr int kSmallMaxRows = 512;  // few-rows forms are not looked at above

W8A8Form w8a8_form(int M, int N, int K) {
  auto rounds = [&](long long rows, long long cols) {
    const long long tiles = (M + rows - 1) / rows * ((N + cols - 1) / cols);
    return static_cast<double>((tiles + kModelCUs - 1) / kModelCUs);
  };
  const double kt = (K + kT8KT - 1) / kT8KT;
  const struct {
    W8A8Form f;
    int rows, cols;
    double us;          // per k-tile and round
    bool one, several;  // rounds it is for
  } tiles[] = {{kT256x192, 256, 192, 1.1, true, true},         {kT128x192Shared, 128, 192, 0.66, false, true},
               {kT128x192, 128, 192, 0.64, true, false},       {kT128x128Shared, 128, 128, 0.48, false, true},
               {kT128x128, 128, 128, 0.47, true, false},       {kT64x128, 64, 128, 0.34, true, false},
               {kT64x64, 64, 64, 0.24, true, false}};
  const struct {
    W8A8Form f;
    int mb, nb;
  } small[] = {{kS2x4, 2, 4}, {kS2x3, 2, 3}, {kS2x2, 2, 2}, {kS1x2, 1, 2}, {kS1x1, 1, 1}};
  W8A8Form best = kT256x192;
  double t = 1e30;  // of equal ones the first: fewest reads of the operands
  auto consider = [&](W8A8Form f, double us) {
    if (us < t) {
      best = f;
      t = us;
    }
  };
  if (M > 16)
    for (const auto& s : tiles) {
      const double r = rounds(s.rows, s.cols);
      if (r > 1 ? s.several : s.one) consider(s.f, 3.0 + kt * s.us * r);
    }
  if (M <= kSmallMaxRows)
    for (const auto& s : small) {
      if (s.mb > 1 && M <= 8 * s.mb) continue;  // half the row blocks hold as many rows
      const double r = rounds(16 * s.mb, 16 * s.nb);
      const double rows = M < 16 * s.mb ? M : 16 * s.mb;
      consider(s.f, 3.0 + r * (r >= 3 ? 1.2 : 1.0) * (rows + 16 * s.nb + 8) * K / (M > 16 * s.mb ? 60000.0 : 45000.0));
    }
  return best;
}

}  // namespace

hipError_t launch_w8a8(const W8A8Args& a, hipStream_t stream) {
  switch (w8a8_form(a.M, a.N, a.K)) {
    case kS1x1: return launch_small<1, 1, 16, true>(a, stream);
    // read in operand order up to 8 rows: 7.9 against 8.0 us at M = 1, N =
    // 7168, K = 5120, 4.7 against 5.9 at N = 896; at 16 rows 9.4 against 9.1
    case kS1x2: return a.M <= 8 ? launch_small<1, 2, 8, false>(a, stream) : launch_small<1, 2, 8, true>(a, stream);
    case kS2x2: return launch_small<2, 2, 8, true>(a, stream);
    case kS2x3: return launch_small<2, 3, 8, true>(a, stream);
    case kS2x4: return launch_small<2, 4, 8, true>(a, stream);
    case kT64x64: return launch_tile<2, 2, 2, 2, 4>(a, stream);
    case kT64x128: return launch_tile<2, 2, 2, 4, 4>(a, stream);
    case kT128x128: return launch_tile<2, 4, 4, 2, 4>(a, stream);
    case kT128x128Shared: return launch_tile<2, 4, 4, 2, 2>(a, stream);
    case kT128x192: return launch_tile<2, 4, 4, 3, 3>(a, stream);
    case kT128x192Shared: return launch_tile<2, 4, 4, 3, 2>(a, stream);
    default: return launch_tile<4, 2, 4, 6, 2>(a, stream);
  }
}

}  // namespace w4a16_internal

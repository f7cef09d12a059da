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
//    waves form WM x WN and each an MB x NB grid of 16 x 16 blocks.
//    Activations are staged through LDS (double-buffered, XOR-swizzled), the
//    weight tiles go straight into registers. Bound by MFMA.
//
// The last k step may be partial: its weight codes past K are zero, so the
// activation codes there may be anything; their addresses are clamped into the
// row.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "w4a16_device.h"
#include "w4a16_moe_launch.h"

namespace w4a16_internal {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// --------------------------------------------------------------- few rows

template <int MB, int NB, int WAVES, int P>
__global__ __launch_bounds__(64 * WAVES) void w8a8_small_kernel(const W8A8Args a) {
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int c16 = lane & 15, lg = lane >> 4;
  const int S = (a.K + 63) / 64, NCB = (a.N + 15) / 16;
  const int b0 = blockIdx.x * NB, m0 = blockIdx.y * 16 * MB;
  const int s0 = static_cast<int>(static_cast<long long>(S) * wave / WAVES);
  const int s1 = static_cast<int>(static_cast<long long>(S) * (wave + 1) / WAVES);
  extern __shared__ __attribute__((aligned(16))) int q8s_red[];

  gptr<const i32x4> wbase[NB];
  gptr<const uint8_t> xrow[MB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)  // past the last block: clamped, not stored
    wbase[nb] = reinterpret_cast<gptr<const i32x4>>(
                    to_global(a.qweight) + static_cast<size_t>(min(b0 + nb, NCB - 1)) * S * 1024) + lane;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)  // past the last row: repeats it, not stored
    xrow[mb] = to_global(a.xq) + static_cast<size_t>(min(m0 + 16 * mb + c16, a.M - 1)) * a.K;

  struct Stage {
    i32x4 w[NB], x[MB];
  };
  auto load = [&](Stage& st, int s) {
    s = min(s, s1 - 1);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) st.w[nb] = __builtin_nontemporal_load(wbase[nb] + static_cast<size_t>(s) * 64);
    const int k = min(64 * s + 16 * lg, a.K - 16);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) st.x[mb] = *reinterpret_cast<gptr<const i32x4>>(xrow[mb] + k);
  };
  i32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = i32x4{0, 0, 0, 0};
  if (s1 > s0) {
    Stage st[P];
#pragma unroll
    for (int p = 0; p < P; ++p) load(st[p], s0 + p);
    for (int c = s0; c < s1; c += P) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (c + p < s1) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_i8(st[p].x[mb], st[p].w[nb], acc[mb][nb]);
          load(st[p], c + p + P);
        }
    }
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        q8s_red[(((wave * MB + mb) * NB + nb) * 4 + r) * 64 + lane] = acc[mb][nb][r];
  __syncthreads();
  for (int e = threadIdx.x; e < MB * NB * 256; e += 64 * WAVES) {
    const int l = e & 63, r = (e >> 6) & 3, blk = e >> 8;
    const int mb = blk / NB, nb = blk - mb * NB;
    const int m = m0 + 16 * mb + 4 * (l >> 4) + r;
    const int n = (b0 + nb) * 16 + (l & 15);
    if (m >= a.M || n >= a.N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += q8s_red[(((w * MB + mb) * NB + nb) * 4 + r) * 64 + l];
    to_global(a.y)[static_cast<size_t>(m) * a.N + n] =
        f32_to_bf16_bits(static_cast<float>(sum) * (a.sx[m] * a.sw[n]));
  }
}

template <int MB, int NB, int WAVES, int P>
hipError_t launch_small(const W8A8Args& a, hipStream_t stream) {
  const int NCB = (a.N + 15) / 16;
  const size_t lds = static_cast<size_t>(WAVES) * MB * NB * 1024;
  const void* fn = reinterpret_cast<const void*>(&w8a8_small_kernel<MB, NB, WAVES, P>);
  if (lds > 48 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  W8A8Args args = a;
  void* kargs[] = {&args};
  return hipLaunchKernel(fn, dim3((NCB + NB - 1) / NB, (a.M + 16 * MB - 1) / (16 * MB)),
                         dim3(64 * WAVES), kargs, lds, stream);
}

// -------------------------------------------------------------- many rows

constexpr int kT8KT = 128;               // k per k-tile
constexpr int kT8Pieces = kT8KT / 16;    // 16-byte pieces of a row

// LDS slot of piece p of a 128-byte row: conflict-free for the staging writes
// (eight rows a wave) and the fragment reads (sixteen rows, one piece).
__device__ __forceinline__ int t8_slot(int piece, int row) {
  return piece ^ (row & 7) ^ ((row >> 3) & 1);
}

template <int WM, int WN, int MB, int NB>
struct T8Cfg {
  static constexpr int Threads = 64 * WM * WN;
  static constexpr int Rows = WM * MB * 16;
  static constexpr int Blocks = WN * NB;
  static constexpr int Loads = Rows * kT8Pieces / Threads;
  static constexpr int RowStep = Threads / kT8Pieces;
  static constexpr int ABytes = Rows * kT8KT;
  static constexpr size_t Lds = 2 * static_cast<size_t>(ABytes);
};

template <int WM, int WN, int MB, int NB>
__global__ __launch_bounds__(64 * WM * WN, 8 / (WM * WN)) void w8a8_tile_kernel(const W8A8Args a, int MT, int NT) {
  using C = T8Cfg<WM, WN, MB, NB>;
  extern __shared__ __attribute__((aligned(16))) unsigned char t8_lds[];
  const int tile = xcd_grouped(blockIdx.x, MT * NT);
  const int mt = tile % MT, nt = tile / MT;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int c16 = lane & 15, lg = lane >> 4;
  const int m0 = mt * C::Rows;
  const int S = (a.K + 63) / 64, NCB = (a.N + 15) / 16, KT = (a.K + kT8KT - 1) / kT8KT;
  const int spiece = tid % kT8Pieces, srow0 = tid / kT8Pieces;

  const uint8_t* xbase = a.xq + static_cast<size_t>(m0) * a.K;
  const uint32_t xbytes = static_cast<uint32_t>(min(a.M - m0, C::Rows)) * static_cast<uint32_t>(a.K);
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.qweight, static_cast<uint32_t>(NCB) * static_cast<uint32_t>(S) * 1024u);
  uint32_t boff[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
    boff[nb] = static_cast<uint32_t>(min((nt * C::Blocks + wn * NB + nb), NCB - 1)) * S * 1024u;

  u32x4 sr[C::Loads];
  auto stage_load = [&](int t) {
    // rows past the last read as zero; so does a piece past the end of the
    // tile's last row, and one past the end of another row holds the next
    // row's codes, which meet zero weights
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(xbase + t * kT8KT, xbytes - static_cast<uint32_t>(t) * kT8KT);
#pragma unroll
    for (int i = 0; i < C::Loads; ++i)
      sr[i] = __builtin_amdgcn_raw_buffer_load_b128(
          rx, static_cast<uint32_t>(srow0 + i * C::RowStep) * a.K + spiece * 16, 0, 0);
  };
  auto stage_store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < C::Loads; ++i) {
      const int row = srow0 + i * C::RowStep;
      *reinterpret_cast<u32x4*>(t8_lds + buf * C::ABytes + row * kT8KT + t8_slot(spiece, row) * 16) = sr[i];
    }
  };
  struct B {
    i32x4 w[2][NB];
  };
  auto load_b = [&](B& b, int t) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int step = min(2 * t + s, S - 1);  // past the last: re-read, not used
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        b.w[s][nb] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(rq, lane * 16, static_cast<int>(boff[nb] + step * 1024u), 0));
    }
  };
  i32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = i32x4{0, 0, 0, 0};
  auto compute = [&](const B& b, int t, int buf) {
    const unsigned char* base = t8_lds + buf * C::ABytes + (wm * MB * 16 + c16) * kT8KT;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * t + s >= S) break;  // uniform
      i32x4 af[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
        af[mb] = *reinterpret_cast<const i32x4*>(base + mb * 16 * kT8KT + t8_slot(4 * s + lg, c16) * 16);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_i8(af[mb], b.w[s][nb], acc[mb][nb]);
    }
  };

  B b0, b1;
  stage_load(0);
  load_b(b0, 0);
  stage_store(0);
  lds_barrier();
  auto iter = [&](int t, const B& cur, B& nxt) {
    const int tn = t + 1 < KT ? t + 1 : t;
    stage_load(tn);
    load_b(nxt, tn);
    __builtin_amdgcn_sched_barrier(0);  // issue the loads before the math
    compute(cur, t, t & 1);
    stage_store((t & 1) ^ 1);
    lds_barrier();
  };
  for (int t = 0; t < KT; t += 2) {
    iter(t, b0, b1);
    if (t + 1 < KT) iter(t + 1, b1, b0);
  }

  gptr<uint16_t> yg = to_global(a.y);
  float rs[MB][4];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      rs[mb][r] = to_global(a.sx)[min(m0 + (wm * MB + mb) * 16 + 4 * lg + r, a.M - 1)];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int col = (nt * C::Blocks + wn * NB + nb) * 16 + c16;
    if (col >= a.N) continue;
    const float cs = to_global(a.sw)[col];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = m0 + (wm * MB + mb) * 16 + 4 * lg + r;
        if (row < a.M)
          yg[static_cast<size_t>(row) * a.N + col] =
              f32_to_bf16_bits(static_cast<float>(acc[mb][nb][r]) * (rs[mb][r] * cs));
      }
  }
}

template <int WM, int WN, int MB, int NB>
hipError_t launch_tile(const W8A8Args& a, hipStream_t stream) {
  using C = T8Cfg<WM, WN, MB, NB>;
  const int NCB = (a.N + 15) / 16;
  int MT = static_cast<int>((static_cast<long long>(a.M) + C::Rows - 1) / C::Rows);
  int NT = (NCB + C::Blocks - 1) / C::Blocks;
  const long long blocks = static_cast<long long>(MT) * NT;
  if (blocks * C::Threads > 0xFFFFFFFFLL) return hipErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&w8a8_tile_kernel<WM, WN, MB, NB>);
  const hipError_t e =
      hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::Lds));
  if (e != hipSuccess) return e;
  W8A8Args args = a;
  void* kargs[] = {&args, &MT, &NT};
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(C::Threads), kargs, C::Lds, stream);
}

}  // namespace

hipError_t launch_w8a8(const W8A8Args& a, hipStream_t stream) {
  if (a.M <= 16) return launch_small<1, 2, 8, 2>(a, stream);
  if (a.M <= 32) return launch_small<2, 2, 8, 2>(a, stream);
  if (a.M <= 128) return launch_small<4, 2, 8, 2>(a, stream);
  return launch_tile<2, 4, 8, 4>(a, stream);
}

}  // namespace w4a16_internal

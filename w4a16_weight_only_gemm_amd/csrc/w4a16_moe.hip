// w4a16_moe.hip -- routing of tokens to experts, and the weighted sum of the
// experts' rows back into token order.
//
// Routing (w4a16_moe_route). One wave per token: lane l holds the P experts l P
// .. l P + P - 1. Each expert gets an integer key whose order is the order of
// choice; top_k rounds of a wave-wide maximum (DPP, no LDS) take the choices,
// and a ballot finds the first lane that holds it: the lowest index of equal
// ones.
//  * Without bias and groups the choice is by score, which grows with the
//    logit: the key is the logit's own bits, order-preserving. No arithmetic,
//    so nothing can round.
//  * With a bias or groups the choice values are what the interface defines in
//    64 bits: in fp32 two experts a few 1e-8 apart could swap places. They are
//    first formed in fp32; where a decision (a choice against the next one, a
//    group against another) is nearer than a margin that covers every fp32
//    rounding on the way, the token is decided again in fp64. That is one token
//    of some hundreds with a router of 256 experts, and every exact tie.
// The weights need the scores of the chosen experts only, in fp64: lane j
// computes the j-th choice's (softmax without renormalisation also sums over
// all experts, in fp64).
//
// Lists. Slots are ordered by expert and ascending within one, so the result
// does not depend on timing: a workgroup owns a chunk of consecutive tokens,
// counts its slots per expert, and places slot s at (experts before) + (chunks
// before) + (equal slots before s in the chunk). One chunk does all of it in
// one launch; several write their counts, a byte each (a token names an expert
// once), to the workspace, and a second launch sums those of the chunks
// before; more than kRtSumChunks chunks are summed by a launch in between.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "w4a16_device.h"
#include "w4a16_moe_launch.h"

namespace w4a16_internal {
namespace {

constexpr int kRtThreads = 1024;
constexpr int kRtWaves = kRtThreads / 64;
constexpr int kRtMaxExperts = 1024;
// Tokens per workgroup (a wave takes one after the other), by the number of
// tokens. A token takes a wave some 3 to 8 us of dependent steps, so few tokens
// are spread over many workgroups; the second launch reads every chunk's
// counts in every workgroup, so many tokens are not. Measured at 256 experts,
// 8 per token (us, plain top-k / bias and groups):
//   1 token: one workgroup and launch 5.1 / 7.9
//   16 tokens: one workgroup and launch 8.2 / 12.3, 4 per workgroup and two
//     launches 8.6 / 11.3
//   64 tokens: 16 per workgroup 11.3 / 18.8, 4 per workgroup 9.2 / 15.9
//   4096 tokens: 16 per workgroup 14.3 / 22.1, 32 per workgroup 18.3 / 29.1
constexpr int kRtOneLaunchTokens = 8;   // one launch up to here, and up to
constexpr int kRtOneLaunchExperts = 256;
constexpr int kRtFewTokens = 1024;      // up to here 4 tokens and 4 waves
constexpr int kRtFewChunk = 4;
constexpr int kRtMidTokens = 4096;      // up to here 16 tokens
constexpr int kRtMidChunk = 16;
constexpr int kRtChunk = 32;
constexpr int kRtSumChunks = 256;       // up to here the list kernel sums the chunks itself
constexpr int kRtMaxSlots = kRtChunk * 32;  // slots of a chunk (top_k <= 32)

// Order-preserving bits: a < b as numbers iff key(a) < key(b) as unsigned.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double f) {
  const uint64_t b = __builtin_bit_cast(uint64_t, f);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// The number an fp32 key stands for.
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// v of another lane: CTRL as in dpp_f32, for any 4- or 8-byte type; lanes that
// the pattern does not reach (ROWS: the rows written) keep v.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_of(T v) {
  if constexpr (sizeof(T) == 4) {
    const int b = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(b, b, CTRL, ROWS, 0xF, false));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const int lo = static_cast<int>(b), hi = static_cast<int>(b >> 32);
    const uint32_t nlo = __builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xF, false);
    const uint32_t nhi = __builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(T, static_cast<uint64_t>(nhi) << 32 | nlo);
  }
}

// v of lane `src` (uniform) in every lane.
template <typename T>
__device__ __forceinline__ T lane_of(T v, int src) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), src));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), src);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), src);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
  }
}

// Maximum over the wave, in every lane: within quads, half rows and rows of 16
// lanes, then from row to row into lane 63. Lanes a step does not reach meet
// their own value.
template <typename T>
__device__ __forceinline__ T wave_max_of(T v) {
  auto step = [](T a, T b) { return b > a ? b : a; };
  v = step(v, dpp_of<0xB1, 0xF>(v));
  v = step(v, dpp_of<0x4E, 0xF>(v));
  v = step(v, dpp_of<0x141, 0xF>(v));
  v = step(v, dpp_of<0x140, 0xF>(v));
  v = step(v, dpp_of<0x142, 0xA>(v));  // row_bcast 15: rows 1 and 3
  v = step(v, dpp_of<0x143, 0xC>(v));  // row_bcast 31: rows 2 and 3
  return lane_of(v, 63);
}
// Sum over the wave, in every lane, in the order of wave_max_of.
template <typename T>
__device__ __forceinline__ T wave_sum_of(T v) {
  v += dpp_of<0xB1, 0xF>(v);
  v += dpp_of<0x4E, 0xF>(v);
  v += dpp_of<0x141, 0xF>(v);
  v += dpp_of<0x140, 0xF>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, size_t i) {
  if (a.bf16)
    return __builtin_bit_cast(
        float, static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[i]) << 16);
  return static_cast<const float*>(a.logits)[i];
}

// Whether an expert can be chosen (not -inf, not NaN), and its logit with
// +inf as the largest finite value and -0 as 0.
__device__ __forceinline__ bool live_logit(float& v) {
  const bool live = v > -__builtin_inff();
  v = (v > FLT_MAX ? FLT_MAX : v) + 0.0f;
  return live;
}

// Decisions of fp32 choice values nearer than a margin are made again in fp64.
// A sigmoid's score is off by less than 3e-7 whatever the logit (the
// exponential's part that grows with |z| falls as |z| exp(-|z|)), a softmax's
// by 3e-6 of the largest score (exponentials, 22 additions deep, quotient), and
// the bias and a group's sum round at the value's own size. A decision compares
// two values, or two sums of two.
constexpr float kRtMarginSigmoid = 2e-6f;
constexpr float kRtMarginSoftmax = 1.6e-5f;  // of the largest score
constexpr float kRtMarginValue = 5e-7f;      // of the values' magnitude

template <typename S>
__device__ __forceinline__ S exp_of(S x) {
  if constexpr (sizeof(S) == 4)
    return __expf(x);
  else
    return exp(x);
}
template <typename S>
__device__ __forceinline__ S reciprocal(S x) {
  if constexpr (sizeof(S) == 4)
    return __builtin_amdgcn_rcpf(x);  // 1 ulp
  else
    return 1.0 / x;
}

// What a wave knows of a token: the logits of its lane's experts, which of
// them can be chosen, and the largest.
template <int P>
struct Token {
  float z[P];
  bool live[P];
  float zmax;
};

// The top_k largest keys (0: never), one after the other: lane j gets the j-th
// choice (-1 where nothing is left) and its logit. seen(j, key) is called for
// every choice and once more for the best that was left.
template <int P, typename Key, typename F>
__device__ __forceinline__ void take(Key (&key)[P], const Token<P>& tk, int top_k, int lane, int& id,
                                     float& logit, F seen) {
  id = -1;
  logit = 0.f;
  for (int j = 0;; ++j) {
    Key best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < P; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    const Key top = wave_max_of(best);
    if (top == 0) break;
    if (!seen(j, top) || j == top_k) break;
    const int owner = __builtin_ctzll(__ballot(best == top));
    float bz = tk.z[0];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i > 0 && bi == i) bz = tk.z[i];
      if (bi == i && lane == owner) key[i] = 0;
    }
    const int e = owner * P + __builtin_amdgcn_readlane(bi, owner);
    const float ez = lane_of(bz, owner);
    if (lane == j) {
      id = e;
      logit = ez;
    }
  }
}

// Choice by values (bias or groups) in S. Returns whether every decision is
// further than the margin (S = double: always). vals: the wave's LDS.
template <int P, typename S>
__device__ __forceinline__ bool choose_by_value(const RouteArgs& a, const Token<P>& tk, int lane,
                                                S* vals, int& id, float& logit) {
  constexpr bool kCheck = sizeof(S) == 4;
  bool sure = true;
  S margin = kRtMarginSigmoid;
  auto apart = [&](S hi, S lo) {
    if constexpr (!kCheck) return true;
    const S m = hi > -lo ? hi : -lo;  // the larger magnitude, as hi >= lo
    return hi - lo > margin + kRtMarginValue * m;
  };
  S v[P];
  S part = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const S x = tk.z[i];
    v[i] = 0;
    if (tk.live[i]) v[i] = a.sigmoid ? reciprocal<S>(1 + exp_of<S>(-x)) : exp_of<S>(x - static_cast<S>(tk.zmax));
    part += v[i];
  }
  if (!a.sigmoid) {
    const S sum = wave_sum_of(part);  // 0: nothing is live
    margin = kRtMarginSoftmax / sum;  // the largest score is 1 / sum
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = tk.live[i] ? v[i] / sum : 0;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane * P + i;
    if (a.bias && e < a.E) v[i] += static_cast<S>(a.bias[e]);
  }
  typename std::conditional<kCheck, uint32_t, uint64_t>::type key[P];
#pragma unroll
  for (int i = 0; i < P; ++i) key[i] = tk.live[i] ? order_key(v[i]) : 0;
  if (a.groups > 1) {
    // a group's two largest values, by lg lanes (a power of two) each
    const S none = -static_cast<S>(__builtin_inff());
    S t1 = none, t2 = none;
    auto put = [&](S x) {
      t2 = x > t1 ? t1 : x > t2 ? x : t2;
      t1 = x > t1 ? x : t1;
    };
    const int per = a.per, lg = a.group_lanes, g = lane / lg;
    if (a.group_whole) {  // the lanes that hold the group's experts
#pragma unroll
      for (int i = 0; i < P; ++i) put(tk.live[i] ? v[i] : none);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (lane * P + i < a.E) vals[lane * P + i] = tk.live[i] ? v[i] : none;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (g < a.groups)
        for (int j = lane % lg; j < per; j += lg) put(vals[g * per + j]);
    }
    for (int o = 1; o < lg; o <<= 1) {
      const S o1 = __shfl_xor(t1, o), o2 = __shfl_xor(t2, o);
      const S lo = t1 < o1 ? t1 : o1, hi2 = t2 > o2 ? t2 : o2;
      t1 = t1 > o1 ? t1 : o1;
      t2 = lo > hi2 ? lo : hi2;
    }
    S value = t1;
    if (a.group_top == 2 && t2 > none) value = t1 + t2;
    int rank = 0;
    bool near = false;
    for (int q = 0; q < a.groups; ++q) {
      const S ov = lane_of(value, q * lg);
      if (ov > value || (ov == value && q < g)) ++rank;
      if (kCheck && q != g && value > none && ov > none)
        near |= !(ov > value ? apart(ov, value) : apart(value, ov));
    }
    sure = !__any(g < a.groups && near);
    const uint64_t kept = __ballot(g < a.groups && rank < a.groups_kept);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane * P + i;
      const int eg = a.group_whole ? g : static_cast<int>(__umulhi(e, a.per_inverse));  // e / per
      if (e < a.E && !((kept >> (eg * lg)) & 1)) key[i] = 0;
    }
  }
  if (!sure) return false;
  S last = 0;
  take<P>(key, tk, a.top_k, lane, id, logit, [&](int j, auto k) {
    if constexpr (kCheck) {
      const S x = value_of(k);
      if (j > 0 && !apart(last, x)) sure = false;
      last = x;
      return sure;
    } else {
      return j < a.top_k;
    }
  });
  return sure;
}

// The choices of token t, by one wave. P: experts per lane. WIDE: bias or
// groups. vals: this wave's LDS for E choice values (WIDE). Lane j < top_k
// returns the j-th choice (or -1) in id and its weight.
template <int P, bool WIDE>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int lane, double* vals, int& id,
                                       float& weight) {
  const size_t row = static_cast<size_t>(t) * a.E;
  Token<P> tk;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane * P + i;
    tk.z[i] = e < a.E ? load_logit(a, row + e) : -__builtin_inff();
  }
#pragma unroll
  for (int i = 0; i < P; ++i) tk.live[i] = live_logit(tk.z[i]);
  tk.zmax = -FLT_MAX;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < P; ++i) tk.zmax = tk.live[i] && tk.z[i] > tk.zmax ? tk.z[i] : tk.zmax;
    tk.zmax = wave_max_of(tk.zmax);
  }
  float logit;
  if constexpr (WIDE) {
    if (!choose_by_value<P, float>(a, tk, lane, reinterpret_cast<float*>(vals), id, logit))
      choose_by_value<P, double>(a, tk, lane, vals, id, logit);
  } else {
    uint32_t key[P];
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = tk.live[i] ? order_key(tk.z[i]) : 0;
    take<P>(key, tk, a.top_k, lane, id, logit, [&](int j, uint32_t) { return j < a.top_k; });
  }
  double s = 0.0;
  if (id >= 0)
    s = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(logit)))
                  : exp(static_cast<double>(logit) - tk.zmax);
  double total = 1.0;
  if (a.renormalize) {  // the softmax's own sum cancels
    total = wave_sum_of(s);
  } else if (!a.sigmoid) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (tk.live[i]) part += exp(static_cast<double>(tk.z[i]) - tk.zmax);
    total = wave_sum_of(part);
  }
  weight = total > 0.0 ? static_cast<float>(s * static_cast<double>(a.scale) / total) : 0.f;
}

struct RouteLds {
  alignas(16) int ids[kRtMaxSlots];  // this chunk's, in whole groups of four
  int count[kRtMaxExperts];          // this chunk's slots per expert
  int total[kRtMaxExperts];          // all chunks'
  int before[kRtMaxExperts];         // the chunks' before this one; then the place of the first slot
  int wave[kRtWaves];
};

// Exclusive prefix sum of v over the workgroup's threads, and the total.
__device__ __forceinline__ int block_prefix(int v, int* wave_sums, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  if (lane == 63) wave_sums[wave] = s;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRtWaves; ++w) {
    const int x = wave_sums[w];
    if (w < wave) base += x;
    all += x;
  }
  total = all;
  return base + s - v;
}

// Bytes of a chunk's row of counts.
__host__ __device__ constexpr int count_stride(int E) { return (E + 3) / 4 * 4; }

// Places the chunk's slots, given ids, total and before per expert in
// lds (every thread of the workgroup; `n` slots from global slot `first`).
__device__ __forceinline__ void place(const RouteArgs& a, RouteLds& l, int n, int first,
                                      int chunk) {
  const int tid = threadIdx.x;
  const int mine = tid < a.E ? l.total[tid] : 0;
  int routed;
  const int start = block_prefix(mine, l.wave, routed);
  if (tid < a.E) l.before[tid] += start;
  if (chunk == 0) {
    if (tid < a.E) a.offsets[tid] = start;
    if (tid == 0) a.offsets[a.E] = routed;
  }
  __syncthreads();
  // four lanes a slot count equal slots before it, four at a time
  const int sub = tid & 3;
  for (int s0 = 0; s0 < n; s0 += kRtThreads / 4) {
    const int s = s0 + tid / 4;
    const int e = s < n ? l.ids[s] : -1;
    int rank = 0;
    if (e >= 0)
      for (int q = 4 * sub; q < s; q += 16) {
        const int4 v = *reinterpret_cast<const int4*>(l.ids + q);
        rank += (v.x == e) + (v.y == e && q + 1 < s) + (v.z == e && q + 2 < s) + (v.w == e && q + 3 < s);
      }
    rank += __shfl_xor(rank, 1);
    rank += __shfl_xor(rank, 2);
    if (e >= 0 && sub == 0) a.rows[l.before[e] + rank] = first + s;
  }
  const int slots = a.T * a.top_k;
  for (long long p = static_cast<long long>(routed) + chunk * kRtThreads + tid; p < slots;
       p += static_cast<long long>(a.chunks) * kRtThreads)
    a.rows[p] = -1;
}

// One workgroup of W waves per chunk of tokens. ONE: the only chunk, lists and
// all (16 waves).
template <int P, bool WIDE, bool ONE, int W>
__global__ __launch_bounds__(64 * W) void route_kernel(const RouteArgs a) {
  static_assert(!ONE || 64 * W == kRtThreads, "place() takes the whole workgroup");
  __shared__ RouteLds l;
  extern __shared__ __attribute__((aligned(16))) double rt_vals[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * a.chunk;
  const int tokens = min(a.chunk, a.T - t0);
  for (int e = tid; e < count_stride(a.E); e += 64 * W) l.count[e] = 0;
  __syncthreads();
  for (int i = wave; i < tokens; i += W) {
    int id;
    float w;
    choose<P, WIDE>(a, t0 + i, lane, rt_vals + static_cast<size_t>(wave) * a.E, id, w);
    if (lane < a.top_k) {
      const size_t s = static_cast<size_t>(t0 + i) * a.top_k + lane;
      a.ids[s] = id;
      a.weights[s] = w;
      if constexpr (ONE) l.ids[i * a.top_k + lane] = id;
      if (id >= 0) atomicAdd(&l.count[id], 1);  // integer sums: the order does not matter
    }
  }
  __syncthreads();
  if constexpr (ONE) {
    if (tid < a.E) {
      l.total[tid] = l.count[tid];
      l.before[tid] = 0;
    }
    __syncthreads();
    place(a, l, tokens * a.top_k, 0, 0);
  } else {
    const int words = count_stride(a.E) / 4;
    for (int i = tid; i < words; i += 64 * W)
      reinterpret_cast<uint32_t*>(a.counts)[static_cast<size_t>(blockIdx.x) * words + i] =
          l.count[4 * i] | l.count[4 * i + 1] << 8 | l.count[4 * i + 2] << 16 |
          static_cast<uint32_t>(l.count[4 * i + 3]) << 24;
  }
}

// For many chunks: the counts of the chunks before each chunk, and behind the
// last the totals, as ints; a workgroup per 16 experts, 64 runs of chunks each.
__global__ __launch_bounds__(kRtThreads) void route_scan_kernel(const RouteArgs a) {
  __shared__ int part[64][17];
  const int ex = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + ex, stride = count_stride(a.E);
  const int c0 = static_cast<int>(static_cast<long long>(a.chunks) * seg / 64);
  const int c1 = static_cast<int>(static_cast<long long>(a.chunks) * (seg + 1) / 64);
  int sum = 0;
  if (e < a.E)
    for (int c = c0; c < c1; ++c) sum += a.counts[static_cast<size_t>(c) * stride + e];
  part[seg][ex] = sum;
  __syncthreads();
  int run = 0;
  for (int s = 0; s < seg; ++s) run += part[s][ex];
  if (e >= a.E) return;
  for (int c = c0; c < c1; ++c) {
    a.sums[static_cast<size_t>(c) * a.E + e] = run;
    run += a.counts[static_cast<size_t>(c) * stride + e];
  }
  if (seg == 63) a.sums[static_cast<size_t>(a.chunks) * a.E + e] = run;
}

// The lists, from the chunks' counts. SCANNED: route_scan_kernel has run.
template <bool SCANNED>
__global__ __launch_bounds__(kRtThreads) void route_list_kernel(const RouteArgs a) {
  __shared__ RouteLds l;
  const int tid = threadIdx.x, c = blockIdx.x;
  const int t0 = c * a.chunk;
  const int n = min(a.chunk, a.T - t0) * a.top_k;
  const int first = t0 * a.top_k;
  for (int s = tid; s < n; s += kRtThreads) l.ids[s] = a.ids[static_cast<size_t>(first) + s];
  if constexpr (SCANNED) {
    if (tid < a.E) {
      l.before[tid] = a.sums[static_cast<size_t>(c) * a.E + tid];
      l.total[tid] = a.sums[static_cast<size_t>(a.chunks) * a.E + tid];
    }
  } else {
    if (tid < count_stride(a.E)) l.before[tid] = l.total[tid] = 0;
    __syncthreads();
    // four experts (one word of a chunk's counts) per thread, the chunks dealt
    // out over the threads left
    const int words = count_stride(a.E) / 4;
    int width = 1;
    while (width < words) width <<= 1;
    const int wd = tid & (width - 1), step = kRtThreads / width;
    if (wd < words) {
      int tot[4] = {0, 0, 0, 0}, bef[4] = {0, 0, 0, 0};
      const uint32_t* h = reinterpret_cast<const uint32_t*>(a.counts) + wd;
#pragma unroll 8
      for (int r = tid / width; r < a.chunks; r += step) {
        const uint32_t v = h[static_cast<size_t>(r) * words];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = (v >> (8 * i)) & 255;
          tot[i] += x;
          bef[i] += r < c ? x : 0;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (tot[i]) atomicAdd(&l.total[4 * wd + i], tot[i]);
        if (bef[i]) atomicAdd(&l.before[4 * wd + i], bef[i]);
      }
    }
  }
  __syncthreads();
  place(a, l, n, first, c);
}

int experts_per_lane(int E) {
  int p = 1;
  while (64 * p < E) p *= 2;
  return p;
}
bool route_one(int T, int E) { return T <= kRtOneLaunchTokens && E <= kRtOneLaunchExperts; }
int route_chunk(int T) { return T <= kRtFewTokens ? kRtFewChunk : T <= kRtMidTokens ? kRtMidChunk : kRtChunk; }
int route_chunks(int T) {
  const long long n = (static_cast<long long>(T) + route_chunk(T) - 1) / route_chunk(T);
  return n > 0 ? static_cast<int>(n) : 1;  // no tokens: one workgroup writes the offsets
}
// Workspace: the chunks' counts, then (many chunks) their running sums.
size_t counts_bytes(int T, int E) {
  return (static_cast<size_t>(route_chunks(T)) * count_stride(E) + 15) / 16 * 16;
}

template <int P, bool WIDE, bool ONE, int W>
hipError_t launch_route_t(RouteArgs a, hipStream_t stream) {
  const size_t lds = WIDE && a.groups > 1 && !a.group_whole ? static_cast<size_t>(W) * a.E * 8 : 0;
  const void* fn = reinterpret_cast<const void*>(&route_kernel<P, WIDE, ONE, W>);
  if (lds > 32 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  void* kargs[] = {&a};
  return hipLaunchKernel(fn, dim3(a.chunks), dim3(64 * W), kargs, lds, stream);
}

template <int P, bool WIDE>
hipError_t launch_route_p(RouteArgs a, hipStream_t stream) {
  if constexpr (P * 64 <= kRtOneLaunchExperts) {
    if (route_one(a.T, a.E)) return launch_route_t<P, WIDE, true, 16>(a, stream);
  }
  // 8 and more experts per lane need the registers of fewer waves
  constexpr int W = P <= 4 ? 16 : 8;
  hipError_t e = a.chunk == kRtFewChunk ? launch_route_t<P, WIDE, false, kRtFewChunk>(a, stream)
                                        : launch_route_t<P, WIDE, false, W>(a, stream);
  if (e != hipSuccess) return e;
  void* kargs[] = {&a};
  const bool scan = a.chunks > kRtSumChunks;
  if (scan) {
    e = hipLaunchKernel(reinterpret_cast<const void*>(&route_scan_kernel), dim3((a.E + 15) / 16),
                        dim3(kRtThreads), kargs, 0, stream);
    if (e != hipSuccess) return e;
  }
  const void* fn = scan ? reinterpret_cast<const void*>(&route_list_kernel<true>)
                        : reinterpret_cast<const void*>(&route_list_kernel<false>);
  return hipLaunchKernel(fn, dim3(a.chunks), dim3(kRtThreads), kargs, 0, stream);
}

template <bool WIDE>
hipError_t launch_route_w(const RouteArgs& a, hipStream_t stream) {
  switch (experts_per_lane(a.E)) {
    case 1: return launch_route_p<1, WIDE>(a, stream);
    case 2: return launch_route_p<2, WIDE>(a, stream);
    case 4: return launch_route_p<4, WIDE>(a, stream);
    case 8: return launch_route_p<8, WIDE>(a, stream);
    default: return launch_route_p<16, WIDE>(a, stream);
  }
}

// ------------------------------------------------------------------ combine

constexpr int kCbThreads = 256;

// VEC consecutive columns of one token per thread: 8 (16-byte accesses) where
// the rows keep that alignment (N % 8 == 0), else 1.
template <int VEC>
__global__ __launch_bounds__(kCbThreads) void combine_kernel(const CombineArgs a) {
  typedef uint16_t vec __attribute__((ext_vector_type(VEC)));
  const int per = (a.N + VEC - 1) / VEC;
  const long long all = static_cast<long long>(per) * a.T;
  const long long step = static_cast<long long>(gridDim.x) * kCbThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kCbThreads + threadIdx.x; i < all; i += step) {
    const int t = static_cast<int>(i / per);
    const int n = static_cast<int>(i - static_cast<long long>(t) * per) * VEC;
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
    const size_t at = static_cast<size_t>(t) * a.N + n;
    if (a.base) {
      const vec b = *reinterpret_cast<const vec*>(a.base + at);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        acc[v] = __builtin_bit_cast(float, static_cast<uint32_t>(b[v]) << 16);
    }
    const size_t slot0 = static_cast<size_t>(t) * a.top_k;
#pragma unroll 4
    for (int j = 0; j < a.top_k; ++j) {
      if (a.ids[slot0 + j] < 0) continue;
      const float w = a.weights[slot0 + j];
      const vec y = *reinterpret_cast<const vec*>(a.y + (slot0 + j) * a.N + n);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        acc[v] = __builtin_fmaf(w, __builtin_bit_cast(float, static_cast<uint32_t>(y[v]) << 16), acc[v]);
    }
    vec o;
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = f32_to_bf16_bits(acc[v]);
    *reinterpret_cast<vec*>(a.out + at) = o;
  }
}

}  // namespace

size_t route_workspace_bytes(int T, int E) {
  if (route_one(T, E)) return 0;
  size_t n = counts_bytes(T, E);
  if (route_chunks(T) > kRtSumChunks) n += (static_cast<size_t>(route_chunks(T)) + 1) * E * sizeof(int);
  return n;
}

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  a.chunk = route_one(a.T, a.E) ? kRtOneLaunchTokens : route_chunk(a.T);
  a.chunks = route_one(a.T, a.E) ? 1 : route_chunks(a.T);
  a.per = a.E / a.groups;
  a.per_inverse = static_cast<uint32_t>(0xFFFFFFFFu / a.per + 1);  // not used for one expert per group (then whole)
  const int held = experts_per_lane(a.E);
  a.group_lanes = a.per / held;
  a.group_whole = a.per % held == 0 && (a.group_lanes & (a.group_lanes - 1)) == 0;
  if (!a.group_whole) {
    a.group_lanes = 64;
    while (a.group_lanes * a.groups > 64) a.group_lanes >>= 1;
  }
  a.counts = static_cast<uint8_t*>(a.workspace);
  a.sums = a.workspace ? reinterpret_cast<int*>(a.counts + counts_bytes(a.T, a.E)) : nullptr;
  return a.bias || a.groups > 1 ? launch_route_w<true>(a, stream) : launch_route_w<false>(a, stream);
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  const int vec = a.N % 8 == 0 ? 8 : 1;
  const long long threads = static_cast<long long>(a.T) * ((a.N + vec - 1) / vec);
  long long blocks = (threads + kCbThreads - 1) / kCbThreads;
  if (blocks > 1 << 20) blocks = 1 << 20;  // the rest by grid stride
  CombineArgs args = a;
  void* kargs[] = {&args};
  const void* fn = vec == 8 ? reinterpret_cast<const void*>(&combine_kernel<8>)
                            : reinterpret_cast<const void*>(&combine_kernel<1>);
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kCbThreads), kargs, 0, stream);
}

}  // namespace w4a16_internal

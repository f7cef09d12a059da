// w4a16_moe.hip -- routing of tokens to experts, and the weighted sum of the
// experts' rows back into token order.
//
// Routing (w4a16_moe_route). One wave per token: lane l holds experts l, l +
// 64, ... Each expert gets a 64-bit key whose unsigned order is the order of
// choice, and top_k rounds of a wave-wide maximum take the choices.
//  * Without bias and groups the choice is by score, which grows with the
//    logit: the key is the logit's own bits, order-preserving, above the
//    complement of the index. No arithmetic, so nothing can round, and equal
//    logits go to the lowest index.
//  * With a bias or groups the choice values are formed in fp64. In fp32 two
//    experts a few 1e-8 apart could swap places with another order of the
//    same operations; a router of 256 experts meets such a pair in about one
//    token of ten thousand.
// The weights need the scores of the chosen experts only: lane j computes the
// j-th choice's (softmax without renormalisation, or with bias or groups, also
// sums over all experts).
//
// Lists. Slots are ordered by expert and ascending within one, so the result
// does not depend on timing: a workgroup owns a chunk of consecutive tokens,
// counts its slots per expert, and places slot s at (experts before) + (chunks
// before) + (equal slots before s in the chunk). One chunk does all of it in
// one launch; several write their counts to the workspace and a second launch
// sums those of the chunks before; more than kRouteSumChunks chunks sum them
// with a launch of their own in between.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "w4a16_device.h"
#include "w4a16_moe_launch.h"

namespace w4a16_internal {
namespace {

constexpr int kRtThreads = 1024;
constexpr int kRtWaves = kRtThreads / 64;
constexpr int kRtMaxExperts = 1024;
constexpr int kRtOneLaunchTokens = 32;  // at most this many tokens: one workgroup, one launch
constexpr int kRtChunk = 32;            // tokens per workgroup otherwise
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

template <typename T>
__device__ __forceinline__ T wave_max_of(T v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const T u = __shfl_xor(v, o);
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ double wave_sum_of(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
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

// The choices of token t, by one wave. P: experts per lane. WIDE: bias or
// groups. vals: this wave's LDS for E choice values (WIDE). Lane j < top_k
// returns the j-th choice (or -1) in id and its weight.
template <int P, bool WIDE>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int lane, double* vals, int& id,
                                       float& weight) {
  const size_t row = static_cast<size_t>(t) * a.E;
  float z[P];
  bool live[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = i * 64 + lane;
    z[i] = e < a.E ? load_logit(a, row + e) : -__builtin_inff();
    live[i] = live_logit(z[i]);
  }
  // softmax: the largest logit and the sum over all experts
  float zmax = -FLT_MAX;
  double sum = 1.0;
  const bool all = !a.sigmoid && (WIDE || !a.renormalize);
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < P; ++i) zmax = live[i] && z[i] > zmax ? z[i] : zmax;
    zmax = wave_max_of(zmax);
  }
  double score[P];
  if (WIDE || all) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      score[i] = 0.0;
      if (live[i]) {
        if (a.sigmoid)
          score[i] = 1.0 / (1.0 + exp(-static_cast<double>(z[i])));
        else
          score[i] = exp(static_cast<double>(z[i]) - zmax);
      }
      part += score[i];
    }
    if (all) {
      sum = wave_sum_of(part);
      if (sum == 0.0) sum = 1.0;  // nothing live
    }
  }
  uint64_t key[P];
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = i * 64 + lane;
      const double s = a.sigmoid ? score[i] : score[i] / sum;
      const double v = s + (a.bias && e < a.E ? static_cast<double>(a.bias[e]) : 0.0);
      key[i] = live[i] ? order_key(v) : 0;
      if (a.groups > 1 && e < a.E) vals[e] = live[i] ? v : -__builtin_inf();
    }
    if (a.groups > 1) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      // lg lanes (a power of two) per group; each scans part of it
      int lg = 64;
      while (lg * a.groups > 64) lg >>= 1;
      const int per = a.E / a.groups, g = lane / lg;
      double t1 = -__builtin_inf(), t2 = t1;
      if (g < a.groups)
        for (int j = lane % lg; j < per; j += lg) {
          const double v = vals[g * per + j];
          t2 = v > t1 ? t1 : v > t2 ? v : t2;
          t1 = v > t1 ? v : t1;
        }
      for (int o = 1; o < lg; o <<= 1) {
        const double o1 = __shfl_xor(t1, o), o2 = __shfl_xor(t2, o);
        const double lo = t1 < o1 ? t1 : o1, hi2 = t2 > o2 ? t2 : o2;
        t1 = t1 > o1 ? t1 : o1;
        t2 = lo > hi2 ? lo : hi2;
      }
      double value = t1;
      if (a.group_top == 2 && t2 > -__builtin_inf()) value = t1 + t2;
      int rank = 0;
      for (int q = 0; q < a.groups; ++q) {
        const double ov = __shfl(value, q * lg);
        if (ov > value || (ov == value && q < g)) ++rank;
      }
      const uint64_t kept = __ballot(g < a.groups && rank < a.groups_kept);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int e = i * 64 + lane;
        if (e < a.E && !((kept >> (e / per * lg)) & 1)) key[i] = 0;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i)
      key[i] = live[i] ? static_cast<uint64_t>(order_key(z[i])) << 32 |
                             (0xFFFFFFFFu - static_cast<uint32_t>(i * 64 + lane))
                       : 0;
  }
  id = -1;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = key[0];
    int be = lane;
#pragma unroll
    for (int i = 1; i < P; ++i)
      if (key[i] > best) {
        best = key[i];
        be = i * 64 + lane;
      }
    const uint64_t top = wave_max_of(best);
    if (top == 0) break;
    const uint64_t owners = __ballot(best == top);
    int e;
    if (__popcll(owners) == 1) {
      e = __builtin_amdgcn_readlane(be, __builtin_ctzll(owners));
    } else {  // equal choice values (WIDE): the lowest index
      int c = best == top ? -be : -kRtMaxExperts;
      e = -wave_max_of(c);
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i * 64 + lane == e) key[i] = 0;
    if (lane == j) id = e;
  }
  double s = 0.0;
  if (id >= 0) {
    float v = load_logit(a, row + id);
    live_logit(v);
    s = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v)))
                  : exp(static_cast<double>(v) - zmax) / sum;
  }
  if (a.renormalize) {
    const double total = wave_sum_of(s);
    s = total > 0.0 ? s / total : 0.0;
  }
  weight = static_cast<float>(s * static_cast<double>(a.scale));
}

struct RouteLds {
  int ids[kRtMaxSlots];
  int count[kRtMaxExperts];   // this chunk's slots per expert
  int total[kRtMaxExperts];   // all chunks'
  int before[kRtMaxExperts];  // the chunks' before this one; then the place of the first slot
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

// Places the chunk's slots, given total and before per expert in lds (every
// thread of the workgroup; `n` slots from global slot `first`).
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
  for (int s = tid; s < n; s += kRtThreads) {
    const int e = l.ids[s];
    if (e < 0) continue;
    int rank = 0;
    for (int q = 0; q < s; ++q) rank += l.ids[q] == e;
    a.rows[l.before[e] + rank] = first + s;
  }
  const int slots = a.T * a.top_k;
  for (long long p = static_cast<long long>(routed) + chunk * kRtThreads + tid; p < slots;
       p += static_cast<long long>(a.chunks) * kRtThreads)
    a.rows[p] = -1;
}

// One workgroup per chunk of tokens. ONE: the only chunk, lists and all.
template <int P, bool WIDE, bool ONE>
__global__ __launch_bounds__(kRtThreads) void route_kernel(const RouteArgs a) {
  __shared__ RouteLds l;
  extern __shared__ __attribute__((aligned(16))) double rt_vals[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * a.chunk;
  const int tokens = min(a.chunk, a.T - t0);
  if (tid < a.E) l.count[tid] = 0;
  __syncthreads();
  for (int i = wave; i < tokens; i += kRtWaves) {
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
    if (tid < a.E) a.hist[static_cast<size_t>(blockIdx.x) * a.E + tid] = l.count[tid];
  }
}

// Counts of the chunks before each chunk, in place, and the totals behind them
// (for many chunks): a workgroup per 16 experts, 64 runs of chunks each.
__global__ __launch_bounds__(kRtThreads) void route_scan_kernel(const RouteArgs a) {
  __shared__ int part[64][17];
  const int ex = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + ex;
  const int c0 = static_cast<int>(static_cast<long long>(a.chunks) * seg / 64);
  const int c1 = static_cast<int>(static_cast<long long>(a.chunks) * (seg + 1) / 64);
  int sum = 0;
  if (e < a.E)
    for (int c = c0; c < c1; ++c) sum += a.hist[static_cast<size_t>(c) * a.E + e];
  part[seg][ex] = sum;
  __syncthreads();
  int run = 0;
  for (int s = 0; s < seg; ++s) run += part[s][ex];
  if (e >= a.E) return;
  for (int c = c0; c < c1; ++c) {
    int* h = a.hist + static_cast<size_t>(c) * a.E + e;
    const int v = *h;
    *h = run;
    run += v;
  }
  if (seg == 63) a.hist[static_cast<size_t>(a.chunks) * a.E + e] = run;
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
      l.before[tid] = a.hist[static_cast<size_t>(c) * a.E + tid];
      l.total[tid] = a.hist[static_cast<size_t>(a.chunks) * a.E + tid];
    }
  } else {
    if (tid < a.E) l.before[tid] = l.total[tid] = 0;
    __syncthreads();
    int width = 64;
    while (width < a.E) width <<= 1;
    const int e = tid & (width - 1);
    if (e < a.E) {
      int tot = 0, bef = 0;
#pragma unroll 4
      for (int r = tid / width; r < a.chunks; r += kRtThreads / width) {
        const int v = a.hist[static_cast<size_t>(r) * a.E + e];
        tot += v;
        bef += r < c ? v : 0;
      }
      atomicAdd(&l.total[e], tot);
      atomicAdd(&l.before[e], bef);
    }
  }
  __syncthreads();
  place(a, l, n, first, c);
}

int route_chunks(int T) { return static_cast<int>((static_cast<long long>(T) + kRtChunk - 1) / kRtChunk); }

template <int P, bool WIDE>
hipError_t launch_route_t(RouteArgs a, hipStream_t stream) {
  const size_t lds = WIDE && a.groups > 1 ? static_cast<size_t>(kRtWaves) * a.E * 8 : 0;
  void* kargs[] = {&a};
  const bool one = a.T <= kRtOneLaunchTokens;
  const void* fn = one ? reinterpret_cast<const void*>(&route_kernel<P, WIDE, true>)
                       : reinterpret_cast<const void*>(&route_kernel<P, WIDE, false>);
  if (lds > 32 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  hipError_t e = hipLaunchKernel(fn, dim3(a.chunks), dim3(kRtThreads), kargs, lds, stream);
  if (e != hipSuccess || one) return e;
  const bool scan = a.chunks > kRtSumChunks;
  if (scan) {
    e = hipLaunchKernel(reinterpret_cast<const void*>(&route_scan_kernel), dim3((a.E + 15) / 16),
                        dim3(kRtThreads), kargs, 0, stream);
    if (e != hipSuccess) return e;
  }
  fn = scan ? reinterpret_cast<const void*>(&route_list_kernel<true>)
            : reinterpret_cast<const void*>(&route_list_kernel<false>);
  return hipLaunchKernel(fn, dim3(a.chunks), dim3(kRtThreads), kargs, 0, stream);
}

template <bool WIDE>
hipError_t launch_route_w(const RouteArgs& a, hipStream_t stream) {
  if (a.E <= 64) return launch_route_t<1, WIDE>(a, stream);
  if (a.E <= 128) return launch_route_t<2, WIDE>(a, stream);
  if (a.E <= 256) return launch_route_t<4, WIDE>(a, stream);
  if (a.E <= 512) return launch_route_t<8, WIDE>(a, stream);
  return launch_route_t<16, WIDE>(a, stream);
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
  if (T <= kRtOneLaunchTokens) return 0;
  return (static_cast<size_t>(route_chunks(T)) + 1) * E * sizeof(int);
}

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  a.chunk = kRtChunk;
  a.chunks = a.T <= kRtOneLaunchTokens ? 1 : route_chunks(a.T);
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

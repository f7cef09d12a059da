// w4a16_moe_layer.hip -- a whole mixture-of-experts layer for up to 16 tokens.
//
//     z = x Wr^T,  (experts, weights) = choice(z),
//     h_j = silu(x G_e) * (x U_e),  out = base + sum_j w_j (h_j D_e)
//
// Few tokens make every expert's product a stream of its weights: with at most 16
// tokens an expert has at most 16 rows, one row block of the matrix instruction,
// whose row t is token t whatever the expert. So no rows are gathered, and what a
// wave needs of the activations does not depend on the expert.
//  * router_kernel: a workgroup per expert, products and sums in fp64 (a bf16 by f32
//    product is exact there), so that the choice does not depend on an order of
//    additions. It also clears down_kernel's counters.
//  * choose_kernel: a workgroup per token chooses its experts from the logits, where that
//    is not done by every workgroup of gate_up_kernel (choose_inside).
//  * gate_up_kernel: a wave owns a range of K and holds its tokens' activations of that
//    range in registers, while the weights of one (expert, 16 gate and 16 up columns)
//    after the other stream by, a whole task ahead. The waves' sums meet in LDS, where
//    SwiGLU is formed. 13 tokens of 128 experts, 5120 x 1024: 393 MB in 60 to 64 us.
//    SwiGLU's values are stored as two bf16 (down_kernel says why).
//  * down_kernel: the active experts' k ranges laid end to end are one long sum for every
//    16 columns of the output, each expert's part weighted by its tokens' weights on the
//    way. A workgroup takes a few column blocks of an even part of it; the parts are
//    added by the last workgroup to finish one, in their order, so results do not depend
//    on timing.
// Bound by HBM from a few tokens on (16 tokens of 128 experts, 5120 x 1024: 118 to 127 us,
// 4.7 to 5.0 TB/s over all of it); at few (one: 28 us) by three launches' ramps, by the chain
// logits, choice, first weights, and by down_kernel's end, where the last workgroup's loads
// of the parts wait for one another (2 values a thread, a load for each part of one).
// Up to 16 tokens: one row block of the matrix instruction. There it is ahead of the router's
// product, w4a16_moe_route, w4a16_gemm_experts twice and w4a16_moe_combine in one graph (us,
// this / those, at 1, 4, 16 tokens): 8 of 128 experts of 5120 x 1024 30 / 45, 60 / 81, 132 /
// 153; 8 of 256 of 5120 x 512 in groups 30 / 42, 48 / 62, 91 / 110; 4 of 32 of 2048 x 768 21 /
// 31, 28 / 35, 41 / 46.
// Gate, up and down in one launch, whose workgroups wait for the inner rows with down's
// first weights on their way, took 30 us at one token and 123 at 16, when separate launches
// took 27 and 122: the rows' way through memory and the polls behind the weights cost more
// than a launch.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "w4a16_device.h"
#include "w4a16_epilogue.h"
#include "w4a16_lanes.h"
#include "w4a16_launch.h"
#include "w4a16_layer_launch.h"
#include "w4a16_sizes.h"

namespace w4a16_internal {
namespace {

constexpr int kMlTokens = W4A16_MOE_LAYER_MAX_TOKENS;
constexpr int kMlMaxK = W4A16_ROUTE_MAX_TOP_K;
constexpr int kMlWaves = 8;
constexpr int kMlThreads = 64 * kMlWaves;
constexpr int kMlMaxNB = 4;            // column blocks of a workgroup of down_kernel
constexpr int kMlRouterThreads = 1024;  // at most
constexpr int kMlPartFloats = 256;     // a 16 x 16 part

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Offsets in the workspace.
struct MlSpace {
  size_t logits, h, parts, total;
};
MlSpace ml_space(int T, int E, int top_k, int H, int I) {
  MlSpace s;
  // the counters are in front
  s.logits = up256((static_cast<size_t>(H) + 15) / 16 * 4);
  s.h = s.logits + up256(static_cast<size_t>(T) * E * 8);
  s.parts = s.h + up256(static_cast<size_t>(T) * top_k * I * 4);
  // 16 x 16 floats for every column block of every split: at most kModelCUs splits
  // of kMlMaxNB blocks (one split needs none)
  s.total = s.parts + static_cast<size_t>(kModelCUs) * kMlMaxNB * kMlPartFloats * 4;
  return s;
}

struct MlArgs {
  const void* router;
  const float* route_bias;
  const uint32_t* gate_up;
  const uint16_t* gate_up_scales;
  const uint32_t* down;
  const uint16_t* down_scales;
  const uint16_t* x;
  const int* live;
  const uint16_t* base;
  uint16_t* out;
  int* ids;
  float* weights;
  double* logits;   // [T][E]
  uint16_t* h;      // bf16 [T][top_k][I / 8][2][8]: values, what their rounding left
  float* parts;     // [columns][splits][blocks][16][16]
  int* counters;    // [H / 16]: parts that are there of every group of columns
  int T, E, top_k, H, I;
  int sigmoid, groups, groups_kept, group_top, renormalize;
  float scale;
  int most;         // active experts, at most
};

// LDS order within a wave: what its lanes wrote before is there for all of them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------------ router

// TB: tokens it has registers for, T rounded up to a power of two. The row's 16-byte
// pieces go round the threads.
template <bool HALF, int TB>
__global__ __launch_bounds__(kMlRouterThreads) void router_kernel(const MlArgs a) {
  __shared__ double part[kMlRouterThreads / 64][TB];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int threads = blockDim.x;
  for (int i = blockIdx.x * threads + tid; i < (a.H + 15) / 16; i += gridDim.x * threads)
    to_global(a.counters)[i] = 0;
  double acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.0;
  for (int c = tid * 8; c < a.H; c += threads * 8) {
    u32x4 x[TB];  // tokens past the last repeat it
#pragma unroll
    for (int t = 0; t < TB; ++t)
      x[t] = *reinterpret_cast<gptr<const u32x4>>(to_global(a.x) + static_cast<size_t>(min(t, a.T - 1)) * a.H + c);
    double w[8];
    if constexpr (HALF) {
      const u32x4 d = *reinterpret_cast<gptr<const u32x4>>(to_global(static_cast<const uint16_t*>(a.router)) +
                                                           static_cast<size_t>(e) * a.H + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = static_cast<double>(__builtin_bit_cast(float, j % 2 ? d[j / 2] & 0xFFFF0000u : d[j / 2] << 16));
    } else {
      const gptr<const float> p = to_global(static_cast<const float*>(a.router)) + static_cast<size_t>(e) * a.H + c;
      const f32x4 lo = *reinterpret_cast<gptr<const f32x4>>(p), hi = *reinterpret_cast<gptr<const f32x4>>(p + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = static_cast<double>(j < 4 ? lo[j % 4] : hi[j % 4]);
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xv = __builtin_bit_cast(float, j % 2 ? x[t][j / 2] & 0xFFFF0000u : x[t][j / 2] << 16);
        acc[t] = __builtin_fma(static_cast<double>(xv), w[j], acc[t]);
      }
  }
  // Sums over the wave. With 16 tokens every step within a row of 16 lanes halves the
  // tokens a lane holds: it hands over the half that is its partner's and adds what it is
  // given, 17 additions instead of 112. The partners mirror 16 lanes, then 8, then swap
  // pairs, then neighbours: each agrees with the lane in all bits that were used before,
  // so lane l is left with token l % 16 of its row.
  if constexpr (TB == 16) {
    auto step = [&](auto half_, auto ctrl_, int bit) {
      constexpr int HALF_T = half_.value, CTRL = ctrl_.value;
      const bool upper = lane >> bit & 1;
#pragma unroll
      for (int i = 0; i < HALF_T; ++i) {
        const double keep = upper ? acc[i + HALF_T] : acc[i], give = upper ? acc[i] : acc[i + HALF_T];
        acc[i] = keep + dpp_of<CTRL, 0xF>(give);
      }
    };
    using std::integral_constant;
    step(integral_constant<int, 8>{}, integral_constant<int, 0x140>{}, 3);  // row_mirror
    step(integral_constant<int, 4>{}, integral_constant<int, 0x141>{}, 2);  // row_half_mirror
    step(integral_constant<int, 2>{}, integral_constant<int, 0x4E>{}, 1);   // quad_perm [2,3,0,1]
    step(integral_constant<int, 1>{}, integral_constant<int, 0xB1>{}, 0);   // quad_perm [1,0,3,2]
    acc[0] += __shfl_xor(acc[0], 16);
    acc[0] += __shfl_xor(acc[0], 32);
    if (lane < 16) part[wave][lane] = acc[0];
  } else {
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const double s = wave_sum_of(acc[t]);
      if (lane == 0) part[wave][t] = s;
    }
  }
  __syncthreads();
  if (tid < a.T) {
    double s = part[0][tid];
    for (int w = 1; w < threads / 64; ++w) s += part[w][tid];
    to_global(a.logits)[static_cast<size_t>(tid) * a.E + e] = s;
  }
}

// ------------------------------------------------------------------ choice

// The wave's largest key and, of equal ones, the lowest expert (-1: no key is left),
// taken out of the keys. Keys nearly always differ in their high words, so the low
// ones are compared only among those that share the largest.
template <int P>
__device__ __forceinline__ int take_one(uint32_t (&hi)[P], uint32_t (&lo)[P], int lane) {
  uint32_t best = hi[0];
#pragma unroll
  for (int i = 1; i < P; ++i) best = hi[i] > best ? hi[i] : best;
  const uint32_t top = wave_max_of(best);
  if (top == 0) return -1;  // keys of numbers have a high word
  int many = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) many += __popcll(__ballot(hi[i] == top));
  uint32_t low = 0;
  if (many > 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) low = hi[i] == top && lo[i] > low ? lo[i] : low;
    low = wave_max_of(low);
  }
  int e = -1;
#pragma unroll
  for (int i = P - 1; i >= 0; --i) {
    const uint64_t who = __ballot(hi[i] == top && (many == 1 || lo[i] == low));
    if (who) e = i * 64 + __builtin_ctzll(who);
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (e == i * 64 + lane) hi[i] = 0;
  return e;
}

// Two keys of a group, the larger first, with another lane's two.
__device__ __forceinline__ void merge_two(uint64_t& first, uint64_t& second, uint64_t f, uint64_t s) {
  const uint64_t low = f < first ? f : first, high = s > second ? s : second;
  first = f > first ? f : first;
  second = low > high ? low : high;
}

// One token's experts by the rule of w4a16_moe_route, in fp64 throughout; a wave does all
// of it, or as the part-th of several a share of the scores and of the comparisons. P:
// experts per lane, expert i * 64 + lane the i-th.
template <int P>
struct Choice {
  const MlArgs& a;
  int t, lane, part, parts;
  uint64_t* scratch;  // E keys of LDS, the wave's own
  gptr<const double> logits;
  uint64_t key[P];  // of the logits, then of the choice values; 0: cannot be chosen
  double most, sum;

  static __device__ __forceinline__ double finite(double v) { return (v > DBL_MAX ? DBL_MAX : v) + 0.0; }  // -0 is 0
  // a score, but for softmax's division by the sum
  __device__ __forceinline__ double raw_score(double z) const {
    return a.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - most);
  }

  // shared: with several parts, E scores of LDS of the token and then their sums by 64.
  // beside: loads that may come behind the logits'.
  template <typename F>
  __device__ __forceinline__ Choice(const MlArgs& args, int token, int lane_, int part_, int parts_,
                                    uint64_t* scratch_, double* shared, F beside)
      : a(args), t(token), lane(lane_), part(part_), parts(parts_), scratch(scratch_), most(0.0), sum(1.0) {
    logits = to_global(a.logits) + static_cast<size_t>(t) * a.E;
    const int live = a.live ? to_global(a.live)[t] : 1;
    double z[P];
    float bias[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = min(i * 64 + lane, a.E - 1);
      z[i] = logits[e];
      bias[i] = a.route_bias ? to_global(a.route_bias)[e] : 0.f;
    }
    __builtin_amdgcn_sched_barrier(0);
    beside();
    __builtin_amdgcn_sched_barrier(0);
    const bool here = live != 0;
    uint64_t m = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool open = here && i * 64 + lane < a.E && z[i] > -__builtin_inf();
      key[i] = open ? order_key(finite(z[i])) : 0;
      m = key[i] > m ? key[i] : m;
    }
    if (!a.sigmoid) {
      m = wave_max_of(m);
      most = m ? value_of(m) : 0.0;
    }
    // Scores over all experts matter unless experts are compared by their logits and
    // scores are divided by the sum of the chosen.
    const bool by_value = a.route_bias || a.groups > 1;
    if (by_value || (!a.sigmoid && !a.renormalize)) score_all(shared, by_value, bias);
    if (a.groups > 1) keep_groups();
  }

  __device__ __forceinline__ void score_all(double* shared, bool by_value, const float (&bias)[P]) {
    double score[P];
    double by64[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      score[i] = by64[i] = 0.0;
      if (parts > 1 && i % parts != part) continue;
      score[i] = key[i] ? raw_score(value_of(key[i])) : 0.0;
      if (!a.sigmoid) by64[i] = wave_sum_of(score[i]);
      __builtin_amdgcn_sched_barrier(0);  // one exponential's registers at a time
      if (parts > 1) {
        if (i * 64 + lane < a.E) shared[i * 64 + lane] = score[i];
        if (lane == 0) shared[a.E + i] = by64[i];
      }
    }
    if (parts > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (i % parts == part) continue;
        score[i] = shared[min(i * 64 + lane, a.E - 1)];
        by64[i] = shared[a.E + i];
      }
    }
    if (!a.sigmoid) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < P; ++i) sum += by64[i];
    }
    if (!by_value) return;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (key[i]) key[i] = order_key(score[i] / sum + static_cast<double>(bias[i]) + 0.0);
  }

  __device__ __forceinline__ void keep_groups() {
    // A group's largest value, or the sum of its two largest, from a run of lanes: 64
    // over the groups, rounded up to a power of two. Lane g * run holds group g's.
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i * 64 + lane < a.E) scratch[i * 64 + lane] = key[i];
    wave_sync();
    const int per = a.E / a.groups;
    const int shift = a.groups <= 1 ? 6 : __builtin_clz(a.groups - 1) - 26, run = 1 << shift;
    const int g = lane >> shift;
    uint64_t first = 0, second = 0;
    if (g < a.groups)
      for (int i = lane & (run - 1); i < per; i += run) merge_two(first, second, scratch[g * per + i], 0);
    for (int o = 1; o < run; o <<= 1) merge_two(first, second, __shfl_xor(first, o), __shfl_xor(second, o));
    uint64_t value = first;
    if (a.group_top == 2 && second) value = order_key(value_of(first) + value_of(second) + 0.0);
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) {
      const uint64_t other = lane_of(value, o << shift);
      rank += other > value || (other == value && o < g);
    }
    const uint64_t kept = __ballot(g < a.groups && rank < a.groups_kept);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = i * 64 + lane;
      if (e < a.E && !(kept >> (e / per << shift) & 1)) key[i] = 0;
    }
    wave_sync();
  }

  // How many of the experts of the part-th of the parts' ranges have a larger high word,
  // for each of the lane's.
  __device__ __forceinline__ void count_larger(int (&larger)[P]) const {
    uint32_t* const words = reinterpret_cast<uint32_t*>(scratch);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i * 64 + lane < (a.E + 3) / 4 * 4) words[i * 64 + lane] = key[i] >> 32;  // 0 past the last
      larger[i] = 0;
    }
    wave_sync();
    const int quads = (a.E + 3) / 4;
    for (int q = quads * part / parts; q < quads * (part + 1) / parts; ++q) {
      const u32x4 other = reinterpret_cast<const u32x4*>(words)[q];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) larger[i] += other[j] > static_cast<uint32_t>(key[i] >> 32);
    }
    wave_sync();
  }

  // The lane's choice (lane j the j-th, -1 past the last) from the counts over all
  // experts. Keys that share a high word leave a place empty or make too many: then,
  // and where there are no counts, one choice after the other is taken.
  __device__ __forceinline__ int order(const int* larger) {
    int live = 0, few = 0;
    bool counted = larger != nullptr;
    if (counted) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        live += __popcll(__ballot(key[i] != 0));
        few += __popcll(__ballot(key[i] != 0 && larger[i] < a.top_k));
      }
      const int want = min(live, a.top_k);
      int* const places = reinterpret_cast<int*>(scratch);
      if (lane < a.top_k) places[lane] = -1;
      wave_sync();
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (key[i] && larger[i] < a.top_k) places[larger[i]] = i * 64 + lane;
      wave_sync();
      const int id = lane < a.top_k ? places[lane] : -1;
      wave_sync();
      if (few == want && __popcll(__ballot(id >= 0)) == want) return id;
    }
    uint32_t hi[P], lo[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      hi[i] = static_cast<uint32_t>(key[i] >> 32);
      lo[i] = static_cast<uint32_t>(key[i]);
    }
    int id = -1;
    for (int j = 0; j < a.top_k; ++j) {
      const int e = take_one<P>(hi, lo, lane);
      if (e < 0) break;
      if (lane == j) id = e;
    }
    return id;
  }

  // ids and weights of the token; `write`: to the caller's arrays too.
  __device__ __forceinline__ void finish(int id, short* ids, float* weights, bool write) const {
    double w = id >= 0 ? raw_score(finite(logits[id])) / sum : 0.0;
    if (a.renormalize) {
      const double s = wave_sum_of(w);
      w = s > 0.0 ? w / s : 0.0;
    }
    if (lane < a.top_k) {
      ids[lane] = static_cast<short>(id);
      weights[lane] = static_cast<float>(w * a.scale);
      if (write) {
        to_global(a.ids)[t * a.top_k + lane] = id;
        to_global(a.weights)[t * a.top_k + lane] = static_cast<float>(w * a.scale);
      }
    }
  }
};

// LDS of a choice: E keys a wave; E + P doubles and E counts for each token whose work
// several waves share.
__host__ __device__ constexpr size_t choice_bytes(int E, int shared_tokens) {
  const size_t keys = static_cast<size_t>(kMlWaves) * ((E + 3) / 4 * 4) * 8;
  return (keys + shared_tokens * ((static_cast<size_t>(E) + 16) * 8 + static_cast<size_t>(E) * 4) + 15) / 16 * 16;
}

// The experts of tokens t0 .. t0 + T - 1 (T = 1 or 2), the waves shared evenly, into
// ids[i][kMlMaxK] and chosen of the i-th. Every thread. Places are counted where that is
// less work than top_k rounds over the wave (us of the whole layer, counted / by rounds, 8
// per token: 1 token of 128 experts 28.9 / 29.3, of 256 20.8 / 21.7; 4 tokens of 512 36.8 /
// 36.3). beside: loads of every wave that are wanted behind the choice.
template <int P, typename F>
__device__ __forceinline__ void choose_together(const MlArgs& a, int t0, int T, unsigned char* lds,
                                                short (*ids)[kMlMaxK], float (*chosen)[kMlMaxK], bool write, F beside) {
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int keys = (a.E + 3) / 4 * 4;
  double* const shared = reinterpret_cast<double*>(lds) + kMlWaves * keys;
  int* const counts = reinterpret_cast<int*>(shared + T * (a.E + 16));
  for (int i = tid; i < T * a.E; i += kMlThreads) counts[i] = 0;
  __syncthreads();
  const int parts = kMlWaves / T, i0 = wave / parts;
  Choice<P> c(a, t0 + i0, lane, wave % parts, parts, reinterpret_cast<uint64_t*>(lds) + wave * keys,
              shared + i0 * (a.E + 16), beside);
  int larger[P];
  const bool count = P * P <= 4 * parts;
  if (count) {
    c.count_larger(larger);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i * 64 + lane < a.E) atomicAdd(&counts[i0 * a.E + i * 64 + lane], larger[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; ++i) larger[i] = counts[i0 * a.E + min(i * 64 + lane, a.E - 1)];
  }
  if (wave % parts == 0) c.finish(c.order(count ? larger : nullptr), ids[i0], chosen[i0], write);
}

// The experts, up to 64, of up to kMlWaves tokens, a wave for a token.
template <typename F>
__device__ __forceinline__ void choose_each(const MlArgs& a, unsigned char* lds, short (*ids)[kMlMaxK],
                                            float (*chosen)[kMlMaxK], bool write, F beside) {
  const int lane = threadIdx.x & 63, t = uniform(threadIdx.x >> 6);
  if (t >= a.T) return beside();
  Choice<1> c(a, t, lane, 0, 1, reinterpret_cast<uint64_t*>(lds) + t * 64, nullptr, beside);
  int larger[1];
  c.count_larger(larger);
  c.finish(c.order(larger), ids[t], chosen[t], write);
}

// Whether every workgroup of gate_up_kernel makes the choice itself: up to 64 experts a
// wave does a token, and up to two tokens the 8 waves share the work. Otherwise a launch
// of its own, a workgroup per token, is ahead. us of the whole layer, inside / its own
// launch, 8 experts per token: 128 experts of 5120 x 1024 at 1 token 28.9 / 29.8, at 16
// 120 / 114; 256 of 2048 x 512 at 1 token 20.8 / 21.8, at 2 26.4 / 26.0; 128 at 2 23.8 /
// 24.2; 64 at 1 18.5 / 19.7, at 8 33.3 / 33.4; 4 of 64 at 16 37.6 / 35.7.
__host__ __device__ constexpr bool choose_inside(int T, int E) {
  return E <= 64 ? T <= kMlWaves : T <= 2 && T * E <= 256;
}

template <int P>
__global__ __launch_bounds__(kMlThreads) void choose_kernel(const MlArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char ml_lds[];
  __shared__ short ids[1][kMlMaxK];
  __shared__ float chosen[1][kMlMaxK];
  choose_together<P>(a, blockIdx.x, 1, ml_lds, ids, chosen, true, [] {});
}

// ------------------------------------------------------------------ plan

// What a workgroup knows of the choices, in LDS.
struct MlPlan {
  short ids[kMlTokens][kMlMaxK];
  float chosen[kMlTokens][kMlMaxK];
  int active;  // experts with tokens
  // behind it, `most` entries each:
  //   float weight[most][16], uint8 place[most][16], short expert[most], short
  //   mask[most] (a bit per token); then uint32 tokens[E]: while the plan is made an
  //   expert's bits, then its entry
};
__host__ __device__ constexpr size_t ml_plan_bytes(int most, int E) {
  return (sizeof(MlPlan) + 15) / 16 * 16 + static_cast<size_t>(most) * (64 + 2 + 2 + 16) +
         static_cast<size_t>(E) * 4 + 64;
}

struct MlTables {
  MlPlan* plan;
  float* weight;     // [most][16]
  uint32_t* tokens;  // [E] while the plan is made: a bit per token, then the entry
  uint8_t* place;    // [most][16]
  short* expert;     // [most]
  short* mask;       // [most]
  __device__ __forceinline__ MlTables(unsigned char* lds, int most) {
    plan = reinterpret_cast<MlPlan*>(lds);
    weight = reinterpret_cast<float*>(lds + (sizeof(MlPlan) + 15) / 16 * 16);
    place = reinterpret_cast<uint8_t*>(weight + most * 16);
    expert = reinterpret_cast<short*>(place + most * 16);
    mask = expert + most;
    tokens = reinterpret_cast<uint32_t*>(mask + most);  // 2 shorts an entry: 4-byte aligned
  }
};

// The active experts, ascending. Thread t * kMlMaxK + j brings token t's j-th choice (id
// -1: none) and its weight; the tables were cleared in front of a barrier.
static_assert(kMlThreads == kMlTokens * kMlMaxK, "a thread per choice");
__device__ __forceinline__ void clear_plan(const MlArgs& a, const MlTables& tb) {
  for (int e = threadIdx.x; e < a.E; e += kMlThreads) tb.tokens[e] = 0;
  for (int i = threadIdx.x; i < a.most * 16; i += kMlThreads) tb.weight[i] = 0.f;
}
__device__ __forceinline__ void make_plan(const MlArgs& a, const MlTables& tb, int id, float weight) {
  const int tid = threadIdx.x, lane = tid & 63, t = tid / kMlMaxK, j = tid % kMlMaxK;
  if (id >= 0) atomicOr(&tb.tokens[id], 1u << t);
  __syncthreads();
  if (tid < 64) {
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const uint32_t m = e0 + lane < a.E ? tb.tokens[e0 + lane] : 0;
      const uint64_t some = __ballot(m != 0);
      const int at = n + __popcll(some & ((1ull << lane) - 1));
      if (m) {
        tb.expert[at] = static_cast<short>(e0 + lane);
        tb.mask[at] = static_cast<short>(m);
        tb.tokens[e0 + lane] = at;
      }
      n += __popcll(some);
    }
    if (lane == 0) tb.plan->active = n;
  }
  __syncthreads();
  if (id >= 0) {
    const int at = tb.tokens[id];
    tb.place[at * 16 + t] = static_cast<uint8_t>(j);
    tb.weight[at * 16 + t] = weight;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- products

// A unit is max(group, 128) of K: F matrix steps of 32 k, in G groups.
template <int GS>
struct MlUnit {
  static constexpr int K = GS > 128 ? GS : 128;
  static constexpr int F = K / 32;
  static constexpr int G = K / GS;
  static constexpr int WPL = GS / 32;
};

// One block's weights and scales of a unit, as loaded.
template <int GS>
struct MlWeights {
  uint32_t w[MlUnit<GS>::F];
  uint32_t s[MlUnit<GS>::G];
};

// One expert's packed words and scales, as buffers, and whether there is one: loads of an
// absent one lie past the buffers and return zeros without reading memory, so that
// every load is issued and the waits stay exact.
struct MlMatrix {
  __amdgpu_buffer_rsrc_t w, s;
  bool there;
};
// words, scales: 32-bit words and fp16 scales of one expert's matrix, below 4 GB.
__device__ __forceinline__ MlMatrix matrix_at(const uint32_t* w, const uint16_t* s, uint32_t words, uint32_t scales,
                                              int expert, bool there) {
  return {make_rsrc(w + static_cast<size_t>(expert) * words, words * 4u),
          make_rsrc(s + static_cast<size_t>(expert) * scales, scales * 2u), there};
}

// Unit u of a column block whose first tile is `tile` (block * groups); of groups past the
// last the last is read again and not used.
template <int GS>
__device__ __forceinline__ void load_unit(MlWeights<GS>& r, const MlMatrix& m, int tile, int u, int groups, int lane) {
  using U = MlUnit<GS>;
  constexpr int kOnce = 2;  // the instruction's nt bit
  const uint32_t far = 0xFFFFFE00u;
  const uint32_t wl = m.there ? lane * U::WPL * 4 : far, sl = m.there ? (lane & 14) * 2 : far;
#pragma unroll
  for (int g = 0; g < U::G; ++g) {
    const uint32_t at = tile + (U::G > 1 ? unit_group(u, U::G, g, groups) : u);
    const int wat = static_cast<int>(at * (256u * U::WPL));
    if constexpr (U::WPL >= 4) {
#pragma unroll
      for (int q = 0; q < U::WPL / 4; ++q) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(m.w, wl + 16 * q, wat, kOnce);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[g * U::WPL + 4 * q + i] = v[i];
      }
    } else if constexpr (U::WPL == 2) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(m.w, wl, wat, kOnce);
      r.w[g * 2] = v[0];
      r.w[g * 2 + 1] = v[1];
    } else {
      r.w[g] = __builtin_amdgcn_raw_buffer_load_b32(m.w, wl, wat, kOnce);
    }
    r.s[g] = __builtin_amdgcn_raw_buffer_load_b32(m.s, sl, static_cast<int>(at * 32u), 0);
  }
}

// A unit's activation fragments: F pieces of 8 of the lane's row; groups past the
// last are not used.
template <int GS>
struct MlRows {
  u32x4 d[MlUnit<GS>::F];
};
template <int GS>
__device__ __forceinline__ void load_rows(MlRows<GS>& r, gptr<const uint16_t> row, int u, int groups) {
  using U = MlUnit<GS>;
  const int lg = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int g = 0; g < U::G; ++g) {
    const int grp = unit_group(u, U::G, g, groups);
#pragma unroll
    for (int w = 0; w < U::WPL; ++w)
      r.d[g * U::WPL + w] =
          *reinterpret_cast<gptr<const u32x4>>(row + static_cast<size_t>(grp) * GS + (lg * U::WPL + w) * 8);
  }
}

// The fp16 scale of the lane's column.
__device__ __forceinline__ float scale_of(uint32_t pair, int lane) {
  return fp16_bits_to_f32(static_cast<uint16_t>(pair >> (16 * (lane & 1))));
}

// Bytes of LDS in front of gate_up_kernel's plan: the choice's, then the waves' sums of a
// task, twice.
__host__ __device__ constexpr size_t gate_up_front(int T, int E) {
  const size_t choice = choose_inside(T, E) ? choice_bytes(E < 64 ? 64 : E, 2) : 0;
  const size_t sums = 2 * kMlWaves * 2 * 1024;
  return sums > choice ? sums : choice;
}

// KU: units of K per wave, held in registers (0: any number, read again for every
// task, two ahead).
template <int GS, int KU>
__global__ __launch_bounds__(kMlThreads) void gate_up_kernel(const MlArgs a) {
  using U = MlUnit<GS>;
  extern __shared__ __attribute__((aligned(16))) unsigned char ml_lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c16 = lane & 15, lg = lane >> 4;
  float* const red = reinterpret_cast<float*>(ml_lds);
  const MlTables tb(ml_lds + gate_up_front(a.T, a.E), a.most);
  const bf16x8 bias = bias_operand();
  // this wave's units of K, and its tokens' activations of them
  const int up_groups = a.H / GS, up_units = (up_groups + U::G - 1) / U::G;
  const int u0 = up_units * wave / kMlWaves, n = up_units * (wave + 1) / kMlWaves - u0;
  constexpr int kHeld = KU > 0 ? KU : 1;
  MlRows<GS> x[kHeld];
  // rows past the last token repeat it; no expert's list holds them
  const gptr<const uint16_t> row = to_global(a.x) + static_cast<size_t>(min(c16, a.T - 1)) * a.H;
  auto load_x = [&] {
    if constexpr (KU > 0) {
#pragma unroll
      for (int k = 0; k < KU; ++k) load_rows<GS>(x[k], row, min(u0 + k, up_units - 1), up_groups);
    }
  };

  clear_plan(a, tb);
  int id = -1;
  float weight = 0.f;
  const int t = tid / kMlMaxK, j = tid % kMlMaxK;
  const bool place = t < a.T && j < a.top_k;
  if (choose_inside(a.T, a.E)) {
    const bool write = blockIdx.x == 0;
    if (a.T > 2)
      choose_each(a, ml_lds, tb.plan->ids, tb.plan->chosen, write, load_x);
    else if (a.E <= 64)
      choose_together<1>(a, 0, a.T, ml_lds, tb.plan->ids, tb.plan->chosen, write, load_x);
    else if (a.E <= 128)
      choose_together<2>(a, 0, a.T, ml_lds, tb.plan->ids, tb.plan->chosen, write, load_x);
    else
      choose_together<4>(a, 0, a.T, ml_lds, tb.plan->ids, tb.plan->chosen, write, load_x);
    __syncthreads();
    if (place) {
      id = tb.plan->ids[t][j];
      weight = tb.plan->chosen[t][j];
    }
  } else {
    if (place) {
      id = to_global(a.ids)[t * a.top_k + j];
      weight = to_global(a.weights)[t * a.top_k + j];
    }
    load_x();
    __syncthreads();
  }
  make_plan(a, tb, id, weight);

  // A task is 16 columns of the gate half and of the up half of an expert.
  const int ct = a.I / 16;
  const int tasks = tb.plan->active * ct, stride = gridDim.x;
  // of one expert
  const uint32_t up_words = static_cast<uint32_t>(2 * ct) * up_groups * 64 * U::WPL;
  const uint32_t up_scales = static_cast<uint32_t>(2 * ct) * up_groups * 16;
  struct Where {
    MlMatrix m;
    int tile;  // the gate block's first
  };
  const int up_tiles = ct * up_groups;  // from a gate block's to its up block's
  auto find = [&](int task) {
    const bool there = task < tasks;
    const int at = there ? task / ct : 0, c = there ? task - at * ct : 0;
    return Where{matrix_at(a.gate_up, a.gate_up_scales, up_words, up_scales, there ? uniform(tb.expert[at]) : 0, there),
                 uniform(c * up_groups)};
  };
  constexpr int kAhead = KU > 0 ? KU : 2;
  MlWeights<GS> st[kAhead][2];
  MlRows<GS> xs[KU > 0 ? 1 : kAhead];
  auto load = [&](int k, int slot, const Where& p) {
    MlMatrix m = p.m;
    m.there = m.there && k < n;
    const int u = min(u0 + k, up_units - 1);
#pragma unroll
    for (int q = 0; q < 2; ++q) load_unit<GS>(st[slot][q], m, p.tile + q * up_tiles, u, up_groups, lane);
    if constexpr (KU == 0) load_rows<GS>(xs[slot], row, u, up_groups);
  };
  constexpr int kTaskFloats = kMlWaves * 2 * 256;  // red: [2][waves][2][4][64]
  int turn = 0, task = blockIdx.x;
  if (task >= tasks) return;
  Where here = find(task);
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(k, k, here);
  for (; task < tasks; task += stride) {
    const Where there = find(task + stride);
    f32x4 y[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    auto unit = [&](const MlRows<GS>& xr, const MlWeights<GS> (&wt)[2], int u) {
#pragma unroll
      for (int g = 0; g < U::G; ++g) {
        if (U::G > 1 && u * U::G + g >= up_groups) break;  // uniform: K ends inside the unit
        f32x4 accb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < U::WPL; ++w) accb = mfma16(act_frag(xr.d[g * U::WPL + w]), bias, accb);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          f32x4 acc = accb;
#pragma unroll
          for (int w = 0; w < U::WPL; ++w)
            acc = mfma16(act_frag(xr.d[g * U::WPL + w]), dequant_biased(wt[q].w[g * U::WPL + w]), acc);
          const float s = scale_of(wt[q].s[g], lane);
#pragma unroll
          for (int r = 0; r < 4; ++r) y[q][r] = __builtin_fmaf(s, acc[r], y[q][r]);
        }
      }
    };
    if constexpr (KU > 0) {
#pragma unroll
      for (int k = 0; k < KU; ++k) {
        if (k < n) unit(x[k], st[k], u0 + k);
        load(k, k, there);
      }
    } else {
      for (int k = 0; k < n; k += kAhead) {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
          if (k + p < n) unit(xs[p], st[p], u0 + k + p);
          if (k + p + kAhead < n) load(k + p + kAhead, p, here);
        }
      }
#pragma unroll
      for (int p = 0; p < kAhead; ++p) load(p, p, there);
    }

    // the waves' sums, in wave order; consecutive tasks use the two halves in turn, so
    // one barrier a task is enough
    float* const mine = red + turn * kTaskFloats;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) mine[((wave * 2 + q) * 4 + r) * 64 + lane] = y[q][r];
    lds_barrier();
    if (tid < 256) {
      const int at = task / ct, c = task - at * ct;
      const int t = 4 * lg + (tid >> 6);
      if (tb.mask[at] >> t & 1) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < kMlWaves; ++w) {
          gate += mine[(w * 2 * 4 + (tid >> 6)) * 64 + lane];
          up += mine[((w * 2 + 1) * 4 + (tid >> 6)) * 64 + lane];
        }
        const size_t slot = static_cast<size_t>(t) * a.top_k + tb.place[at * 16 + t];
        const float v = silu(gate) * up;
        const uint16_t hi = f32_to_bf16_bits(v);
        const gptr<uint16_t> h = to_global(a.h) + slot * (2 * static_cast<size_t>(a.I)) + c * 32 + (c16 & 8) * 2 + (c16 & 7);
        h[0] = hi;
        h[8] = f32_to_bf16_bits(v - bf16_bits_to_f32(hi));
      }
    }
    turn ^= 1;
    here = there;
  }
}

// NB: column blocks of a workgroup, which share the loads of its inner rows; AHEAD: units
// of them a wave has on the way. 4 and 2: 4 blocks, 3 and 4 units and 5 blocks, 2 units
// took up to 1.5 us more at 1, 3, 4 and 16 tokens. For one token of 8 experts, inner rows
// through LDS, 2 blocks and all of a wave's 8 units on the way without splits: the same.
// Inner rows are two bf16 each, the value and what its rounding left (16 bits in all):
// rounded to one, their error would be as large as the output's own rounding. PAIR, up to
// 8 tokens: the second of token t is row t + 8 of the same matrix instructions, and the
// rows' sums are added at the end. More tokens take a second instruction on the same
// weights. us of the whole layer with one bf16, two in pairs, two in two instructions: 1
// token of 128 experts, 5120 x 1024, 28.5 / 28.8 / 30.3, 4 of 256 45.3 / 45.6 / 47.1, 16 of
// 128 113 / - / 118 (pairs wherever an expert's tokens allow it: 118).
template <int GS, int NB, int AHEAD, bool PAIR>
__global__ __launch_bounds__(kMlThreads) void down_kernel(const MlArgs a, int most_splits) {
  using U = MlUnit<GS>;
  extern __shared__ __attribute__((aligned(16))) unsigned char ml_lds[];
  __shared__ int last_flag;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c16 = lane & 15, lg = lane >> 4;
  float* const red = reinterpret_cast<float*>(ml_lds);  // [waves][NB][4][64]
  const MlTables tb(ml_lds + kMlWaves * NB * 1024, a.most);
  const bf16x8 bias = bias_operand();
  const int groups = a.I / GS, units = (groups + U::G - 1) / U::G;  // of one expert
  const int blocks = a.H / 16;
  const int column = static_cast<int>(blockIdx.x) / most_splits, split = static_cast<int>(blockIdx.x) % most_splits;
  const int b0 = column * NB;  // first column block
  int id = -1;
  float chosen = 0.f;
  {
    const int t = tid / kMlMaxK, j = tid % kMlMaxK;
    if (t < a.T && j < a.top_k) {
      id = to_global(a.ids)[t * a.top_k + j];
      chosen = to_global(a.weights)[t * a.top_k + j];
    }
  }
  const uint32_t h_bytes = static_cast<uint32_t>(a.T * a.top_k) * a.I * 4;
  const __amdgpu_buffer_rsrc_t rh = make_rsrc(a.h, h_bytes);
  // Value i of the tile: block i / 256, row 4 (lane / 16) + i / 64 % 4 and column lane %
  // 16 of it, lane = i % 64. Whether there is such a value, and what is added to it.
  auto value_at = [&](int i, int& t, int& col) {
    t = 4 * ((i & 63) >> 4) + (i >> 6 & 3);
    col = (b0 + (i >> 8)) * 16 + (i & 15);
    return i < NB * 256 && t < a.T && col < a.H;
  };
  constexpr int kValues = (NB * 256 + kMlThreads - 1) / kMlThreads;  // a thread's
  uint16_t base[kValues];
#pragma unroll
  for (int j = 0; j < kValues; ++j) {
    int t, col;
    const bool there = value_at(tid + j * kMlThreads, t, col);
    base[j] = there && a.base ? to_global(a.base)[static_cast<size_t>(t) * a.H + col] : 0;
  }
  clear_plan(a, tb);
  __syncthreads();
  make_plan(a, tb, id, chosen);

  const int all = tb.plan->active * units;  // units of the long sum
  // as many parts as leave every wave a unit
  const int splits = max(1, min(most_splits, all / kMlWaves));
  if (split >= splits) return;
  // of one expert
  const uint32_t words = static_cast<uint32_t>(blocks) * groups * 64 * U::WPL;
  const uint32_t scales = static_cast<uint32_t>(blocks) * groups * 16;
  struct Stage {
    MlWeights<GS> w[NB];
    MlRows<GS> h, l;
    int at, u;  // entry and unit of the expert
  };
  Stage ds[AHEAD];
  // a wave's way through the units of its part: every kMlWaves-th of them
  const int first = static_cast<int>(static_cast<long long>(all) * split / splits) + wave;
  const int end = static_cast<int>(static_cast<long long>(all) * (split + 1) / splits);
  const int n = max(0, (end - first + kMlWaves - 1) / kMlWaves);
  const int at_step = kMlWaves / units, u_step = kMlWaves - at_step * units;
  int next_at = first / units, next_u = first - next_at * units, left = n;
  auto load_weights = [&](Stage& s) {
    const bool there = left > 0;
    s.at = there ? next_at : -1;
    s.u = there ? next_u : 0;
    const MlMatrix m =
        matrix_at(a.down, a.down_scales, words, scales, there ? uniform(tb.expert[next_at]) : 0, there);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      MlMatrix mb = m;
      mb.there = there && b0 + b < blocks;
      load_unit<GS>(s.w[b], mb, min(b0 + b, blocks - 1) * groups, s.u, groups, lane);
    }
    next_at += at_step;
    next_u += u_step;
    if (next_u >= units) {
      next_u -= units;
      ++next_at;
    }
    --left;
    __builtin_amdgcn_sched_barrier(0);  // one unit's buffers in scalar registers at a time
  };
  auto load_inner = [&](Stage& s) {
    // other tokens' rows lie past the buffer and read as zeros, as do groups past
    // the last (its end is one of them)
    const int t = PAIR ? c16 & 7 : c16;
    const bool mine = s.at >= 0 && tb.mask[s.at] >> t & 1;
    const uint32_t slot = mine ? t * a.top_k + tb.place[s.at * 16 + t] : 0;
    const uint32_t second = PAIR ? (c16 & 8) * 2 : 0;
#pragma unroll
    for (int g = 0; g < U::G; ++g) {
      const int grp = s.u * U::G + g;
      const uint32_t at = mine && grp < groups ? (slot * a.I + grp * GS + lg * U::WPL * 8) * 4 + second : 0xFFFFFE00u;
#pragma unroll
      for (int w = 0; w < U::WPL; ++w) {
        s.h.d[g * U::WPL + w] = __builtin_amdgcn_raw_buffer_load_b128(rh, at, 32 * w, 0);
        if constexpr (!PAIR) s.l.d[g * U::WPL + w] = __builtin_amdgcn_raw_buffer_load_b128(rh, at, 32 * w + 16, 0);
      }
    }
  };
#pragma unroll
  for (int p = 0; p < AHEAD; ++p) load_weights(ds[p]);
#pragma unroll
  for (int p = 0; p < AHEAD; ++p) load_inner(ds[p]);
  f32x4 y[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) y[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto unit = [&](const Stage& s) {
    const int t0 = 4 * (PAIR ? lg & 1 : lg);  // the token of the lane's first row
    const f32x4 wt = *reinterpret_cast<const f32x4*>(tb.weight + s.at * 16 + t0);
    const int live = static_cast<uint16_t>(tb.mask[s.at]) >> t0;
#pragma unroll
    for (int g = 0; g < U::G; ++g) {
      if (U::G > 1 && s.u * U::G + g >= groups) break;  // uniform: K ends inside the unit
      f32x4 accb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < U::WPL; ++w) {
        accb = mfma16(act_frag(s.h.d[g * U::WPL + w]), bias, accb);
        if constexpr (!PAIR) accb = mfma16(act_frag(s.l.d[g * U::WPL + w]), bias, accb);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x4 acc = accb;
#pragma unroll
        for (int w = 0; w < U::WPL; ++w) {
          const bf16x8 q = dequant_biased(s.w[b].w[g * U::WPL + w]);
          acc = mfma16(act_frag(s.h.d[g * U::WPL + w]), q, acc);
          if constexpr (!PAIR) acc = mfma16(act_frag(s.l.d[g * U::WPL + w]), q, acc);
        }
        const float sc = scale_of(s.w[b].s[g], lane);
        // a row that is not the expert's takes nothing from it, whatever its values
#pragma unroll
        for (int r = 0; r < 4; ++r)
          y[b][r] = live >> r & 1 ? __builtin_fmaf(sc * wt[r], acc[r], y[b][r]) : y[b][r];
      }
    }
  };
  for (int k = 0; k < n; k += AHEAD) {
#pragma unroll
    for (int p = 0; p < AHEAD; ++p) {
      if (k + p < n) unit(ds[p]);
      load_weights(ds[p]);
      load_inner(ds[p]);
    }
  }

  if constexpr (PAIR) {  // rows t and t + 8 are 32 lanes apart
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) y[b][r] += __shfl_xor(y[b][r], 32);
  }
  // the waves' sums, in wave order
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[((wave * NB + b) * 4 + r) * 64 + lane] = y[b][r];
  lds_barrier();
  auto write = [&](int t, int col, float v, uint16_t base_bits) {
    if (a.base) v += bf16_bits_to_f32(base_bits);
    to_global(a.out)[static_cast<size_t>(t) * a.H + col] = f32_to_bf16_bits(v);
  };
  float* const part = a.parts + static_cast<size_t>(column) * most_splits * NB * 256;
#pragma unroll
  for (int j = 0; j < kValues; ++j) {
    const int i = tid + j * kMlThreads;
    int t, col;
    if (!value_at(i, t, col)) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kMlWaves; ++w) v += red[w * NB * 256 + i];
    if (splits == 1)
      write(t, col, v, base[j]);
    else
      __hip_atomic_store(part + split * NB * 256 + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (splits == 1) return;
  // The last of the splits to count itself in adds their parts, in their order.
  wait_vmem_all();
  __syncthreads();
  if (tid == 0)
    last_flag = __hip_atomic_fetch_add(a.counters + column, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
  __syncthreads();
  if (!last_flag) return;
#pragma unroll
  for (int j = 0; j < kValues; ++j) {
    const int i = tid + j * kMlThreads;
    int t, col;
    if (!value_at(i, t, col)) continue;
    float v = 0.f;
    for (int s = 0; s < splits; ++s)
      v += __hip_atomic_load(part + s * NB * 256 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    write(t, col, v, base[j]);
  }
}

// ---------------------------------------------------------------- launches

template <typename... Params, typename... Args>
hipError_t launch(void (*kernel)(Params...), int grid, int threads, size_t lds, hipStream_t stream, Args... args) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (lds >= 60 * 1024) {  // with the kernels' own variables past the 64 KB that need no leave
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  static_assert((std::is_same_v<Params, Args> && ...), "arguments are passed by address");
  void* kargs[] = {&args...};
  return hipLaunchKernel(fn, dim3(grid), dim3(threads), kargs, lds, stream);
}

template <int P>
hipError_t launch_choose_t(const MlArgs& a, hipStream_t stream) {
  return launch(&choose_kernel<P>, a.T, kMlThreads, choice_bytes(a.E, 1), stream, a);
}

hipError_t launch_choose(const MlArgs& a, hipStream_t stream) {
  if (a.E <= 64) return launch_choose_t<1>(a, stream);
  if (a.E <= 128) return launch_choose_t<2>(a, stream);
  if (a.E <= 256) return launch_choose_t<4>(a, stream);
  if (a.E <= 512) return launch_choose_t<8>(a, stream);
  return launch_choose_t<16>(a, stream);
}

template <bool HALF>
hipError_t launch_router(const MlArgs& a, hipStream_t stream) {
  // as few rounds as 1024 threads allow, and no more threads than they need
  const int pieces = a.H / 8, rounds = (pieces + kMlRouterThreads - 1) / kMlRouterThreads;
  const int threads = ((pieces + rounds - 1) / rounds + 63) / 64 * 64;
  if (a.T == 1) return launch(&router_kernel<HALF, 1>, a.E, threads, 0, stream, a);
  if (a.T == 2) return launch(&router_kernel<HALF, 2>, a.E, threads, 0, stream, a);
  if (a.T <= 4) return launch(&router_kernel<HALF, 4>, a.E, threads, 0, stream, a);
  if (a.T <= 8) return launch(&router_kernel<HALF, 8>, a.E, threads, 0, stream, a);
  return launch(&router_kernel<HALF, 16>, a.E, threads, 0, stream, a);
}

template <int GS, int KU>
hipError_t launch_gate_up(const MlArgs& a, hipStream_t stream) {
  const size_t lds = gate_up_front(a.T, a.E) + ml_plan_bytes(a.most, a.E);
  const long long tasks = static_cast<long long>(a.most) * (a.I / 16);
  const int grid = static_cast<int>(tasks < kModelCUs ? tasks : kModelCUs);
  return launch(&gate_up_kernel<GS, KU>, grid, kMlThreads, lds, stream, a);
}

template <int GS, int NB, int AHEAD, bool PAIR>
hipError_t launch_down(const MlArgs& a, hipStream_t stream) {
  static_assert(NB <= kMlMaxNB, "room for the parts");
  const size_t lds = static_cast<size_t>(kMlWaves) * NB * 1024 + ml_plan_bytes(a.most, a.E);
  const int columns = (a.H / 16 + NB - 1) / NB;
  const int splits = columns < kModelCUs ? kModelCUs / columns : 1;
  return launch(&down_kernel<GS, NB, AHEAD, PAIR>, columns * splits, kMlThreads, lds, stream, a, splits);
}

template <int GS>
hipError_t launch_moe_layer_g(const MlArgs& a, bool half, hipStream_t stream) {
  using U = MlUnit<GS>;
  hipError_t e = half ? launch_router<true>(a, stream) : launch_router<false>(a, stream);
  if (e != hipSuccess) return e;
  if (!choose_inside(a.T, a.E)) {
    e = launch_choose(a, stream);
    if (e != hipSuccess) return e;
  }
  constexpr int kPer = U::K / 128;
  const int held = ((a.H / GS + U::G - 1) / U::G + kMlWaves - 1) / kMlWaves * kPer;  // 128s of K per wave
  // The next larger form that is built; loads of units that a wave has not are not made. us
  // of the whole layer, 8 of 64 experts of width 1024, at groups of 128 and 64: five units
  // by their own form and by six, 1 token 28.1 / 28.5 and 31.6 / 33.2, 16 tokens 102 / 105
  // and 115 / 119; three by four and by a form of their own 24.0 / 23.9 and 26.5 / 25.4,
  // 67.6 / 66.1 and 80.4 / 75.4; seven by eight and by their own 33.0 / 32.4, 134 / 132.
  if (held <= 2)
    e = launch_gate_up<GS, 2 / kPer>(a, stream);
  else if (held <= 4)
    e = launch_gate_up<GS, 4 / kPer>(a, stream);
  else if (held == 5 && kPer == 1)
    e = launch_gate_up<GS, kPer == 1 ? 5 : 0>(a, stream);
  else if (held <= 6)
    e = launch_gate_up<GS, 6 / kPer>(a, stream);
  else if (held <= 8 && GS >= 128)  // groups of 32 and 64 and their scales would spill
    e = launch_gate_up<GS, GS >= 128 ? 8 / kPer : 0>(a, stream);
  else
    e = launch_gate_up<GS, 0>(a, stream);
  if (e != hipSuccess) return e;
  constexpr int kAhead = U::F == 4 ? 2 : 1;
  return a.T <= 8 ? launch_down<GS, 4, kAhead, true>(a, stream) : launch_down<GS, 4, kAhead, false>(a, stream);
}

}  // namespace

size_t moe_layer_workspace_bytes(int T, int E, int top_k, int H, int I) { return ml_space(T, E, top_k, H, I).total; }

hipError_t launch_moe_layer(const MoeLayerArgs& m, hipStream_t stream) {
  const w4a16_moe_layer_args& l = m.layer;
  const w4a16_route_config& r = l.route;
  const MlSpace s = ml_space(m.T, r.experts, r.top_k, l.hidden, l.width);
  MlArgs a = {};
  a.router = l.router;
  a.route_bias = l.route_bias;
  a.gate_up = static_cast<const uint32_t*>(l.gate_up);
  a.gate_up_scales = static_cast<const uint16_t*>(l.gate_up_scales);
  a.down = static_cast<const uint32_t*>(l.down);
  a.down_scales = static_cast<const uint16_t*>(l.down_scales);
  a.x = m.x;
  a.live = m.live;
  a.base = m.base;
  a.out = m.out;
  a.ids = m.ids;
  a.weights = m.weights;
  a.counters = reinterpret_cast<int*>(m.workspace);
  a.logits = reinterpret_cast<double*>(m.workspace + s.logits);
  a.h = reinterpret_cast<uint16_t*>(m.workspace + s.h);
  a.parts = reinterpret_cast<float*>(m.workspace + s.parts);
  a.T = m.T;
  a.E = r.experts;
  a.top_k = r.top_k;
  a.H = l.hidden;
  a.I = l.width;
  a.sigmoid = r.scoring == W4A16_ROUTE_SIGMOID;
  a.groups = r.groups;
  a.groups_kept = r.groups_kept;
  a.group_top = r.group_top;
  a.renormalize = r.renormalize != 0;
  a.scale = r.scale;
  a.most = m.T * r.top_k < r.experts ? m.T * r.top_k : r.experts;
  const bool half = l.router_type == W4A16_LOGITS_BF16;
  switch (l.group) {
    case 32: return launch_moe_layer_g<32>(a, half, stream);
    case 64: return launch_moe_layer_g<64>(a, half, stream);
    case 128: return launch_moe_layer_g<128>(a, half, stream);
    case 256: return launch_moe_layer_g<256>(a, half, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w4a16_internal

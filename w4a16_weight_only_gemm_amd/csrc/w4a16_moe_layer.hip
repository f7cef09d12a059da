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
//    additions. It also clears the counters of the last kernel.
//  * gate_up_kernel: every workgroup chooses the experts itself, from the logits
//    (E doubles a token), and lists those that are active; a wave owns a range of K
//    and holds its tokens' activations of that range in registers for as long as
//    the workgroup lives, while the weights of one (expert, 16 gate and 16 up
//    columns) after the other stream by, a whole task ahead. The waves' sums meet
//    in LDS, where SwiGLU is formed.
//  * down_kernel: the active experts' k ranges laid end to end are one long sum for
//    every 16 columns of the output, each expert's part weighted by its tokens'
//    weights on the way. The (16 columns, expert, k) units are dealt out evenly to
//    the workgroups; columns that lie with several are joined through the
//    workspace by the last to arrive, in the order of the workgroups, so results
//    do not depend on timing.
// Bound by HBM from a few tokens on; at one token by the launches and by the chain
// logits, choice, first weights.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "w4a16_device.h"
#include "w4a16_epilogue.h"
#include "w4a16_lanes.h"
#include "w4a16_launch.h"
#include "w4a16_layer_launch.h"

namespace w4a16_internal {
namespace {

constexpr int kMlTokens = W4A16_MOE_LAYER_MAX_TOKENS;
constexpr int kMlMaxK = W4A16_ROUTE_MAX_TOP_K;
constexpr int kMlWaves = 8;
constexpr int kMlThreads = 64 * kMlWaves;
constexpr int kMlMaxGrid = 512;        // workgroups of the product kernels
constexpr int kMlRouterThreads = 256;
constexpr int kMlPartFloats = 256;     // a 16 x 16 part

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Offsets in the workspace.
struct MlSpace {
  size_t logits, h, parts, total;
};
MlSpace ml_space(int T, int E, int top_k, int H, int I) {
  MlSpace s;
  s.logits = up256((static_cast<size_t>(H) + 15) / 16 * 4);  // the counters are in front
  s.h = s.logits + up256(static_cast<size_t>(T) * E * 8);
  s.parts = s.h + up256(static_cast<size_t>(T) * top_k * I * 2);
  s.total = s.parts + static_cast<size_t>(kMlMaxGrid) * 2 * kMlPartFloats * 4;
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
  uint16_t* h;      // bf16 [T][top_k][I]
  float* parts;     // [workgroups][2][16][16]
  int* counters;    // [H / 16]
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

template <bool HALF>
__global__ __launch_bounds__(kMlRouterThreads) void router_kernel(const MlArgs a) {
  __shared__ double part[kMlRouterThreads / 64][kMlTokens];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = blockIdx.x * kMlRouterThreads + tid; i < (a.H + 15) / 16; i += gridDim.x * kMlRouterThreads)
    to_global(a.counters)[i] = 0;
  double acc[kMlTokens];
#pragma unroll
  for (int t = 0; t < kMlTokens; ++t) acc[t] = 0.0;
  for (int c = tid * 8; c < a.H; c += kMlRouterThreads * 8) {
    float w[8];
    if constexpr (HALF) {
      const u32x4 d = *reinterpret_cast<gptr<const u32x4>>(to_global(static_cast<const uint16_t*>(a.router)) +
                                                           static_cast<size_t>(e) * a.H + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = __builtin_bit_cast(float, j % 2 ? d[j / 2] & 0xFFFF0000u : d[j / 2] << 16);
    } else {
      const gptr<const float> p = to_global(static_cast<const float*>(a.router)) + static_cast<size_t>(e) * a.H + c;
      const f32x4 lo = *reinterpret_cast<gptr<const f32x4>>(p), hi = *reinterpret_cast<gptr<const f32x4>>(p + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < 4 ? lo[j % 4] : hi[j % 4];
    }
#pragma unroll
    for (int t = 0; t < kMlTokens; ++t) {
      if (t >= a.T) continue;
      const u32x4 d = *reinterpret_cast<gptr<const u32x4>>(to_global(a.x) + static_cast<size_t>(t) * a.H + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xv = __builtin_bit_cast(float, j % 2 ? d[j / 2] & 0xFFFF0000u : d[j / 2] << 16);
        acc[t] = __builtin_fma(static_cast<double>(xv), static_cast<double>(w[j]), acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kMlTokens; ++t) {
    if (t >= a.T) continue;
    const double s = wave_sum_of(acc[t]);
    if (lane == 0) part[wave][t] = s;
  }
  __syncthreads();
  if (tid < a.T) {
    double s = part[0][tid];
#pragma unroll
    for (int w = 1; w < kMlRouterThreads / 64; ++w) s += part[w][tid];
    to_global(a.logits)[static_cast<size_t>(tid) * a.E + e] = s;
  }
}

// ------------------------------------------------------------------ choice

// One wave chooses one token's experts: the rule of w4a16_moe_route in fp64
// throughout. scratch: E keys of LDS.
template <int P>
__device__ __forceinline__ void choose(const MlArgs& a, int t, uint64_t* scratch, int lane, short* ids, float* weights) {
  const bool here = !a.live || a.live[t] != 0;
  const gptr<const double> logits = to_global(a.logits) + static_cast<size_t>(t) * a.E;
  auto finite = [](double v) { return (v > DBL_MAX ? DBL_MAX : v) + 0.0; };  // and -0 is 0
  uint64_t key[P];  // of the logits, then of the choice values; 0: cannot be chosen
  uint64_t m = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = i * 64 + lane;
    const double v = e < a.E ? logits[e] : -__builtin_inf();
    key[i] = here && v > -__builtin_inf() ? order_key(finite(v)) : 0;
    m = key[i] > m ? key[i] : m;
  }
  double most = 0.0, sum = 0.0;
  if (!a.sigmoid) {
    m = wave_max_of(m);
    most = m ? value_of(m) : 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      sum += key[i] ? exp(value_of(key[i]) - most) : 0.0;
      __builtin_amdgcn_sched_barrier(0);  // one exponential's registers at a time
    }
    sum = wave_sum_of(sum);
  }
  auto score = [&](double z) { return a.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - most) / sum; };
  if (a.route_bias || a.groups > 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = i * 64 + lane;
      const double bias = a.route_bias && e < a.E ? to_global(a.route_bias)[e] : 0.f;
      if (key[i]) key[i] = order_key(score(value_of(key[i])) + bias + 0.0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (a.groups > 1) {
    // lane g looks at group g: its largest value, or the sum of its two largest
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i * 64 + lane < a.E) scratch[i * 64 + lane] = key[i];
    wave_sync();
    const int per = a.E / a.groups;
    uint64_t first = 0, second = 0;
    if (lane < a.groups)
      for (int i = 0; i < per; ++i) {
        const uint64_t k = scratch[lane * per + i];
        const uint64_t lower = k < first ? k : first;
        first = k > first ? k : first;
        second = lower > second ? lower : second;
      }
    uint64_t value = first;
    if (a.group_top == 2 && second) value = order_key(value_of(first) + value_of(second) + 0.0);
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t other = lane_of(value, g);
      rank += other > value || (other == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.groups_kept);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = i * 64 + lane;
      if (e < a.E && !(kept >> (e / per) & 1)) key[i] = 0;
    }
    wave_sync();
  }
  const int id = take<P, false>(key, a.top_k, lane);
  double w = id >= 0 ? score(finite(logits[id])) : 0.0;
  if (a.renormalize) {
    const double s = wave_sum_of(w);
    w = s > 0.0 ? w / s : 0.0;
  }
  if (lane < a.top_k) {
    ids[lane] = static_cast<short>(id);
    weights[lane] = static_cast<float>(w * a.scale);
  }
}

// ------------------------------------------------------------------ plan

// What a workgroup knows of the choices, in LDS.
struct MlPlan {
  short ids[kMlTokens][kMlMaxK];
  float chosen[kMlTokens][kMlMaxK];
  int active;  // experts with tokens
  // behind it, `most` entries each:
  //   float weight[most][16], short expert[most], short tokens[most] (a bit each),
  //   uint8 place[most][16]; then short index[E]
};
__host__ __device__ constexpr size_t ml_plan_bytes(int most, int E) {
  return (sizeof(MlPlan) + 15) / 16 * 16 + static_cast<size_t>(most) * (64 + 2 + 2 + 16) +
         static_cast<size_t>(E) * 4 + 64;
}

struct MlTables {
  MlPlan* plan;
  float* weight;     // [most][16]
  uint32_t* tokens;  // [E] while the plan is made: a bit per token
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

// The active experts, ascending, from plan->ids and plan->chosen. Every thread.
__device__ __forceinline__ void make_plan(const MlArgs& a, const MlTables& tb) {
  const int tid = threadIdx.x, lane = tid & 63;
  for (int e = tid; e < a.E; e += kMlThreads) tb.tokens[e] = 0;
  for (int i = tid; i < a.most * 16; i += kMlThreads) tb.weight[i] = 0.f;
  __syncthreads();
  static_assert(kMlThreads == kMlTokens * kMlMaxK, "a thread per place");
  const int t = tid / kMlMaxK, j = tid % kMlMaxK;
  int id = -1;
  if (t < a.T && j < a.top_k) id = tb.plan->ids[t][j];
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
    tb.weight[at * 16 + t] = tb.plan->chosen[t][j];
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

// Unit u of a block whose packed words and scales start at w and s (already at the
// lane's place); groups past the last re-read it and are not used.
template <int GS>
__device__ __forceinline__ void load_unit(MlWeights<GS>& r, gptr<const uint32_t> w, gptr<const uint32_t> s, int u,
                                          int groups) {
  using U = MlUnit<GS>;
#pragma unroll
  for (int g = 0; g < U::G; ++g) {
    const int grp = min(u * U::G + g, groups - 1);
    const gptr<const uint32_t> p = w + static_cast<size_t>(grp) * 64 * U::WPL;
    if constexpr (U::WPL >= 4) {
#pragma unroll
      for (int q = 0; q < U::WPL / 4; ++q) {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<gptr<const u32x4>>(p) + q);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[g * U::WPL + 4 * q + i] = v[i];
      }
    } else if constexpr (U::WPL == 2) {
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<gptr<const u32x2>>(p));
      r.w[g * 2] = v[0];
      r.w[g * 2 + 1] = v[1];
    } else {
      r.w[g] = __builtin_nontemporal_load(p);
    }
    r.s[g] = s[static_cast<size_t>(grp) * 8];
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
    const int grp = min(u * U::G + g, groups - 1);
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

// LDS in front of gate_up_kernel's plan: the waves' sums, twice, and before them
// the choice's scratch, E keys a wave.
__host__ __device__ constexpr size_t gate_up_scratch(int E) {
  const size_t sums = 2 * kMlWaves * 2 * 256 * 4, scratch = (static_cast<size_t>(kMlWaves) * E * 8 + 15) / 16 * 16;
  return sums > scratch ? sums : scratch;
}

// KU: units of K per wave, held in registers (0: any number, read again for every
// task, two ahead).
template <int GS, int KU>
__global__ __launch_bounds__(kMlThreads) void gate_up_kernel(const MlArgs a) {
  using U = MlUnit<GS>;
  extern __shared__ __attribute__((aligned(16))) unsigned char ml_lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c16 = lane & 15;
  float* const red = reinterpret_cast<float*>(ml_lds);  // [2][waves][2][4][64]
  constexpr int kRedFloats = kMlWaves * 2 * 256;
  // the scratch of the choice lies where the sums meet later
  const MlTables tb(ml_lds + gate_up_scratch(a.E), a.most);
  // this wave's units of K
  const int groups = a.H / GS, units = (groups + U::G - 1) / U::G;
  const int u0 = units * wave / kMlWaves, n = units * (wave + 1) / kMlWaves - u0;

  // The tokens' activations do not need the choice.
  constexpr int kHeld = KU > 0 ? KU : 1;
  MlRows<GS> x[kHeld];
  // rows past the last token repeat it; no expert's list holds them
  const gptr<const uint16_t> row = to_global(a.x) + static_cast<size_t>(min(c16, a.T - 1)) * a.H;
  if constexpr (KU > 0) {
#pragma unroll
    for (int k = 0; k < KU; ++k) load_rows<GS>(x[k], row, min(u0 + k, units - 1), groups);
  }

  uint64_t* const scratch = reinterpret_cast<uint64_t*>(ml_lds) + static_cast<size_t>(wave) * a.E;
  for (int t = wave; t < a.T; t += kMlWaves) {
    short* const ids = tb.plan->ids[t];
    float* const chosen = tb.plan->chosen[t];
    if (a.E <= 64)
      choose<1>(a, t, scratch, lane, ids, chosen);
    else if (a.E <= 128)
      choose<2>(a, t, scratch, lane, ids, chosen);
    else if (a.E <= 256)
      choose<4>(a, t, scratch, lane, ids, chosen);
    else if (a.E <= 512)
      choose<8>(a, t, scratch, lane, ids, chosen);
    else
      choose<16>(a, t, scratch, lane, ids, chosen);
    if (blockIdx.x == 0 && lane < a.top_k) {
      to_global(a.ids)[t * a.top_k + lane] = ids[lane];
      to_global(a.weights)[t * a.top_k + lane] = chosen[lane];
    }
  }
  __syncthreads();
  make_plan(a, tb);

  const int ct = a.I / 16;  // column blocks of a half
  const int tasks = tb.plan->active * ct;
  const size_t words = static_cast<size_t>(2 * ct) * groups * 64 * U::WPL;  // of one expert
  const size_t scales = static_cast<size_t>(2 * ct) * groups * 16;
  // the lane's places in the gate and the up block of a task
  struct Where {
    gptr<const uint32_t> w[2], s[2];
  };
  auto find = [&](int task) {
    const int at = task / ct, c = task - at * ct, e = tb.expert[at];
    Where p;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const size_t b = static_cast<size_t>(c + q * ct) * groups;
      p.w[q] = to_global(a.gate_up) + e * words + b * 64 * U::WPL + lane * U::WPL;
      p.s[q] = reinterpret_cast<gptr<const uint32_t>>(to_global(a.gate_up_scales) + e * scales + b * 16 + (c16 & ~1));
    }
    return p;
  };
  constexpr int kAhead = KU > 0 ? KU : 2;
  MlWeights<GS> st[kAhead][2];
  MlRows<GS> xs[KU > 0 ? 1 : kAhead];
  int task = blockIdx.x;
  if (task >= tasks) return;
  Where here = find(task);
  auto load = [&](int k, int slot, const Where& p) {
    const int u = min(u0 + min(k, max(n, 1) - 1), units - 1);  // past the wave's last: not used
#pragma unroll
    for (int q = 0; q < 2; ++q) load_unit<GS>(st[slot][q], p.w[q], p.s[q], u, groups);
    if constexpr (KU == 0) load_rows<GS>(xs[slot], row, u, groups);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(k, k, here);

  const bf16x8 bias = bias_operand();
  int turn = 0;
  for (; task < tasks; task += gridDim.x) {
    const int next = task + static_cast<int>(gridDim.x);
    const Where there = find(min(next, tasks - 1));
    f32x4 y[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    auto unit = [&](const MlRows<GS>& xr, const MlWeights<GS> (&wt)[2], int u) {
#pragma unroll
      for (int g = 0; g < U::G; ++g) {
        if (U::G > 1 && u * U::G + g >= groups) break;  // uniform: K ends inside the unit
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
          // the next unit of this task, or past its last one those of the next
          if (k + p + kAhead < n)
            load(k + p + kAhead, p, here);
        }
      }
#pragma unroll
      for (int p = 0; p < kAhead; ++p) load(p, p, there);
    }

    // the waves' sums, in wave order
    float* const mine = red + turn * kRedFloats;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) mine[((wave * 2 + q) * 4 + r) * 64 + lane] = y[q][r];
    lds_barrier();
    if (tid < 256) {
      const int at = task / ct, c = task - at * ct;
      const int t = 4 * (lane >> 4) + (tid >> 6);
      if (tb.mask[at] >> t & 1) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < kMlWaves; ++w) {
          gate += mine[(w * 2 * 4 + (tid >> 6)) * 64 + lane];
          up += mine[((w * 2 + 1) * 4 + (tid >> 6)) * 64 + lane];
        }
        const size_t slot = static_cast<size_t>(t) * a.top_k + tb.place[at * 16 + t];
        to_global(a.h)[slot * a.I + c * 16 + c16] = f32_to_bf16_bits(silu(gate) * up);
      }
    }
    turn ^= 1;
    here = there;
  }
}

// AHEAD: units a wave has on the way.
template <int GS, int AHEAD>
__global__ __launch_bounds__(kMlThreads) void down_kernel(const MlArgs a) {
  using U = MlUnit<GS>;
  extern __shared__ __attribute__((aligned(16))) unsigned char ml_lds[];
  __shared__ int last_flag;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c16 = lane & 15, lg = lane >> 4;
  float* const red = reinterpret_cast<float*>(ml_lds);  // [2][waves][4][64]
  constexpr int kRedFloats = kMlWaves * 256;
  const MlTables tb(ml_lds + 2 * kRedFloats * 4, a.most);
  {
    const int t = tid / kMlMaxK, j = tid % kMlMaxK;
    if (t < a.T && j < a.top_k) {
      tb.plan->ids[t][j] = static_cast<short>(to_global(a.ids)[t * a.top_k + j]);
      tb.plan->chosen[t][j] = to_global(a.weights)[t * a.top_k + j];
    }
  }
  __syncthreads();
  make_plan(a, tb);

  const int groups = a.I / GS, units = (groups + U::G - 1) / U::G;  // of one expert
  const int blocks = a.H / 16;
  const int per = tb.plan->active * units;  // units of a column block
  const long long total = static_cast<long long>(per) * blocks;
  // the finished values of a block's rows
  auto write = [&](int b, int t, int col, float v) {
    const size_t at = static_cast<size_t>(t) * a.H + b * 16 + col;
    if (a.base) v += bf16_bits_to_f32(to_global(a.base)[at]);
    to_global(a.out)[at] = f32_to_bf16_bits(v);
  };
  if (total == 0) {  // no live token
    for (int i = blockIdx.x * kMlThreads + tid; i < a.T * a.H; i += gridDim.x * kMlThreads)
      write(i % a.H / 16, i / a.H, i % 16, 0.f);
    return;
  }
  // every workgroup that takes part holds a unit, so it counts itself in
  const int NW = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  if (static_cast<int>(blockIdx.x) >= NW) return;
  auto first_of = [&](int w) { return total * w / NW; };
  // the workgroup that holds a unit
  auto owner_of = [&](long long u) { return static_cast<int>(((u + 1) * NW - 1) / total); };
  const long long begin = first_of(blockIdx.x), end = first_of(blockIdx.x + 1);
  const size_t words = static_cast<size_t>(blocks) * groups * 64 * U::WPL;  // of one expert
  const size_t scales = static_cast<size_t>(blocks) * groups * 16;

  // The workgroup's units, block by block: a step is a unit for each of its waves,
  // and a block's last step may leave some without one. Loads run AHEAD steps
  // before the arithmetic, over the blocks' ends; the two places move alike.
  struct Walk {
    int b;                 // block
    long long pos, stop;   // first unit of the step; end of this block's units here
  };
  auto start = [&](Walk& k) {
    k.b = static_cast<int>(begin / per);
    k.pos = begin;
    k.stop = min(end, static_cast<long long>(k.b + 1) * per);
  };
  auto advance = [&](Walk& k) {
    k.pos += kMlWaves;
    if (k.pos >= k.stop) {
      k.pos = k.stop;
      if (k.stop < end) {
        ++k.b;
        k.stop = min(end, k.stop + per);
      }
    }
  };
  struct Stage {
    MlWeights<GS> w;
    MlRows<GS> h;
    int at, u;  // entry and unit of the expert
  };
  Stage st[AHEAD];
  auto load = [&](Stage& s, const Walk& k) {
    const long long unit = min(k.pos + wave, k.stop - 1);  // past the last: not used
    const int rest = static_cast<int>(unit - static_cast<long long>(k.b) * per);
    s.at = rest / units;
    s.u = rest - s.at * units;
    const int e = tb.expert[s.at];
    const size_t off = static_cast<size_t>(k.b) * groups;
    load_unit<GS>(s.w, to_global(a.down) + e * words + off * 64 * U::WPL + lane * U::WPL,
                  reinterpret_cast<gptr<const uint32_t>>(to_global(a.down_scales) + e * scales + off * 16 + (c16 & ~1)),
                  s.u, groups);
    // rows of other tokens: any row, their results are left out
    const bool mine = tb.mask[s.at] >> c16 & 1;
    const size_t slot = mine ? static_cast<size_t>(c16) * a.top_k + tb.place[s.at * 16 + c16] : 0;
    load_rows<GS>(s.h, to_global(a.h) + slot * a.I, s.u, groups);
  };
  Walk now, then;
  start(now);
  start(then);
#pragma unroll
  for (int p = 0; p < AHEAD; ++p) {
    load(st[p], then);
    advance(then);
  }

  const bf16x8 bias = bias_operand();
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  auto unit = [&](const Stage& s) {
    const f32x4 wt = *reinterpret_cast<const f32x4*>(tb.weight + s.at * 16 + 4 * lg);
    const int live = static_cast<uint16_t>(tb.mask[s.at]) >> (4 * lg);
#pragma unroll
    for (int g = 0; g < U::G; ++g) {
      if (U::G > 1 && s.u * U::G + g >= groups) break;  // uniform: K ends inside the unit
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < U::WPL; ++w) acc = mfma16(act_frag(s.h.d[g * U::WPL + w]), bias, acc);
#pragma unroll
      for (int w = 0; w < U::WPL; ++w)
        acc = mfma16(act_frag(s.h.d[g * U::WPL + w]), dequant_biased(s.w.w[g * U::WPL + w]), acc);
      const float sc = scale_of(s.w.s[g], lane);
      // a row that is not the expert's takes nothing from it, whatever its values
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = live >> r & 1 ? __builtin_fmaf(sc * wt[r], acc[r], y[r]) : y[r];
    }
  };
  int turn = 0, side = 0;
  // the end of the units [seg, stop) of block b
  auto finish = [&](int b, long long stop) {
    float* const mine = red + turn * kRedFloats;
    turn ^= 1;
#pragma unroll
    for (int r = 0; r < 4; ++r) mine[(wave * 4 + r) * 64 + lane] = y[r];
    y = f32x4{0.f, 0.f, 0.f, 0.f};
    lds_barrier();
    const int t = 4 * lg + (tid >> 6);  // of threads 0 .. 255
    float v = 0.f;
    if (tid < 256) {
#pragma unroll
      for (int w = 0; w < kMlWaves; ++w) v += mine[(w * 4 + (tid >> 6)) * 64 + lane];
    }
    const long long b0 = static_cast<long long>(b) * per;
    if (begin <= b0 && stop == b0 + per) {
      if (tid < 256 && t < a.T) write(b, t, c16, v);
    } else {
      // The block lies with several workgroups: the last to count itself in adds
      // the parts in the order of the workgroups. A workgroup's part of the block
      // it starts in is its first, of a later one its second.
      const int w0 = owner_of(b0), w1 = owner_of(b0 + per - 1);
      if (tid < 256)
        __hip_atomic_store(a.parts + (static_cast<size_t>(blockIdx.x) * 2 + side) * kMlPartFloats + tid, v,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      wait_vmem_all();
      __syncthreads();
      if (tid == 0)
        last_flag = __hip_atomic_fetch_add(a.counters + b, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == w1 - w0;
      __syncthreads();
      if (last_flag && tid < 256 && t < a.T) {
        float s = 0.f;
        for (int w = w0; w <= w1; ++w) {
          const int its = first_of(w) >= b0 ? 0 : 1;
          s += __hip_atomic_load(a.parts + (static_cast<size_t>(w) * 2 + its) * kMlPartFloats + tid, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
        }
        write(b, t, c16, s);
      }
    }
    side = 1;
  };
  for (bool done = false; !done;) {
#pragma unroll
    for (int p = 0; p < AHEAD; ++p) {
      if (done) continue;
      if (now.pos + wave < now.stop) unit(st[p]);
      load(st[p], then);
      advance(then);
      const Walk was = now;
      advance(now);
      if (was.pos + kMlWaves >= was.stop) {
        finish(was.b, was.stop);
        done = was.stop >= end;
      }
    }
  }
}

// ---------------------------------------------------------------- launches

template <typename F>
hipError_t with_lds(F* kernel, size_t lds) {
  if (lds <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(lds));
}

template <int GS, int KU>
hipError_t launch_gate_up(const MlArgs& a, hipStream_t stream) {
  const size_t lds = gate_up_scratch(a.E) + ml_plan_bytes(a.most, a.E);
  auto* kernel = &gate_up_kernel<GS, KU>;
  const hipError_t e = with_lds(kernel, lds);
  if (e != hipSuccess) return e;
  const long long tasks = static_cast<long long>(a.most) * (a.I / 16);
  const int grid = static_cast<int>(tasks < kModelCUs ? tasks : kModelCUs);
  kernel<<<dim3(grid), dim3(kMlThreads), lds, stream>>>(a);
  return hipGetLastError();
}

template <int GS>
hipError_t launch_moe_layer_g(const MlArgs& a, bool half, hipStream_t stream) {
  using U = MlUnit<GS>;
  if (half)
    router_kernel<true><<<dim3(a.E), dim3(kMlRouterThreads), 0, stream>>>(a);
  else
    router_kernel<false><<<dim3(a.E), dim3(kMlRouterThreads), 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = a.H / GS, units = (groups + U::G - 1) / U::G;
  const int held = (units + kMlWaves - 1) / kMlWaves * U::F / 4;  // 128s of K per wave
  if (held <= 2)
    e = launch_gate_up<GS, 2 * 4 / U::F>(a, stream);
  else if (held <= 4)
    e = launch_gate_up<GS, 4 * 4 / U::F>(a, stream);
  else if (held == 5 && U::F == 4)
    e = launch_gate_up<GS, U::F == 4 ? 5 : 0>(a, stream);
  else if (held <= 6)
    e = launch_gate_up<GS, 6 * 4 / U::F>(a, stream);
  else
    e = launch_gate_up<GS, 0>(a, stream);
  if (e != hipSuccess) return e;
  const size_t lds = 2 * kMlWaves * 256 * 4 + ml_plan_bytes(a.most, a.E);
  constexpr int kAhead = U::F == 4 ? 4 : 2;
  auto* kernel = &down_kernel<GS, kAhead>;
  e = with_lds(kernel, lds);
  if (e != hipSuccess) return e;
  kernel<<<dim3(kModelCUs), dim3(kMlThreads), lds, stream>>>(a);
  return hipGetLastError();
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

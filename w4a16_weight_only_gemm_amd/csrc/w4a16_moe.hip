// w4a16_moe.hip -- routing of tokens to experts, and the weighted sum of the
// experts' rows back into token order.
//
// Routing (w4a16_moe_route). One wave per token, each lane holding P experts.
// An expert gets an integer key whose order is the order of choice, with the
// expert's place in its lane in the lowest bits. A lane sorts its keys once;
// each choice is then one maximum over the lanes' first keys (six DPP steps, no
// LDS), the lane that holds it moving up by one. Keys too near to tell are
// sorted out afterwards, and only among the choices and those next to them:
//  * Without bias and groups the choice is by score, which grows with the
//    logit: the key is the logit's own bits, order-preserving. bf16 keys are
//    exact; fp32 logits whose keys differ in the lowest bits only are compared
//    again as they are.
//  * With a bias or groups the choice values are what the interface defines in
//    64 bits: in fp32 two experts a few 1e-8 apart could swap places. They are
//    first formed in fp32; choices nearer than a margin that covers every fp32
//    rounding on the way are formed in fp64, a lane each, and ordered by that. Of
//    groups only those kept and those dropped have to be apart;
//    where they are not, the token's groups are formed again in fp64. With 256
//    experts in 8 groups, sigmoid scores of normal logits (1.5) and biases (0.05),
//    choices are near for one token in 450, groups for one in 11,000 (this rule
//    over 200,000 tokens).
// The weights need the scores of the chosen experts only, in fp64: a thread per
// slot, after the workgroup's tokens are chosen (softmax without renormalisation
// also sums over all experts, in fp64).
// What bounds it: few tokens, the launches and the chain of dependent steps;
// many, the vector instructions of the rounds (8192 tokens of 256 experts, 8
// each, in groups: 14 us of 21; 6.9 us are the second launch). Choosing from
// unsorted keys with every near token decided again in fp64 took 23 us there.
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
// tokens. A token takes a wave some 2 to 4 us of dependent steps, so few tokens
// are spread over many workgroups; the second launch reads every chunk's
// counts in every workgroup, so many tokens are not. Measured at 256 experts,
// 8 per token (us, plain top-k / bias and groups):
//   1 token: one workgroup and launch 5.3 / 6.7
//   16 tokens: one workgroup and launch 7.0 / 9.6, 4 per workgroup and two
//     launches 8.5 / 9.8
//   64 tokens: 16 per workgroup 9.8 / 12.3, 4 per workgroup 8.9 / 10.1
//   2048 tokens: 4 per workgroup 15.0 / 17.3, 16 per workgroup 12.4 / 15.2
//   4096 tokens: 16 per workgroup 11.8 / 15.6, 32 per workgroup 16.0 / 21.4
constexpr int kRtOneLaunchTokens = 16;  // one launch up to here, and up to
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

// The number a key stands for.
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __builtin_bit_cast(double, k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}

// v of another lane: CTRL as in dpp_f32, for any 4- or 8-byte type; 0 where the
// pattern does not reach (ROWS: the rows written).
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_of(T v) {
  if constexpr (sizeof(T) == 4) {
    const int b = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, b, CTRL, ROWS, 0xF, false));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
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
// lanes, then from row to row into lane 63. A lane a step does not reach meets
// 0, so keys only.
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
// the bias' addition rounds at the choice value's own size. A group's sum of two
// carries both summands' roundings, each of its summand's size however small
// the sum is (biases of opposite sign), and its own. A decision compares two
// values, or two sums of two.
constexpr float kRtMarginSigmoid = 2e-6f;
constexpr float kRtMarginSoftmax = 1.6e-5f;  // of the largest score
constexpr float kRtMarginValue = 5e-7f;      // of the values' (a sum: summands') magnitude

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

// What a wave knows of a token: the logits of its lane's experts, and which of
// them can be chosen.
template <int P>
struct Token {
  size_t row;  // of its first logit
  float z[P];
  bool live[P];
};

// The i-th expert of a lane. Choice by value takes consecutive ones, so that
// groups are whole lanes; choice by logit takes every 64th, so that the order
// of (i, lane) is that of the experts and equal keys need no second look.
template <int P, bool WIDE>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return WIDE ? lane * P + i : i * 64 + lane;
}

// The top_k largest keys (0: never), one after the other, the lowest expert of
// equal ones first: lane j gets the j-th choice, -1 where nothing is left.
template <int P, bool WIDE, typename Key>
__device__ __forceinline__ int take(Key (&key)[P], int top_k, int lane) {
  int id = -1;
  for (int j = 0; j < top_k; ++j) {
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
    const uint32_t back = best == top ? kRtMaxExperts - expert_of<P, WIDE>(lane, bi) : 0;
    const int e = kRtMaxExperts - static_cast<int>(wave_max_of(back));
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (expert_of<P, WIDE>(lane, i) == e) key[i] = 0;
  }
  return id;
}

// The same from 32-bit keys whose low bits (P - 1, a mask) give way to P - 1 -
// i, so that a key names its expert within the lane: a lane's keys are sorted
// once by plain maxima and minima, and a round is one maximum over the lanes'
// first keys, after which the lane that held it moves its keys up.
// Keys that are not apart may be in the wrong order: past top_k the rounds go on
// until one is apart from the key before it. Lane j < the number returned gets
// the j-th key in rank and its expert in id; 65 says that 64 were not enough.
template <int P, bool WIDE, typename F>
__device__ __forceinline__ int take_packed(uint32_t (&key)[P], int top_k, int lane, uint32_t& rank,
                                           int& id, F apart) {
  // odd-even merge sort, descending
#pragma unroll
  for (int p = 1; p < P; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < P; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < P && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t x = key[i + j], y = key[i + j + k];
            key[i + j] = x > y ? x : y;
            key[i + j + k] = x > y ? y : x;
          }
  id = -1;
  rank = 0;
  uint32_t last = 0;
  auto accept = [&](int j, uint32_t top) {
    const int owner = __builtin_ctzll(__ballot(key[0] == top));
    const int e = expert_of<P, WIDE>(owner, P - 1 - static_cast<int>(top & (P - 1)));
    if (lane == j) {
      rank = top;
      id = e;
    }
    last = top;
    const uint32_t mine = lane == owner ? ~0u : 0;
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = (key[i] & ~mine) | ((i + 1 < P ? key[i + 1] : 0) & mine);
  };
  int j = 0;
  for (; j < top_k; ++j) {
    const uint32_t top = wave_max_of(key[0]);
    if (top == 0) return j;
    accept(j, top);
  }
  for (;; ++j) {
    const uint32_t top = wave_max_of(key[0]);
    if (top == 0 || apart(last, top)) return j;
    if (j == 64) return 65;
    accept(j, top);
  }
}

// Lanes 0 .. n - 1 hold different experts and their values: puts the experts in
// order of value, the lowest first among equal ones.
template <typename S>
__device__ __forceinline__ int in_order(int id, S value, int n, int lane) {
  int place = 0;
  for (int q = 0; q < n; ++q) {
    const S ov = lane_of(value, q);
    const int oe = __builtin_amdgcn_readlane(id, q);
    place += ov > value || (ov == value && oe < id);
  }
  return __builtin_amdgcn_ds_permute(4 * (lane < n ? place : lane), id);
}

// Largest logit of the token.
template <int P>
__device__ __forceinline__ float largest(const Token<P>& tk) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t k = tk.live[i] ? order_key(tk.z[i]) : 0;
    m = k > m ? k : m;
  }
  m = wave_max_of(m);
  return m ? value_of(m) : 0.f;
}

// The two largest of the lanes' keys (t1 >= t2) within runs of lg lanes, lg a power
// of two, in every lane of the run.
template <typename Key>
__device__ __forceinline__ void merge_pairs(Key& t1, Key& t2, int lg) {
  auto merge = [&](Key o1, Key o2) {
    const Key lo = t1 < o1 ? t1 : o1, hi2 = t2 > o2 ? t2 : o2;
    t1 = t1 > o1 ? t1 : o1;
    t2 = lo > hi2 ? lo : hi2;
  };
  // after a step all lanes of a run of that length hold the same, so a mirror
  // within twice the length reaches the other run
  if (lg >= 2) merge(dpp_of<0xB1, 0xF>(t1), dpp_of<0xB1, 0xF>(t2));
  if (lg >= 4) merge(dpp_of<0x4E, 0xF>(t1), dpp_of<0x4E, 0xF>(t2));
  if (lg >= 8) merge(dpp_of<0x141, 0xF>(t1), dpp_of<0x141, 0xF>(t2));
  if (lg >= 16) merge(dpp_of<0x140, 0xF>(t1), dpp_of<0x140, 0xF>(t2));
  for (int o = 16; o < lg; o <<= 1) {
    merge(__shfl_xor(t1, o), __shfl_xor(t2, o));
  }
}

// The choice values of the lane's experts in S, as keys (0 where not live), and
// for S = float the margin. sum: the softmax's.
template <int P, typename S, typename Key>
__device__ __forceinline__ void choice_keys(const RouteArgs& a, const Token<P>& tk, float zmax,
                                            int lane, Key (&key)[P], S& sum, float& margin) {
  S v[P];
  sum = 0;
  if (a.sigmoid) {
    margin = kRtMarginSigmoid;
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = reciprocal<S>(1 + exp_of<S>(-static_cast<S>(tk.z[i])));
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = exp_of<S>(static_cast<S>(tk.z[i]) - static_cast<S>(zmax));
      sum += tk.live[i] ? v[i] : 0;
    }
    sum = wave_sum_of(sum);  // 0: nothing is live
    margin = kRtMarginSoftmax / static_cast<float>(sum);  // the largest score is 1 / sum
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = sizeof(S) == 4 ? v[i] * reciprocal<S>(sum) : v[i] / sum;
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      v[i] += static_cast<S>(a.bias[min(expert_of<P, true>(lane, i), a.E - 1)]);
  }
#pragma unroll
  for (int i = 0; i < P; ++i)  // a NaN (from the bias) has no place in an order
    key[i] = tk.live[i] && v[i] == v[i] ? order_key(v[i]) : 0;
}

// Whether fp32 values hi >= lo are further apart than their errors.
__device__ __forceinline__ bool apart_by(float hi, float lo, float margin, float relative) {
  const float m = hi > -lo ? hi : -lo;  // the larger magnitude
  return hi - lo > margin + relative * m;
}

// keep: a bit per expert of the lane, whether its group is kept. Returns false,
// and no bits, where the groups kept and those dropped are not further apart than
// their errors (S = float): a value between the last one kept and the first one
// dropped has to lie outside every group's value +- half the margin. Any group
// may be the one that reaches it, as each errs by its own summands' size. vals: the
// wave's LDS.
template <int P, typename S, typename Key>
__device__ __forceinline__ bool keep_groups(const RouteArgs& a, Key (&key)[P], float margin, int lane,
                                            Key* vals, uint32_t& keep) {
  // a group's two largest values, by lg lanes (a power of two) each
  Key t1 = 0, t2 = 0;
  auto put = [&](Key x) {
    const Key lo = x < t1 ? x : t1;
    t2 = t2 > lo ? t2 : lo;
    t1 = x > t1 ? x : t1;
  };
  const int per = a.per, lg = a.group_lanes, g = lane / lg;
  if (a.group_whole) {  // the lanes that hold the group's experts
#pragma unroll
    for (int i = 0; i < P; ++i) put(key[i]);
  } else {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // behind the reads of an earlier use
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane * P + i < a.E) vals[lane * P + i] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (g < a.groups)
      for (int j = lane % lg; j < per; j += lg) put(vals[g * per + j]);
  }
  merge_pairs(t1, t2, lg);
  const S none = -static_cast<S>(__builtin_inff());
  S value = t1 ? value_of(t1) : none;
  if (a.group_top == 2 && t2) value += value_of(t2);
  // the groups with a larger value, or an equal one and a lower index
  int place = g < a.groups ? 0 : a.groups;
  for (int q = 0; q < a.groups; ++q) {
    const S ov = lane_of(value, q * lg);
    place += ov > value || (ov == value && g > q);
  }
  if constexpr (sizeof(S) == 4) {
    if (a.groups_kept < a.groups) {
      const S low = lane_of(value, __builtin_ctzll(__ballot(place == a.groups_kept - 1)));
      const S high = lane_of(value, __builtin_ctzll(__ballot(place == a.groups_kept)));
      if (high > none) {
        // half the margin a side: 4.2 half steps of fp32 of the summands' size; a
        // summand's rounding, the sum's and that of value +- error are 3. Infinite
        // sums fail either comparison.
        S size = t1 ? __builtin_fabsf(value_of(t1)) : 0.f;
        if (a.group_top == 2 && t2) size += __builtin_fabsf(value_of(t2));
        const S error = 0.5f * (margin + kRtMarginValue * size);
        const S between = 0.5f * low + 0.5f * high;
        const bool clear = place < a.groups_kept ? value - error > between : value + error < between;
        if (__any(g < a.groups && !clear)) return false;
      }
    }
  }
  const bool in = place < a.groups_kept;
  if (a.group_whole) {
    keep = in ? ~0u : 0;
  } else {
    const uint64_t kept = __ballot(in);
    keep = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int eg = static_cast<int>(__umulhi(lane * P + i, a.per_inverse));  // e / per
      keep |= static_cast<uint32_t>(kept >> (eg * lg & 63) & 1) << i;
    }
  }
  return true;
}

// Choice by values (bias or groups): lane j < top_k gets the j-th choice.
// Decisions in fp32, those nearer than the margin again in fp64. vals: the
// wave's LDS.
template <int P>
__device__ __forceinline__ int choose_by_value(const RouteArgs& a, const Token<P>& tk, float zmax,
                                               int lane, double* vals) {
  uint32_t key[P], rank, keep = ~0u;
  uint64_t wide[P];
  float sum, margin, unused;
  double wsum = 1.0;
  choice_keys<P>(a, tk, zmax, lane, key, sum, margin);
  if (a.groups > 1 &&
      !keep_groups<P, float>(a, key, margin, lane, reinterpret_cast<uint32_t*>(vals), keep)) {
    choice_keys<P>(a, tk, zmax, lane, wide, wsum, unused);
    keep_groups<P, double>(a, wide, 0.f, lane, reinterpret_cast<uint64_t*>(vals), keep);
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    key[i] = (keep >> i & 1) && key[i] ? (key[i] & ~static_cast<uint32_t>(P - 1)) | (P - 1 - i) : 0;
  // dropped key bits are at most P - 1 units of 2^-23 of the value
  auto apart = [&](uint32_t hi, uint32_t lo) {
    return apart_by(value_of(hi & ~(P - 1u)), value_of(lo & ~(P - 1u)), margin,
                    kRtMarginValue + P * 0x1p-23f);
  };
  int id;
  const int n = take_packed<P, true>(key, a.top_k, lane, rank, id, apart);
  const uint32_t before = __shfl_up(rank, 1);
  const bool near = lane > 0 && lane < n && !apart(before, rank);
  if (!__any(near)) return id;
  if (n > 64 || !a.sigmoid) choice_keys<P>(a, tk, zmax, lane, wide, wsum, unused);
  if (n > 64) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (!(keep >> i & 1)) wide[i] = 0;
    return take<P, true>(wide, a.top_k, lane);
  }
  // the candidates' own values
  double x = 0.0;
  if (id >= 0) {
    float z = load_logit(a, tk.row + id);
    live_logit(z);
    x = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(z)))
                  : exp(static_cast<double>(z) - static_cast<double>(zmax)) / wsum;
    if (a.bias) x += static_cast<double>(a.bias[id]);
  }
  return in_order(id, x, n, lane);
}

// The choices of token t, by one wave: lane j < top_k gets the j-th, or -1.
// P: experts per lane. WIDE: bias or groups. vals: this wave's LDS for E choice
// values (WIDE). zmax: the largest logit, for a softmax that needs it before
// the choices are known (by value, or not renormalised); sum: the softmax's
// where it is not renormalised.
template <int P, bool WIDE>
__device__ __forceinline__ int choose(const RouteArgs& a, int t, int lane, double* vals, float& zmax,
                                      double& sum) {
  Token<P> tk;
  tk.row = static_cast<size_t>(t) * a.E;
  if (a.bf16) {
    const uint16_t* z = static_cast<const uint16_t*>(a.logits) + tk.row;
#pragma unroll
    for (int i = 0; i < P; ++i)
      tk.z[i] = __builtin_bit_cast(
          float, static_cast<uint32_t>(z[min(expert_of<P, WIDE>(lane, i), a.E - 1)]) << 16);
  } else {
    const float* z = static_cast<const float*>(a.logits) + tk.row;
#pragma unroll
    for (int i = 0; i < P; ++i) tk.z[i] = z[min(expert_of<P, WIDE>(lane, i), a.E - 1)];
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    tk.live[i] = live_logit(tk.z[i]) && expert_of<P, WIDE>(lane, i) < a.E;
  int id;
  zmax = 0.f;
  if (!a.sigmoid && (WIDE || !a.renormalize)) zmax = largest(tk);
  if constexpr (WIDE) {
    id = choose_by_value<P>(a, tk, zmax, lane, vals);
  } else {
    uint32_t key[P], rank;
#pragma unroll
    for (int i = 0; i < P; ++i)
      key[i] = tk.live[i] ? (order_key(tk.z[i]) & ~static_cast<uint32_t>(P - 1)) | (P - 1 - i) : 0;
    // bf16 leaves the low bits free; fp32 keys may differ only there
    auto apart = [&](uint32_t hi, uint32_t lo) { return a.bf16 || (hi ^ lo) >= P; };
    const int n = take_packed<P, false>(key, a.top_k, lane, rank, id, apart);
    const uint32_t before = __shfl_up(rank, 1);
    if (n > 64) {
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = tk.live[i] ? order_key(tk.z[i]) : 0;
      id = take<P, false>(key, a.top_k, lane);
    } else if (__any(lane > 0 && lane < n && !apart(before, rank))) {
      float z = 0.f;
      if (id >= 0) {
        z = load_logit(a, tk.row + id);
        live_logit(z);
      }
      id = in_order(id, z, n, lane);
    }
  }
  sum = 1.0;
  if (!a.sigmoid && !a.renormalize) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (tk.live[i]) part += exp(static_cast<double>(tk.z[i]) - zmax);
    sum = wave_sum_of(part);
  }
  return id;
}

struct RouteLds {
  alignas(16) int ids[kRtMaxSlots];  // this chunk's, in whole groups of four
  double score[kRtMaxSlots];         // the chosen experts'
  double sum[kRtChunk];              // choose()'s, per token
  float zmax[kRtChunk];
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
    float zmax;
    double sum;
    const int id =
        choose<P, WIDE>(a, t0 + i, lane, rt_vals + static_cast<size_t>(wave) * a.E, zmax, sum);
    if (lane < a.top_k) {
      l.ids[i * a.top_k + lane] = id;
      if (id >= 0) atomicAdd(&l.count[id], 1);  // integer sums: the order does not matter
    }
    if (lane == 0) {
      l.zmax[i] = zmax;
      l.sum[i] = sum;
    }
  }
  __syncthreads();
  // the weights, a thread per slot
  const int n = tokens * a.top_k;
  auto logit = [&](int s, int id) {
    float z = load_logit(a, static_cast<size_t>(t0 + s / a.top_k) * a.E + id);
    live_logit(z);
    return z;
  };
  for (int s = tid; s < n; s += 64 * W) {
    const int id = l.ids[s];
    double score = 0.0;
    if (id >= 0) {
      const double z = logit(s, id);
      if (a.sigmoid) {
        score = 1.0 / (1.0 + exp(-z));
      } else {
        const int i = s / a.top_k;  // by logit the first choice has the largest
        const float zmax = WIDE || !a.renormalize ? l.zmax[i] : logit(s, l.ids[i * a.top_k]);
        score = exp(z - zmax);
      }
    }
    l.score[s] = score;
  }
  __syncthreads();
  for (int s = tid; s < n; s += 64 * W) {
    const int i = s / a.top_k;
    double total = l.sum[i];
    if (a.renormalize) {  // the softmax's own sum cancels
      total = 0.0;
      for (int j = 0; j < a.top_k; ++j) total += l.score[i * a.top_k + j];
    }
    const size_t at = static_cast<size_t>(t0) * a.top_k + s;
    a.ids[at] = l.ids[s];
    a.weights[at] = total > 0.0 ? static_cast<float>(l.score[s] * static_cast<double>(a.scale) / total) : 0.f;
  }
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
    if (tid < count_stride(a.E)) l.total[tid] = 0;
    __syncthreads();
    // four experts (one word of a chunk's counts) per thread, the chunks dealt
    // out over the threads left; a total and its part before this chunk share a
    // word, at most kRtSumChunks * kRtChunk each
    static_assert(kRtSumChunks * kRtChunk < 1 << 15, "two counts in a word");
    const int words = count_stride(a.E) / 4;
    int width = 1;
    while (width < words) width <<= 1;
    const int wd = tid & (width - 1), step = kRtThreads / width;
    if (wd < words) {
      uint32_t sum[4] = {0, 0, 0, 0};
      const uint32_t* h = reinterpret_cast<const uint32_t*>(a.counts) + wd;
#pragma unroll 16
      for (int r = tid / width; r < a.chunks; r += step) {
        const uint32_t v = h[static_cast<size_t>(r) * words];
        const uint32_t twice = r < c ? 0x10001u : 1u;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += (v >> (8 * i) & 255) * twice;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (sum[i]) atomicAdd(&l.total[4 * wd + i], static_cast<int>(sum[i]));
    }
    __syncthreads();
    if (tid < a.E) {
      const uint32_t both = l.total[tid];
      l.total[tid] = both & 0xFFFF;
      l.before[tid] = both >> 16;
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

// VEC consecutive columns of one token per thread: 8, or 1 for fewer than 8
// columns. Rows start at any even address; the card's global accesses of 16
// bytes need no more (1472 tokens of 8 rows of 4588: 30 us, column by column 101).
// A row's last piece begins 8 columns before its end, and its thread writes
// only the columns behind the piece before.
template <int VEC>
__global__ __launch_bounds__(kCbThreads) void combine_kernel(const CombineArgs a) {
  typedef uint16_t vec __attribute__((ext_vector_type(VEC), aligned(2)));
  const int per = (a.N + VEC - 1) / VEC;
  const long long all = static_cast<long long>(per) * a.T;
  const long long step = static_cast<long long>(gridDim.x) * kCbThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kCbThreads + threadIdx.x; i < all; i += step) {
    const int t = static_cast<int>(i / per);
    const int n = static_cast<int>(i - static_cast<long long>(t) * per) * VEC;
    const int n0 = min(n, a.N - VEC);
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
    const size_t at = static_cast<size_t>(t) * a.N + n0;
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
      const vec y = *reinterpret_cast<const vec*>(a.y + (slot0 + j) * a.N + n0);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        acc[v] = __builtin_fmaf(w, __builtin_bit_cast(float, static_cast<uint32_t>(y[v]) << 16), acc[v]);
    }
    vec o;
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = f32_to_bf16_bits(acc[v]);
    if (n0 == n) {
      *reinterpret_cast<vec*>(a.out + at) = o;
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (n0 + v >= n) a.out[at + v] = o[v];
    }
  }
}

}  // namespace

// Enough for every number of tokens up to T: chunks are larger for more tokens,
// so the ends of the ranges count too.
size_t route_workspace_bytes(int T, int E) {
  size_t most = 0;
  for (int t : {T < kRtFewTokens ? T : kRtFewTokens, T < kRtMidTokens ? T : kRtMidTokens, T}) {
    if (route_one(t, E)) continue;
    size_t n = counts_bytes(t, E);
    if (route_chunks(t) > kRtSumChunks) n += (static_cast<size_t>(route_chunks(t)) + 1) * E * sizeof(int);
    most = n > most ? n : most;
  }
  return most;
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
  const int vec = a.N >= 8 ? 8 : 1;
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

// w4a16_moe_host.cpp -- host half of include/w4a16_moe.h: sizes, packing and
// argument checks. Nothing here touches a device except the launch calls.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/w4a16_moe.h"
#include "w4a16_moe_launch.h"

namespace {

constexpr long long kMaxSlots = 1LL << 30;
constexpr long long kMaxRoutedSlots = 1LL << 26;
constexpr int kMaxCombineColumns = 0x7FFFFFF8;   // rounded up to 8 still an int
constexpr long long kMaxBuffer = 0xFFFFFE00LL;  // bytes a 32-bit buffer resource may span

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The launchers return hipErrorNotSupported, before any launch, for a grid of
// more than 2^32 threads.
int status(hipError_t e) {
  return e == hipSuccess ? W4A16_OK : e == hipErrorNotSupported ? W4A16_ERR_UNSUPPORTED : W4A16_ERR_LAUNCH;
}

// byte j of a 16-block holds the code of offset kOrder[j] (as w4a8_quantize)
constexpr int kOrder[16] = {0, 4, 1, 5, 2, 6, 3, 7, 8, 12, 9, 13, 10, 14, 11, 15};

}  // namespace

extern "C" {

size_t w4a16_moe_route_workspace_bytes(int T, int experts) {
  if (T < 0 || experts < 1 || experts > W4A16_ROUTE_MAX_EXPERTS) return 0;
  return w4a16_internal::route_workspace_bytes(T, experts);
}

int w4a16_moe_route(const void* logits, const float* bias, const w4a16_route_config* c, int T,
                    int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!c || T < 0) return W4A16_ERR_INVALID_ARG;
  if (c->experts < 1 || c->experts > W4A16_ROUTE_MAX_EXPERTS) return W4A16_ERR_INVALID_ARG;
  if (c->top_k < 1 || c->top_k > W4A16_ROUTE_MAX_TOP_K || c->top_k > c->experts)
    return W4A16_ERR_INVALID_ARG;
  if (c->scoring != W4A16_ROUTE_SOFTMAX && c->scoring != W4A16_ROUTE_SIGMOID)
    return W4A16_ERR_INVALID_ARG;
  if (c->logits_type != W4A16_LOGITS_F32 && c->logits_type != W4A16_LOGITS_BF16)
    return W4A16_ERR_INVALID_ARG;
  if (c->groups < 1 || c->groups > W4A16_ROUTE_MAX_GROUPS || c->experts % c->groups != 0)
    return W4A16_ERR_INVALID_ARG;
  if (c->groups_kept < 1 || c->groups_kept > c->groups) return W4A16_ERR_INVALID_ARG;
  if (c->group_top != 1 && c->group_top != 2) return W4A16_ERR_INVALID_ARG;
  if (!std::isfinite(c->scale)) return W4A16_ERR_INVALID_ARG;
  if (!offsets) return W4A16_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !ids || !weights || !rows)) return W4A16_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * c->top_k > kMaxRoutedSlots) return W4A16_ERR_UNSUPPORTED;
  const size_t need = w4a16_internal::route_workspace_bytes(T, c->experts);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(workspace, 16) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(rows, 4))
    return W4A16_ERR_MISALIGNED;
  w4a16_internal::RouteArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.workspace = workspace;
  a.T = T;
  a.E = c->experts;
  a.top_k = c->top_k;
  a.sigmoid = c->scoring == W4A16_ROUTE_SIGMOID;
  a.bf16 = c->logits_type == W4A16_LOGITS_BF16;
  a.groups = c->groups;
  a.groups_kept = c->groups_kept;
  a.group_top = c->group_top;
  a.renormalize = c->renormalize != 0;
  a.scale = c->scale;
  return status(w4a16_internal::launch_route(a, stream));
}

int w4a16_gemm_experts(const void* x, const void* qweight, const void* scales, void* y,
                       const int32_t* rows, const int32_t* offsets, int slots, int experts,
                       int x_div, int N, int K, int group, int act, hipStream_t stream) {
  if (slots < 0 || N < 0 || K < 0 || x_div < 1 || experts < 1 ||
      experts > W4A16_ROUTE_MAX_EXPERTS)
    return W4A16_ERR_INVALID_ARG;
  if (act != W4A16_ACT_NONE && act != W4A16_ACT_SWIGLU) return W4A16_ERR_INVALID_ARG;
  if (slots == 0) return W4A16_OK;
  if (!x || !qweight || !scales || !y || !rows || !offsets) return W4A16_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128 && group != 256) return W4A16_ERR_UNSUPPORTED;
  if (N < 1 || K < 1 || K % group != 0 || slots > kMaxSlots) return W4A16_ERR_UNSUPPORTED;
  if (act == W4A16_ACT_SWIGLU && N % 32 != 0) return W4A16_ERR_UNSUPPORTED;
  const long long x_rows = (static_cast<long long>(slots) + x_div - 1) / x_div;
  if (x_rows > kMaxBuffer / (2LL * K)) return W4A16_ERR_UNSUPPORTED;
  if (w4a16_qweight_bytes(N, K) > static_cast<size_t>(kMaxBuffer)) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(qweight, 16) || !aligned(scales, 16) || !aligned(y, 16) ||
      !aligned(rows, 4) || !aligned(offsets, 4))
    return W4A16_ERR_MISALIGNED;
  w4a16_internal::ExpertsArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.qweight = static_cast<const uint32_t*>(qweight);
  a.scales = static_cast<const uint16_t*>(scales);
  a.y = static_cast<uint16_t*>(y);
  a.rows = rows;
  a.offsets = offsets;
  a.slots = slots;
  a.E = experts;
  a.x_div = x_div;
  a.N = N;
  a.K = K;
  a.group = group;
  a.swiglu = act == W4A16_ACT_SWIGLU;
  return status(w4a16_internal::launch_experts(a, stream));
}

int w4a16_moe_combine(const void* y, const int32_t* ids, const float* weights, const void* base,
                      void* out, int T, int top_k, int N, hipStream_t stream) {
  if (T < 0 || N < 0 || top_k < 1 || top_k > W4A16_ROUTE_MAX_TOP_K) return W4A16_ERR_INVALID_ARG;
  if (T == 0) return W4A16_OK;
  if (!y || !ids || !weights || !out) return W4A16_ERR_INVALID_ARG;
  if (N < 1 || N > kMaxCombineColumns || static_cast<long long>(T) * top_k > kMaxSlots)
    return W4A16_ERR_UNSUPPORTED;
  if (!aligned(y, 16) || !aligned(base, 16) || !aligned(out, 16) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return W4A16_ERR_MISALIGNED;
  w4a16_internal::CombineArgs a;
  a.y = static_cast<const uint16_t*>(y);
  a.ids = ids;
  a.weights = weights;
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  a.T = T;
  a.top_k = top_k;
  a.N = N;
  return status(w4a16_internal::launch_combine(a, stream));
}

size_t w8a8_qweight_bytes(int N, int K) {
  if (N < 0 || K < 0 || K % 16 != 0) return 0;
  return (static_cast<size_t>(N) + 15) / 16 * 1024 * ((static_cast<size_t>(K) + 63) / 64);
}

int w8a8_pack(const int8_t* q, int8_t* out, int N, int K) {
  if (N < 0 || K < 0 || K % 16 != 0) return W4A16_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return W4A16_OK;
  if (!q || !out) return W4A16_ERR_INVALID_ARG;
  const size_t blocks = (static_cast<size_t>(N) + 15) / 16, steps = (static_cast<size_t>(K) + 63) / 64;
  for (size_t b = 0; b < blocks; ++b)
    for (size_t t = 0; t < steps; ++t)
      for (int l = 0; l < 64; ++l) {
        const size_t n = b * 16 + l % 16, k = t * 64 + 16 * (l / 16);
        const bool there = n < static_cast<size_t>(N) && k < static_cast<size_t>(K);
        for (int j = 0; j < 16; ++j)
          *out++ = there ? q[n * K + k + kOrder[j]] : static_cast<int8_t>(0);
      }
  return W4A16_OK;
}

int w8a8_gemm(const void* xq, const float* sx, const void* qweight, const float* sw, void* y,
              int M, int N, int K, hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0) return W4A16_ERR_INVALID_ARG;
  if (M == 0) return W4A16_OK;
  if (!xq || !sx || !qweight || !sw || !y) return W4A16_ERR_INVALID_ARG;
  if (N < 1 || K < 16 || K % 16 != 0 || K > 131072) return W4A16_ERR_UNSUPPORTED;
  if (w8a8_qweight_bytes(N, K) > static_cast<size_t>(kMaxBuffer)) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(xq, 16) || !aligned(qweight, 16) || !aligned(y, 16) || !aligned(sx, 4) ||
      !aligned(sw, 4))
    return W4A16_ERR_MISALIGNED;
  w4a16_internal::W8A8Args a;
  a.xq = static_cast<const uint8_t*>(xq);
  a.sx = sx;
  a.qweight = static_cast<const uint8_t*>(qweight);
  a.sw = sw;
  a.y = static_cast<uint16_t*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  return status(w4a16_internal::launch_w8a8(a, stream));
}

}  // extern "C"

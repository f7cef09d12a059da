// w4a16_layer_host.cpp -- host half of include/w4a16_layer.h: argument checks.
// Nothing here touches a device except the launch calls.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/w4a16_layer.h"
#include "w4a16_layer_launch.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool group_supported(int group) { return group == 32 || group == 64 || group == 128 || group == 256; }

// The launchers return hipErrorNotSupported, before any launch, for what no grid
// holds.
int status(hipError_t e) {
  return e == hipSuccess ? W4A16_OK : e == hipErrorNotSupported ? W4A16_ERR_UNSUPPORTED : W4A16_ERR_LAUNCH;
}

constexpr int kMaxColumns = 0x7FFFFFF0;      // rounded up to 16 still an int
constexpr size_t kMaxMatrix = 0xFFFFFE00u;  // bytes of one expert's packed matrix

}  // namespace

extern "C" {

int w4a16_gemm_epilogue(const void* x, const void* qweight, const void* scales, const w4a16_epilogue* ep, void* y,
                        int M, int N, int K, int group, hipStream_t stream) {
  if (!ep || M < 0 || N < 0 || K < 0) return W4A16_ERR_INVALID_ARG;
  if (ep->act < W4A16_ACT_NONE || ep->act > W4A16_ACT_GEGLU || !std::isfinite(ep->scale)) return W4A16_ERR_INVALID_ARG;
  if (M == 0) return W4A16_OK;
  if (!x || !qweight || !scales || !y) return W4A16_ERR_INVALID_ARG;
  if (N < 1 || K < 1 || !group_supported(group) || K % group != 0) return W4A16_ERR_UNSUPPORTED;
  if (N > kMaxColumns) return W4A16_ERR_UNSUPPORTED;
  const bool gated = ep->act == W4A16_ACT_SWIGLU || ep->act == W4A16_ACT_GEGLU;
  if (gated && N % 32 != 0) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(qweight, 16) || !aligned(scales, 16) || !aligned(y, 16) ||
      !aligned(ep->residual, 16) || !aligned(ep->bias, 2))
    return W4A16_ERR_MISALIGNED;
  w4a16_internal::GemmArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.qweight = static_cast<const uint32_t*>(qweight);
  a.scales = static_cast<const uint16_t*>(scales);
  a.y = static_cast<uint16_t*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = group;
  w4a16_internal::Epilogue e;
  e.bias = static_cast<const uint16_t*>(ep->bias);
  e.residual = static_cast<const uint16_t*>(ep->residual);
  e.scale = ep->scale;
  e.act = ep->act;
  return status(w4a16_internal::launch_epilogue(a, e, stream));
}

int w4a16_norm(const w4a16_norm_args* a, int T, int N, hipStream_t stream) {
  if (!a || T < 0 || N < 0) return W4A16_ERR_INVALID_ARG;
  if (a->kind != W4A16_NORM_RMS && a->kind != W4A16_NORM_LAYER) return W4A16_ERR_INVALID_ARG;
  if (a->residual_type != W4A16_RESIDUAL_BF16 && a->residual_type != W4A16_RESIDUAL_F32) return W4A16_ERR_INVALID_ARG;
  if (!std::isfinite(a->eps) || a->eps < 0.f) return W4A16_ERR_INVALID_ARG;
  if (a->y && (!std::isfinite(a->scale) || a->gate_rows < 1)) return W4A16_ERR_INVALID_ARG;
  if (!a->xq != !a->sx || (a->xq && a->x)) return W4A16_ERR_INVALID_ARG;
  if (!a->y && !a->residual) return W4A16_ERR_INVALID_ARG;
  if (!a->residual_out && !a->x && !a->xq) return W4A16_ERR_INVALID_ARG;
  if (T == 0) return W4A16_OK;
  if (N < 1 || N > W4A16_NORM_MAX_COLUMNS || (a->xq && N % 16 != 0)) return W4A16_ERR_UNSUPPORTED;
  if (!aligned(a->y, 16) || !aligned(a->residual, 16) || !aligned(a->residual_out, 16) || !aligned(a->x, 16) ||
      !aligned(a->xq, 16) || !aligned(a->sx, 4) || !aligned(a->weight, 2) || !aligned(a->bias, 2))
    return W4A16_ERR_MISALIGNED;
  if (a->y && (!aligned(a->gate, 16) || !aligned(a->post_weight, 2) || !aligned(a->post_bias, 2)))
    return W4A16_ERR_MISALIGNED;
  return status(w4a16_internal::launch_norm(*a, T, N, stream));
}

size_t w4a16_moe_layer_workspace_bytes(int T, int experts, int top_k, int hidden, int width) {
  if (T < 0 || T > W4A16_MOE_LAYER_MAX_TOKENS || experts < 1 || experts > W4A16_ROUTE_MAX_EXPERTS || top_k < 1 ||
      top_k > W4A16_ROUTE_MAX_TOP_K || top_k > experts || hidden < 1 || width < 1)
    return 0;
  return w4a16_internal::moe_layer_workspace_bytes(T, experts, top_k, hidden, width);
}

int w4a16_moe_layer(const w4a16_moe_layer_args* l, const void* x, const int32_t* live, const void* base, void* out,
                    int32_t* ids, float* weights, int T, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!l || T < 0 || l->hidden < 0 || l->width < 0) return W4A16_ERR_INVALID_ARG;
  const w4a16_route_config& c = l->route;
  if (c.experts < 1 || c.experts > W4A16_ROUTE_MAX_EXPERTS) return W4A16_ERR_INVALID_ARG;
  if (c.top_k < 1 || c.top_k > W4A16_ROUTE_MAX_TOP_K || c.top_k > c.experts) return W4A16_ERR_INVALID_ARG;
  if (c.scoring != W4A16_ROUTE_SOFTMAX && c.scoring != W4A16_ROUTE_SIGMOID) return W4A16_ERR_INVALID_ARG;
  if (c.groups < 1 || c.groups > W4A16_ROUTE_MAX_GROUPS || c.experts % c.groups != 0) return W4A16_ERR_INVALID_ARG;
  if (c.groups_kept < 1 || c.groups_kept > c.groups) return W4A16_ERR_INVALID_ARG;
  if (c.group_top != 1 && c.group_top != 2) return W4A16_ERR_INVALID_ARG;
  if (!std::isfinite(c.scale)) return W4A16_ERR_INVALID_ARG;
  if (l->router_type != W4A16_LOGITS_F32 && l->router_type != W4A16_LOGITS_BF16) return W4A16_ERR_INVALID_ARG;
  if (T == 0) return W4A16_OK;
  if (!x || !out || !ids || !weights || !l->router || !l->gate_up || !l->gate_up_scales || !l->down || !l->down_scales)
    return W4A16_ERR_INVALID_ARG;
  if (T > W4A16_MOE_LAYER_MAX_TOKENS) return W4A16_ERR_UNSUPPORTED;
  const int H = l->hidden, I = l->width, group = l->group;
  if (H < 1 || I < 1 || !group_supported(group) || H % group != 0 || I % group != 0) return W4A16_ERR_UNSUPPORTED;
  // the matrices, and the inner rows, are read through 32-bit offsets
  if (I > 0x3FFFFFFF || w4a16_qweight_bytes(2 * I, H) > kMaxMatrix ||
      static_cast<size_t>(T) * c.top_k * I * 4 > kMaxMatrix)
    return W4A16_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < w4a16_moe_layer_workspace_bytes(T, c.experts, c.top_k, H, I))
    return W4A16_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(l->router, 16) || !aligned(l->gate_up, 16) || !aligned(l->gate_up_scales, 16) ||
      !aligned(l->down, 16) || !aligned(l->down_scales, 16) || !aligned(base, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256) || !aligned(live, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(l->route_bias, 4))
    return W4A16_ERR_MISALIGNED;
  w4a16_internal::MoeLayerArgs a;
  a.layer = *l;
  a.x = static_cast<const uint16_t*>(x);
  a.live = live;
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  a.ids = ids;
  a.weights = weights;
  a.workspace = static_cast<char*>(workspace);
  a.T = T;
  return status(w4a16_internal::launch_moe_layer(a, stream));
}

}  // extern "C"

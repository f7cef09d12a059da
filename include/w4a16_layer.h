/*
 * w4a16_layer.h -- C ABI of the operators that join the 4-bit products of a
 * decoder layer (libw4a16.so, MI355X / gfx950), beside w4a16.h and w4a16_moe.h:
 *
 *     w4a16_gemm_epilogue  w4a16_gemm with bias, activation (gated ones too),
 *                          scale and residual in its epilogue
 *     w4a16_norm           the norms behind and before a block with the block's
 *                          gate, its scale and the residual sum between them,
 *                          as bf16 rows or as the codes w4a8_quantize writes
 *     w4a16_moe_layer      a whole mixture-of-experts layer for a few tokens
 *
 * Ownership, threading, streams and errors are those of w4a16.h: the caller
 * owns every buffer, calls are asynchronous on `stream`, the library allocates
 * nothing and keeps no state, every check that can be made without reading
 * device memory is made before any launch, and a failed call launches nothing.
 * Every call can be captured into a HIP graph. Calls that can overlap must not
 * share outputs or a workspace. Device pointers belong to the current device.
 */
#ifndef W4A16_LAYER_H
#define W4A16_LAYER_H

#include "w4a16_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of w4a16_gemm_epilogue, beside W4A16_ACT_NONE (0) and
 * W4A16_ACT_SWIGLU (1). */
enum {
  W4A16_ACT_SILU = 2,      /* v / (1 + exp(-v)) */
  W4A16_ACT_GELU = 3,      /* v (1 + erf(v / sqrt 2)) / 2 */
  W4A16_ACT_GELU_TANH = 4, /* v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 */
  W4A16_ACT_RELU = 5,      /* max(v, 0); NaN stays NaN */
  W4A16_ACT_GEGLU = 6      /* columns 0 .. N/2-1 are gates, N/2 .. N-1 are ups:
                              gelu_tanh(gate) * up */
};

/* What follows the product. Checked by w4a16_gemm_epilogue. */
typedef struct w4a16_epilogue {
  const void* bias;     /* device bf16 [N], or NULL for 0 */
  const void* residual; /* device bf16 [M][N_out], or NULL for 0; may be y itself */
  float scale;          /* factor on the activated value, finite */
  int act;              /* W4A16_ACT_* */
} w4a16_epilogue;

/*
 * p[m][n] = sum_k x[m][k] * q[n][k] * s[n][k / group] + bias[n]
 * y[m][n] = residual[m][n] + scale * act(p[m][n])                   (N_out = N)
 * SWIGLU: y[m][n] = residual[m][n] + scale * silu(p[m][n]) * p[m][N/2 + n]
 * GEGLU:  the same with gelu_tanh                                 (N_out = N / 2)
 * with fp32 accumulation and epilogue and one rounding to bf16 (nearest even).
 * A residual is added last; without one nothing is added, so that -0 stays.
 * Without bias, residual and activation, and with scale 1, y has w4a16_gemm's
 * bits.
 *   x, qweight, scales, y and the supported M, N, K and group: as w4a16_gemm;
 *   y is bf16 [M][N_out] and overlaps no input but a residual of the same
 *   address. The gated activations need N % 32 == 0.
 * x, qweight, scales, y, residual 16-byte aligned, bias 2-byte. M == 0 launches
 * nothing. Needs no workspace. Returns W4A16_OK, W4A16_ERR_INVALID_ARG (null
 * pointer, negative size, act, scale), W4A16_ERR_UNSUPPORTED (shape),
 * W4A16_ERR_MISALIGNED or W4A16_ERR_LAUNCH.
 */
int w4a16_gemm_epilogue(const void* x, const void* qweight, const void* scales,
                        const w4a16_epilogue* epilogue, void* y, int M, int N, int K, int group,
                        struct ihipStream_t* stream);

#define W4A16_NORM_MAX_COLUMNS 65536

typedef enum {
  W4A16_NORM_RMS = 0,  /* v / sqrt(mean(v^2) + eps) */
  W4A16_NORM_LAYER = 1 /* (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) */
} w4a16_norm_kind;

typedef enum { W4A16_RESIDUAL_BF16 = 0, W4A16_RESIDUAL_F32 = 1 } w4a16_residual_type;

/* Everything w4a16_norm reads and writes. Checked by w4a16_norm. */
typedef struct w4a16_norm_args {
  /* the block that ends: y NULL for none, then the next six count for nothing */
  const void* y;           /* device bf16 [T][N], or NULL */
  int post_norm;           /* nonzero: y is normalised */
  int gate_rows;           /* rows of y that share a row of gate, >= 1 */
  const void* post_weight; /* device bf16 [N], or NULL for no weight */
  const void* post_bias;   /* device bf16 [N], or NULL for 0 */
  const void* gate;        /* device bf16 [ceil(T / gate_rows)][N], or NULL for 1 */
  float scale;             /* factor on the block's term, finite */
  /* the residual stream */
  int residual_type;    /* W4A16_RESIDUAL_*, of both */
  const void* residual; /* device [T][N], or NULL for 0 */
  void* residual_out;   /* device [T][N], or NULL: not written; may be residual itself */
  /* the next block's input: x, or xq and sx, or none of them */
  const void* weight; /* device bf16 [N], or NULL for no weight */
  const void* bias;   /* device bf16 [N], or NULL for 0 */
  void* x;            /* device bf16 [T][N], or NULL */
  void* xq;           /* device int8 [T][N], or NULL: codes in w4a8_quantize's arrangement */
  float* sx;          /* device f32 [T], or NULL: their scales */
  /* the norms */
  int kind;        /* W4A16_NORM_* */
  int unit_offset; /* nonzero: weights are held as their difference from 1 */
  float eps;       /* finite, >= 0 */
} w4a16_norm_args;

/*
 * For every row t, in fp32 and not rounded between the steps:
 *   u = y[t], normalised, times post_weight, plus post_bias, if post_norm is set
 *   r = residual[t] + scale * gate[t / gate_rows] * u
 *   v = r normalised, times weight, plus bias
 * residual_out[t] = r and x[t] = v, each rounded once (bf16 to nearest even).
 * With xq and sx instead of x: a = max |v|, sx[t] = a / 127, codes v * (127 / a)
 * rounded to the nearest integer (ties to even) in -127 .. 127; 0 and sx 0 for a
 * row of zeros. Inputs of rows that are written as codes must be finite.
 * The mean of squares of a layer norm is taken of the deviations themselves, which
 * are 0 in a row of equal values, whatever they are. A mean of squares past fp32 is
 * infinite, and its row comes out as zeros (and biases), as the formula in fp32
 * has it; a sum on the way to a mean inside fp32 may be past it.
 * Supported: T >= 0, 1 <= N <= W4A16_NORM_MAX_COLUMNS, for codes N % 16 == 0; a
 * grid of fewer than 2^32 threads (else W4A16_ERR_UNSUPPORTED). y, gate, residual,
 * residual_out, x and xq 16-byte aligned, the vectors 2-byte, sx 4-byte. Outputs
 * overlap no input (residual_out may be residual) and not each other. T == 0
 * launches nothing. At least one of y and residual, and one output, must be
 * given; xq needs sx and excludes x.
 * Returns W4A16_OK, W4A16_ERR_INVALID_ARG, W4A16_ERR_UNSUPPORTED,
 * W4A16_ERR_MISALIGNED or W4A16_ERR_LAUNCH.
 */
int w4a16_norm(const w4a16_norm_args* args, int T, int N, struct ihipStream_t* stream);

#define W4A16_MOE_LAYER_MAX_TOKENS 16

/* The layer's shape and weights, as a program keeps them. Checked by
 * w4a16_moe_layer. */
typedef struct w4a16_moe_layer_args {
  w4a16_route_config route; /* its logits_type does not matter */
  int router_type;          /* W4A16_LOGITS_*: the type of the router's weights */
  int hidden;               /* H */
  int width;                /* I, an expert's inner width */
  int group;
  const void* router;       /* device f32 or bf16 [E][H] */
  const float* route_bias;  /* device f32 [E], or NULL */
  const void* gate_up;      /* device, E packed matrices of N = 2 I, K = H (gates first) */
  const void* gate_up_scales;
  const void* down;         /* device, E packed matrices of N = H, K = I */
  const void* down_scales;
} w4a16_moe_layer_args;

/* Workspace bytes of w4a16_moe_layer (0 for bad arguments); enough for fewer
 * tokens too. 256-byte aligned; its contents before and after a call do not
 * matter. */
size_t w4a16_moe_layer_workspace_bytes(int T, int experts, int top_k, int hidden, int width);

/*
 * A whole mixture-of-experts layer for T tokens:
 *   logits[t][e] = sum_i x[t][i] * router[e][i], held in 64 bits
 *   ids, weights: the choice that w4a16_moe_route defines, from these logits;
 *     a token whose `live` is 0 is routed nowhere (ids -1, weights 0)
 *   h[t][j] = silu(x[t] . gate half) * (x[t] . up half) of expert ids[t][j],
 *     held to 16 bits (two bf16); past what bf16 holds the token's row is NaN
 *   out[t] = base[t] + sum_j weights[t][j] * (h[t][j] . down of expert ids[t][j])
 * with fp32 products and sums and one rounding to bf16 at the end. A result
 * does not depend on timing: the same call gives the same bits.
 *   x    : device bf16 [T][H]; finite in live rows (rows of padding tokens may
 *          hold anything)
 *   live : device int32 [T], or NULL: every token is
 *   base : device bf16 [T][H], or NULL for 0
 *   out  : device bf16 [T][H]; may be base, otherwise overlaps no input
 *   ids  : device int32 [T][top_k]; weights : device f32 [T][top_k]
 *   workspace : w4a16_moe_layer_workspace_bytes(...) bytes
 * Supported: 0 <= T <= W4A16_MOE_LAYER_MAX_TOKENS, group in {32, 64, 128, 256},
 * hidden % group == 0, width % group == 0, one expert's packed matrix and
 * 4 * T * top_k * width bytes below 4 GB (else W4A16_ERR_UNSUPPORTED; more tokens take
 * w4a16_moe_route and the calls behind it). x, router, the packed weights and
 * scales, base and out 16-byte aligned, workspace 256-byte, the rest 4-byte.
 * T == 0 launches nothing. Three or four launches on `stream`, which hand ids and
 * weights from one to the next.
 * Returns W4A16_OK, W4A16_ERR_INVALID_ARG (null pointer, bad field, workspace
 * too small), W4A16_ERR_UNSUPPORTED, W4A16_ERR_MISALIGNED or W4A16_ERR_LAUNCH.
 */
int w4a16_moe_layer(const w4a16_moe_layer_args* layer, const void* x, const int32_t* live,
                    const void* base, void* out, int32_t* ids, float* weights, int T,
                    void* workspace, size_t workspace_bytes, struct ihipStream_t* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_LAYER_H */

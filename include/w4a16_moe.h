/*
 * w4a16_moe.h -- C ABI of the quantized mixture-of-experts operators of the
 * W4A16 library (libw4a16.so, MI355X / gfx950), beside w4a16.h.
 *
 * A mixture-of-experts layer holds its experts' weights in 4 bits and gives
 * each token to top_k of them; the layers that every token passes through
 * (attention projections, a shared expert) are often kept at 8 bits. One such
 * layer, for T tokens:
 *
 *     w4a16_moe_route     router scores -> experts and weights of every token,
 *                         and the list of rows of every expert
 *     w4a16_gemm_experts  gate and up product of every expert over its rows,
 *                         SwiGLU in the epilogue
 *     w4a16_gemm_experts  down product
 *     w8a8_gemm           the shared expert's 8-bit products (codes from
 *                         w4a8_quantize)
 *     w4a16_moe_combine   weighted sum of each token's expert rows, plus the
 *                         shared expert's row
 *
 * A slot is one of the T * top_k places a token is sent to: slot t * top_k + j
 * is the j-th choice of token t.
 *
 * Ownership, threading, streams and errors are those of w4a16.h: the caller
 * owns every buffer, calls are asynchronous on `stream`, the library allocates
 * nothing and keeps no state, every check that can be made without reading
 * device memory is made before any launch, and a failed call launches nothing.
 * Every call can be captured into a HIP graph. Calls that can overlap must not
 * share outputs or a workspace. Device pointers belong to the current device.
 */
#ifndef W4A16_MOE_H
#define W4A16_MOE_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define W4A16_ROUTE_MAX_EXPERTS 1024
#define W4A16_ROUTE_MAX_TOP_K 32
#define W4A16_ROUTE_MAX_GROUPS 64

typedef enum {
  W4A16_ROUTE_SOFTMAX = 0, /* score = softmax of the token's logits */
  W4A16_ROUTE_SIGMOID = 1  /* score = 1 / (1 + exp(-logit)) */
} w4a16_route_scoring;

typedef enum { W4A16_LOGITS_F32 = 0, W4A16_LOGITS_BF16 = 1 } w4a16_logits_type;

/* How a router chooses. Fields are checked by w4a16_moe_route. */
typedef struct w4a16_route_config {
  int experts;     /* E, 1 .. W4A16_ROUTE_MAX_EXPERTS */
  int top_k;       /* 1 .. min(E, W4A16_ROUTE_MAX_TOP_K) */
  int scoring;     /* W4A16_ROUTE_* */
  int logits_type; /* W4A16_LOGITS_* */
  int groups;      /* groups of E / groups consecutive experts, 1 .. W4A16_ROUTE_MAX_GROUPS,
                      dividing E */
  int groups_kept; /* groups a token may choose from, 1 .. groups */
  int group_top;   /* choice values summed into a group's value: 1 or 2 */
  int renormalize; /* nonzero: a token's weights are divided by their sum */
  float scale;     /* factor on every weight, finite */
} w4a16_route_config;

/* Workspace bytes of w4a16_moe_route for T tokens and E experts (0 for bad
 * arguments, and for the few tokens that need none): enough for fewer tokens or
 * experts too. 16-byte aligned; its contents before and after a call do not
 * matter. */
size_t w4a16_moe_route_workspace_bytes(int T, int experts);

/*
 * Routing. Per token: score[e] from the logits as `scoring` says; choice value
 * v[e] = score[e] + bias[e] (bias NULL: 0). With groups > 1, a group's value
 * is the sum of its group_top largest v (fewer where fewer are there), and
 * only the groups_kept groups of largest value are chosen from. The top_k
 * largest v are the token's experts, in descending order; equal values go to
 * the lowest index, for groups too. With bias NULL and groups = 1 the logits
 * themselves are compared, which scores grow with: logits whose scores are
 * equal in 64 bits (sigmoids of 37 and more are 1; a softmax's scores 746 below
 * the largest are 0) are still told apart there, and are equal values with a
 * bias, be it of zeros, or groups. The weight of a choice is its score
 * (without bias), divided by the sum of the token's chosen scores if
 * `renormalize` is set, times scale. Scores, choice values and sums are held
 * in 64 bits, so that which expert is chosen does not depend on rounding.
 *
 * An expert whose logit is -inf or NaN is never chosen and has score 0; +inf
 * counts as the largest finite value. bias must be finite. A token with fewer
 * than top_k experts left gets id -1 and weight 0 in the remaining places; a
 * padding token is routed nowhere by logits of -inf. A sum of chosen scores of
 * 0 gives weights 0.
 *
 *   logits  : device f32 or bf16 [T][E], contiguous
 *   bias    : device f32 [E], or NULL
 *   ids     : device int32 [T][top_k]
 *   weights : device f32 [T][top_k]
 *   offsets : device int32 [E + 1]; expert e's slots are
 *             rows[offsets[e] .. offsets[e + 1])
 *   rows    : device int32 [T * top_k]; slots ordered by expert, ascending
 *             within an expert; -1 from offsets[E] on
 *   workspace : w4a16_moe_route_workspace_bytes(T, E) bytes (may be NULL if 0)
 * Every pointer 16-byte aligned (ids, weights, offsets, rows, bias: 4-byte).
 * T == 0 writes offsets (all 0) and nothing else. T * top_k <= 2^26.
 * Returns W4A16_OK, W4A16_ERR_INVALID_ARG (bad field, null pointer, negative
 * size, workspace too small), W4A16_ERR_UNSUPPORTED (too many slots),
 * W4A16_ERR_MISALIGNED or W4A16_ERR_LAUNCH.
 */
int w4a16_moe_route(const void* logits, const float* bias, const w4a16_route_config* config,
                    int T, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                    void* workspace, size_t workspace_bytes, struct ihipStream_t* stream);

typedef enum {
  W4A16_ACT_NONE = 0,
  W4A16_ACT_SWIGLU = 1 /* columns 0 .. N/2-1 are gates, N/2 .. N-1 are ups */
} w4a16_activation;

/*
 * The experts' W4A16 products over the rows routed to them, in one launch: for
 * expert e and every slot s in rows[offsets[e] .. offsets[e + 1]),
 *
 *     p[n] = sum_k x[s / x_div][k] * q_e[n][k] * s_e[n][k / group]
 *     W4A16_ACT_NONE:    y[s][n] = p[n]                              (n < N)
 *     W4A16_ACT_SWIGLU:  y[s][n] = p[n] / (1 + exp(-p[n])) * p[N/2 + n]  (n < N/2)
 *
 * with fp32 accumulation and activation and one rounding to bf16.
 *   x       : device bf16 [ceil(slots / x_div)][K]; x_div = top_k reads the
 *             token's row for each of its slots, x_div = 1 the slot's own row
 *   qweight : device, experts' packed weights one after another, each
 *             w4a16_qweight_bytes(N, K) bytes as w4a16_pack writes them
 *   scales  : the same, each w4a16_scales_bytes(N, K, group)
 *   y       : device bf16 [slots][N] (SWIGLU: [slots][N / 2])
 *   rows, offsets : as w4a16_moe_route writes them, for `slots` = T * top_k
 * Rows of y whose slot is in no list are left as they are. Entries of the
 * lists outside 0 .. slots - 1 (and offsets outside 0 .. slots) are ignored;
 * where a slot is listed twice, each value of its row is an unspecified one of
 * its results. Offsets that do not ascend list slots several times: a row of y
 * may then also be left as it is.
 * Supported: 0 <= slots <= 2^30, 1 <= experts <= W4A16_ROUTE_MAX_EXPERTS,
 * x_div >= 1, N >= 1, group in {32, 64, 128, 256}, K % group == 0; SWIGLU needs
 * N % 32 == 0; x and one expert's packed weights below 4 GB each, and a grid
 * of fewer than 2^32 threads (else W4A16_ERR_UNSUPPORTED). x, qweight, scales, y
 * 16-byte aligned, the lists 4-byte. slots == 0 launches nothing. y must not overlap any input.
 */
int w4a16_gemm_experts(const void* x, const void* qweight, const void* scales, void* y,
                       const int32_t* rows, const int32_t* offsets, int slots, int experts,
                       int x_div, int N, int K, int group, int act, struct ihipStream_t* stream);

/*
 * out[t][n] = base[t][n] + sum_j weights[t][j] * y[t * top_k + j][n], summed in
 * fp32 in ascending j (base first), rounded once to bf16. Places with a
 * negative id are left out (their rows of y are not read).
 *   y : device bf16 [T * top_k][N]; ids, weights : device int32 / f32 [T][top_k]
 *   base : device bf16 [T][N], or NULL for 0; out : device bf16 [T][N], may be
 *   base itself, otherwise overlaps no input. y, base, out 16-byte aligned.
 * Supported: T >= 0, 1 <= N <= 2^31 - 8, 1 <= top_k <= W4A16_ROUTE_MAX_TOP_K,
 * T * top_k <= 2^30. T == 0 launches nothing.
 */
int w4a16_moe_combine(const void* y, const int32_t* ids, const float* weights, const void* base,
                      void* out, int T, int top_k, int N, struct ihipStream_t* stream);

/*
 * W8A8: 8-bit integer weights with one fp32 scale per output column, int8
 * activations with one fp32 scale per row:
 *
 *     y[m][n] = sx[m] * sw[n] * sum_k xq[m][k] * q[n][k]
 *
 * the sum exact in int32, the scaling in fp32, y rounded to bf16 (nearest
 * even). sx[m] * sw[n] is formed first: where that product is not a normal fp32
 * number (below 2^-126, or past the largest), y has its loss of digits or its
 * infinity.
 *
 * Packed weights: columns in blocks of 16 (the last padded with zero codes), k
 * in steps of 64 (the last padded with zero codes); int8
 * [ceil(N/16)][ceil(K/64)][64][16]: entry (b, t, l) holds the 16 codes of
 * column 16 b + l % 16 and k = 64 t + 16 (l / 16) .. + 15, byte j holding the
 * code of offset o[j], o as in w4a8_quantize. Such a 1 KB tile is one
 * wavefront's operand of one 64-deep int8 MFMA, and w4a8_quantize's codes are
 * its other operand as they lie.
 */
size_t w8a8_qweight_bytes(int N, int K); /* 0 for negative sizes or K % 16 != 0 */

/* Host-side packing of q (host int8 [N][K], any int8 value) into qweight_out
 * (w8a8_qweight_bytes(N, K) bytes, host). Returns W4A16_OK or
 * W4A16_ERR_INVALID_ARG (bad shape; null pointer with a non-empty shape). */
int w8a8_pack(const int8_t* q, int8_t* qweight_out, int N, int K);

/*
 *   xq : device int8 [M][K], sx : device f32 [M], as w4a8_quantize writes them
 *   qweight : device copy of what w8a8_pack wrote; sw : device f32 [N]
 *   y : device bf16 [M][N], overlapping no input
 * Supported: M >= 0, N >= 1, 16 <= K <= 131072 (so that no int32 sum can
 * overflow), K % 16 == 0, packed weights below 4 GB, a grid of fewer than 2^32
 * threads; other shapes return W4A16_ERR_UNSUPPORTED. Every pointer 16-byte
 * aligned (sw and sx: 4-byte).
 * M == 0 launches nothing. Needs no workspace.
 */
int w8a8_gemm(const void* xq, const float* sx, const void* qweight, const float* sw, void* y,
              int M, int N, int K, struct ihipStream_t* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_MOE_H */

/*
 * moe_block.h - C ABI of the operators of a Mixture-of-Experts transformer block around
 * the routed-expert activation, for AMD Instinct MI355X (gfx950).
 *
 *   block_layer_norm_fwd/_bwd  layer norm of a row, and its gradients
 *   block_linear_act           x W^T with bias, activation and residual in its epilogue
 *   block_moe_route            router product, top-k choice and softmax weights
 *   block_moe_experts          the expert products, activation and combine for a few tokens
 *   block_moe_layer            block_moe_route and block_moe_experts in one call
 *   block_moe_gate_fwd/_bwd    scores, choice of experts and weights from given logits, and their gradient
 *   block_moe_route_gated      the router's product with the gate behind it
 *   block_fp4_*                weights to 4 bits with group scales and back
 *   block_linear_act_fp4       block_linear_act with such weights
 *   block_moe_experts_fp4      block_moe_experts with such weights
 *
 * Conventions shared by every call:
 *   - Pointers are caller-owned DEVICE memory on the calling thread's current HIP device,
 *     contiguous, row-major. 16-bit element types are passed as their bit patterns.
 *     Tensor pointers must be 16-byte aligned, int32 / fp32 vectors 4-byte aligned.
 *   - Work is enqueued on `stream` (0 = the null stream); no host synchronisation, no
 *     allocation, no host read of device data, and no memset nodes: calls can be captured
 *     into a HIP graph and replayed.
 *   - Arguments are checked on the host before anything is launched; on error nothing is
 *     written. An output that overlaps an input, another output or the workspace is an error.
 *   - A call that takes a workspace needs at least the bytes its _workspace function
 *     returns, 16-byte aligned. Its contents need no initialisation and mean nothing after
 *     the call's work has run. Two calls (or two captured graphs) whose work may run at the
 *     same time need a workspace each.
 *   - Sums are formed in a fixed order: the same call gives the same bits every time.
 *   - The library keeps no pointer after a call returns; calls are thread-safe.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_BLOCK_ABI_VERSION 1

#ifdef __cplusplus
#define BLOCK_ENUM_BASE : int
#else
#define BLOCK_ENUM_BASE
#endif

typedef enum block_dtype BLOCK_ENUM_BASE { BLOCK_BF16 = 0, BLOCK_FP16 = 1, BLOCK_FP32 = 2 } block_dtype_t;

typedef enum block_status BLOCK_ENUM_BASE {
    BLOCK_OK = 0,
    BLOCK_ERR_INVALID_ARG = 1, /* NULL required pointer, size out of range, unknown dtype or
                                  activation, bad eps / limit / top_k, overlap, short workspace */
    BLOCK_ERR_ALIGNMENT = 2,   /* misaligned pointer, or a width that must be a multiple of 8 */
    BLOCK_ERR_HIP = 3          /* launch failed; see moe_block_last_hip_error */
} block_status_t;

typedef enum block_act BLOCK_ENUM_BASE {
    BLOCK_ACT_NONE = 0,
    BLOCK_ACT_SILU = 1,          /* z / (1 + e^-z) */
    BLOCK_ACT_GELU_TANH = 2,     /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    BLOCK_ACT_SQUARED_RELU = 3,  /* max(z, 0)^2 */
    BLOCK_ACT_SWIGLU = 4         /* experts only: silu(min(gate, L)) * clamp(up, -L, L) */
} block_act_t;

typedef enum block_scores BLOCK_ENUM_BASE { BLOCK_SCORES_SOFTMAX = 0, BLOCK_SCORES_SIGMOID = 1 } block_scores_t;

/*
 * Layer norm of each row, statistics and arithmetic in fp32, one rounding per output:
 *     mean = (1/C) sum_j x_j     rstd = 1 / sqrt((1/C) sum_j (x_j - mean)^2 + eps)
 *     y_j  = (x_j - mean) rstd weight_j + bias_j
 * The variance is summed about the mean, and the mean corrected by the mean deviation from it, so
 * an offset common to a row costs digits only in mean's own rounding (a constant row is its
 * bias) until the offset nears 10^6 deviations.
 *   x, y: [rows, cols] of dtype; weight, bias: [cols] of weight_dtype (dtype or
 *   BLOCK_FP32), each may be NULL (1 and 0); mean, rstd: fp32 [rows], both or neither NULL.
 *   rows >= 0, 1 <= cols <= 2^20, any width; rows * cols <= 2^48; eps >= 0 and finite.
 */
block_status_t block_layer_norm_fwd(const void *x, const void *weight, const void *bias, void *y,
                                    float *mean, float *rstd, int64_t rows, int64_t cols, float eps,
                                    block_dtype_t dtype, block_dtype_t weight_dtype, hipStream_t stream);

/*
 * Gradients of the layer norm, with n_j = (x_j - mean) rstd and d_j = grad_y_j weight_j:
 *     grad_x_j      = rstd (d_j - (1/C) sum_i d_i - n_j (1/C) sum_i d_i n_i)
 *     grad_weight_j = sum over rows of grad_y_j n_j     grad_bias_j = sum over rows of grad_y_j
 *   mean, rstd: as the forward wrote them. grad_x of dtype, grad_weight and grad_bias of
 *   weight_dtype, each may be NULL (not wanted). weight may be NULL (1). With rows == 0 the
 *   weight's gradients are written as zeros.
 *   workspace: needed when grad_weight or grad_bias is wanted and rows > 0, else may be NULL.
 */
int64_t block_layer_norm_bwd_workspace(int64_t rows, int64_t cols);
block_status_t block_layer_norm_bwd(const void *grad_y, const void *x, const void *weight,
                                    const float *mean, const float *rstd, void *grad_x,
                                    void *grad_weight, void *grad_bias, int64_t rows, int64_t cols,
                                    block_dtype_t dtype, block_dtype_t weight_dtype, void *workspace,
                                    int64_t workspace_bytes, hipStream_t stream);

/*
 * y = act(x W^T + bias) + residual, accumulated and finished in fp32, one rounding.
 *   x: [m, k], weight: [n, k], bias: [n] or NULL, residual: [m, n] or NULL, y: [m, n], all of
 *   dtype BLOCK_BF16 or BLOCK_FP16. m >= 0; n, k >= 8 and multiples of 8, up to 2^20;
 *   m <= 2^24, and each of n * k, m * k and m * n up to 2^36. act: any but BLOCK_ACT_SWIGLU.
 *   workspace: partial products of a split sum; may be NULL where _workspace returns 0.
 */
int64_t block_linear_act_workspace(int64_t m, int64_t n, int64_t k);
block_status_t block_linear_act(const void *x, const void *weight, const void *bias,
                                const void *residual, void *y, int64_t m, int64_t n, int64_t k,
                                block_act_t act, block_dtype_t dtype, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream);

/*
 * Router: logits = x router_weight^T in fp64 (so the choice between two experts is the one
 * exact arithmetic makes, unless their logits differ by less than hidden 2^-53 of the sum of
 * their terms' magnitudes), then per token the top_k largest in descending order, equal logits
 * in increasing expert index, NaN before any number, and their softmax weights, in fp64 too and
 * rounded once to fp32:
 *     probs = e^(l_i - l_max) / sum over all experts      (renormalize == 0)
 *     probs = e^(l_i - l_max) / sum over the chosen ones  (renormalize != 0)
 *   x: bf16 [tokens, hidden]; router_weight: [experts, hidden], bf16 or fp32 (router_dtype);
 *   ids: int32 [tokens, top_k]; probs: fp32 [tokens, top_k].
 *   valid_tokens: device int32 scalar or NULL (= tokens), clamped to 0 .. tokens; rows of ids
 *   and probs at or past it are neither read nor written.
 *   0 <= tokens <= 2^19; hidden a multiple of 8, 8 .. 2^20; 1 <= top_k <= min(experts, 64);
 *   1 <= experts <= 1024; tokens * experts <= 2^25.
 */
int64_t block_moe_route_workspace(int64_t tokens, int64_t hidden, int experts);
block_status_t block_moe_route(const uint16_t *x, const void *router_weight, block_dtype_t router_dtype,
                               int32_t *ids, float *probs, int64_t tokens, int64_t hidden, int experts,
                               int top_k, int renormalize, const int32_t *valid_tokens, void *workspace,
                               int64_t workspace_bytes, hipStream_t stream);

/*
 * The expert products of a few tokens. For token t, slot j with e = ids[t, j] in 0 ..
 * experts-1 (any other id contributes nothing; the same id twice contributes twice):
 *     z = x[t] w_up[e]^T                                      fp32
 *     h = act(z) * probs[t, j]                                fp32 (three bf16 terms, which keep its 24 bits)
 *     y[t] = residual[t] + sum over j of h w_down[e]^T        fp32, one rounding
 * BLOCK_ACT_SWIGLU: w_up is [experts, 2 inter, hidden], gate rows first, and act(z) =
 * silu(min(gate, limit)) * clamp(up, -limit, limit); limit > 0, +inf for none; NaN propagates.
 * BLOCK_ACT_SQUARED_RELU: w_up is [experts, inter, hidden]; limit is not used.
 *   x: bf16 [tokens, hidden]; w_down: bf16 [experts, hidden, inter]; residual: bf16 [tokens,
 *   hidden] or NULL; y: [tokens, hidden] of BLOCK_BF16 or BLOCK_FP32 (y_dtype).
 *   valid_tokens: as for block_moe_route; rows of y at or past it are left as they were.
 *   hidden and inter multiples of 8, 8 .. 2^16; tokens * top_k <= 1024; 1 <= experts <= 1024.
 */
int64_t block_moe_experts_workspace(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k);
block_status_t block_moe_experts(const uint16_t *x, const uint16_t *w_up, const uint16_t *w_down,
                                 const int32_t *ids, const float *probs, const uint16_t *residual,
                                 void *y, block_dtype_t y_dtype, int64_t tokens, int64_t hidden,
                                 int64_t inter, int experts, int top_k, block_act_t act, float limit,
                                 const int32_t *valid_tokens, void *workspace,
                                 int64_t workspace_bytes, hipStream_t stream);

/* block_moe_route, then block_moe_experts on its ids and probs (which are outputs). */
int64_t block_moe_layer_workspace(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k);
block_status_t block_moe_layer(const uint16_t *x, const void *router_weight, block_dtype_t router_dtype,
                               const uint16_t *w_up, const uint16_t *w_down, const uint16_t *residual,
                               void *y, block_dtype_t y_dtype, int32_t *ids, float *probs,
                               int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k,
                               int renormalize, block_act_t act, float limit,
                               const int32_t *valid_tokens, void *workspace,
                               int64_t workspace_bytes, hipStream_t stream);

/*
 * Gate: which experts a token goes to and with what weights, from its logits l:
 *     s_i = 1 / (1 + e^-l_i)  (BLOCK_SCORES_SIGMOID)  or  e^(l_i - l_max) / sum_m e^(l_m - l_max)  (_SOFTMAX)
 *     c_i = s_i + bias_i                                    what experts are ranked by
 * The experts lie in `groups` groups of experts / groups neighbours. A group's worth is the sum of
 * its group_top (1 or 2) largest c; the top_groups groups of largest worth are kept, and of their
 * experts the top_k of largest c are chosen, in descending order. Weights carry no bias:
 *     probs_j = scale s_j   or, with renormalize,   scale s_j / sum over the chosen s
 * Scores, ranks and sums are formed in fp64, each weight is rounded once to fp32. Equal ranks go in
 * increasing index, NaN before any number. Without a bias experts are ranked by their logits, and groups
 * by the largest where group_top is 1: that is the scores' order, kept where the scores themselves
 * run out of digits (the softmax's are 0 from 745 below the largest logit on, the sigmoid's 1 from 37
 * on). In a sum with a bias or of two such scores count as the equal numbers that they are. An expert whose logit is -inf is masked: its score is 0
 * and its rank -inf whatever its bias, so that it is chosen (with weight 0) only where too few
 * others are left; where the chosen scores are all 0, so are the weights. (Renormalised softmax
 * weights are the softmax of the chosen logits, also far below the row's largest; so are those of
 * sigmoid scores down to the least one that is not 0, which near it are e^l.)
 *   logits: [tokens, experts] of logits_dtype, any of block_dtype_t; bias: fp32 [experts] or NULL;
 *   ids: int32 [tokens, top_k]; probs: fp32 [tokens, top_k].
 *   valid_tokens: device int32 scalar or NULL (= tokens), clamped to 0 .. tokens; rows of ids and
 *   probs at or past it are left as they were.
 *   0 <= tokens <= 2^24; 1 <= experts <= 1024; 1 <= groups <= 64, a divisor of experts; 1 <=
 *   top_groups <= groups; group_top <= experts / groups (where groups > 1); 1 <= top_k <= 64 and
 *   <= top_groups (experts / groups); scale finite.
 */
block_status_t block_moe_gate_fwd(const void *logits, block_dtype_t logits_dtype, const float *bias, int32_t *ids,
                                  float *probs, int64_t tokens, int experts, int top_k, block_scores_t scores,
                                  int groups, int top_groups, int group_top, int renormalize, float scale,
                                  const int32_t *valid_tokens, hipStream_t stream);

/*
 * Gradient of the gate's weights: grad_logits from grad_probs, with the choice held fixed (it has
 * no gradient; neither has the bias). s and sums as in the forward pass, in fp64, one rounding.
 * With g_j = scale grad_probs_j and p_j = s_j / sum over the chosen s:
 *     d_j = g_j, or with renormalize (g_j - sum_m g_m p_m) / sum over the chosen s
 *     grad_logits_i = s_i (1 - s_i) d_i                 (sigmoid; d_i = 0 where i was not chosen)
 *     grad_logits_i = s_i (d_i - sum_j s_j d_j)         (softmax)
 *   ids: as the forward wrote them; an id outside the experts contributes nothing, the same id
 *   twice contributes twice. grad_logits: [tokens, experts] of logits_dtype, every element of a row
 *   is written (zeros where all chosen scores are 0); rows at or past valid_tokens are left as
 *   they were. Sizes as in the forward pass.
 */
block_status_t block_moe_gate_bwd(const void *logits, block_dtype_t logits_dtype, const int32_t *ids,
                                  const float *grad_probs, void *grad_logits, int64_t tokens, int experts, int top_k,
                                  block_scores_t scores, int renormalize, float scale, const int32_t *valid_tokens,
                                  hipStream_t stream);

/* block_moe_route's logits (fp64) with the gate behind them; sizes within the limits of both,
 * workspace as block_moe_route_workspace tells. */
block_status_t block_moe_route_gated(const uint16_t *x, const void *router_weight, block_dtype_t router_dtype,
                                     const float *bias, int32_t *ids, float *probs, int64_t tokens, int64_t hidden,
                                     int experts, int top_k, block_scores_t scores, int groups, int top_groups,
                                     int group_top, int renormalize, float scale, const int32_t *valid_tokens,
                                     void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Weights in 4 bits with group scales, the open microscaling format: elements of a sign, two bits
 * of exponent and one of mantissa (0, 0.5, 1, 1.5, 2, 3, 4, 6), a power of two 2^(b - 127) for
 * each 32 neighbours of a row, b a byte, 255 for NaN. A weight's value is the element times the
 * power, as a bf16: exact for b <= 252, an infinity where a larger b takes it past bf16's range.
 * The kernels read matrices [n, k] laid out in tiles of 16 rows by 128 k, the rows and k past the
 * end filled with zeros; matrices of one call follow each other:
 *   codes   [matrices][ceil(n / 16)][ceil(k / 128)][64][4] 32-bit words: word j of lane 16 q + r
 *           holds row r's elements k = 32 j + 8 q + 0 .. 7, the first in the lowest four bits
 *   scales  [matrices][ceil(n / 16)][ceil(k / 128)][16][4] bytes: byte j of row r is that of the
 *           elements k = 32 j .. 32 j + 31
 * k a multiple of 32, 32 .. 2^20; 1 <= n <= 2^20; matrices <= 2^16; at most 2^25 tiles in a call.
 * block_fp4_codes_bytes / _scales_bytes: bytes of one matrix (0 for sizes that are refused).
 *
 * quantize: weight [matrices, n, k] of any block_dtype_t. A group's power is the smallest with
 *   max |w| < 7 2^power (at least 2^-127, at most 2^125), and each element the nearest one to w /
 *   2^power, ties to the even code, past 6 to 6: |w - value| <= 2^power / 4 up to 2 2^power, / 2 up to
 *   4 2^power, 2^power up to 7 2^power. A group of zeros has b = 127; one with an infinity or a NaN b = 255.
 *   (The format's specification describes another choice, the largest power up to max |w| / 4, with
 *   elements past 6 cut off at 6. It differs for groups whose largest is from 7 to 8 of those powers: they
 *   get twice the power here, and the largest is off by one of those at most, not by up to two. pack
 *   takes either.)
 * pack: from the row-major form of checkpoints: elements [matrices, n, k / 2], two a byte, the
 *   first in its lower half; exponents [matrices, n, k / 32].
 * dequantize: the bf16 values, [matrices, n, k].
 */
int64_t block_fp4_codes_bytes(int64_t n, int64_t k);
int64_t block_fp4_scales_bytes(int64_t n, int64_t k);
block_status_t block_fp4_quantize(const void *weight, block_dtype_t dtype, uint8_t *codes, uint8_t *scales,
                                  int64_t matrices, int64_t n, int64_t k, hipStream_t stream);
block_status_t block_fp4_pack(const uint8_t *elements, const uint8_t *exponents, uint8_t *codes, uint8_t *scales,
                              int64_t matrices, int64_t n, int64_t k, hipStream_t stream);
block_status_t block_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, uint16_t *weight, int64_t matrices,
                                    int64_t n, int64_t k, hipStream_t stream);

/*
 * block_linear_act with x, bias, residual and y in bf16 and W [n, k] in 4 bits (one matrix).
 * Products are exact, sums and epilogue fp32, one rounding. n a multiple of 8 and k of 32, within
 * block_linear_act's limits. workspace: partial products of a split sum; may be NULL where
 * _workspace returns 0.
 */
int64_t block_linear_act_fp4_workspace(int64_t m, int64_t n, int64_t k);
block_status_t block_linear_act_fp4(const uint16_t *x, const uint8_t *codes, const uint8_t *scales,
                                    const uint16_t *bias, const uint16_t *residual, uint16_t *y, int64_t m, int64_t n,
                                    int64_t k, block_act_t act, void *workspace, int64_t workspace_bytes,
                                    hipStream_t stream);

/*
 * block_moe_experts with the weights in 4 bits: up_* hold experts matrices [2 inter, hidden] (or
 * [inter, hidden] for BLOCK_ACT_SQUARED_RELU), down_* experts matrices [hidden, inter]. hidden and
 * inter multiples of 32, 32 .. 2^16; everything else as there. An infinite weight gives an infinity
 * or a NaN as the product with it does; of the down product that of the activation, which counts as
 * 0 below 2^-133.
 */
int64_t block_moe_experts_fp4_workspace(int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k);
block_status_t block_moe_experts_fp4(const uint16_t *x, const uint8_t *up_codes, const uint8_t *up_scales,
                                     const uint8_t *down_codes, const uint8_t *down_scales, const int32_t *ids,
                                     const float *probs, const uint16_t *residual, void *y, block_dtype_t y_dtype,
                                     int64_t tokens, int64_t hidden, int64_t inter, int experts, int top_k,
                                     block_act_t act, float limit, const int32_t *valid_tokens, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream);

/* Static text for a status code. Never NULL. */
const char *moe_block_status_string(block_status_t status);

/* hipError_t of the last BLOCK_ERR_HIP returned on the calling thread (0 if none). */
int moe_block_last_hip_error(void);

/* MOE_BLOCK_ABI_VERSION of the loaded library. */
int moe_block_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */

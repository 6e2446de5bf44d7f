/*
 * moe_block.h - C ABI of the operators of a Mixture-of-Experts transformer block around
 * the routed-expert activation, for AMD Instinct MI355X (gfx950).
 *
 *   block_layer_norm_fwd/_bwd  layer norm of a row, and its gradients
 *   block_linear_act           x W^T with bias, activation and residual in its epilogue
 *   block_moe_route            router product, top-k choice and softmax weights
 *   block_moe_experts          the expert products, activation and combine for a few tokens
 *   block_moe_layer            block_moe_route and block_moe_experts in one call
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

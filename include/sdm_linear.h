/*
 * sdm_linear.h - C ABI of linear attention with a decay for each head and of group norm with
 * an activation. Conventions, error codes, sdm_exec and sdm_last_error() are sdm.h's;
 * sdm_delta_shape and sdm_rows are sdm_dense.h's.
 */
#ifndef SDM_LINEAR_H
#define SDM_LINEAR_H

#include "sdm_dense.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay: stream p and value head h own a float32 state S of
 * [head_dim, value_dim]; token t does
 *     S = exp(g) S + k v,  out = scale q S
 * (the gated delta rule without its correction). Value head h reads key head
 * h / (value_heads / key_heads). head_dim and value_dim are at most 256, tokens at
 * most 2^30, P * Hv * ceil(K * V / 256) below 2^24 and P * Hv * (T / 64 + 4) * ceil(max(K, V) / 64)
 * below 2^23; SDM_ERR_RANGE past these limits (sdm_linear_attention_step: head_dim at most 256 and
 * value_dim 65536 as in sdm_gated_delta_step, with that function's limits).
 *
 * log_decay: device float32 [Hv], a decay for each head (decay_per_token 0), or [P, T, Hv],
 * one for each token (1). A decay: <= 0, -inf to clear the state. Larger ones are taken too
 * while the sums over up to 256 neighbouring tokens stay within 80 of zero.
 *
 * Over whole sequences and, from a start state, the state after them.
 *   q, k: [P, T, Hk, K]; v: [P, T, Hv, V] (strided rows, element alignment).
 *   state: device float32 [P, Hv, K, V], or NULL for zeros. state_out: the same shape, or
 *     NULL (not wanted); it may be `state` itself (advanced in place), but must not overlap
 *     it, or another input, otherwise.
 *   valid_tokens, out [P, T, Hv, V]: as for sdm_fwd.
 *   kept: NULL, or a device buffer of sdm_linear_attention_kept_bytes(shape) bytes, 256-byte
 *     aligned, in which the call leaves what sdm_linear_attention_bwd then does not compute again.
 *   exec->workspace: sdm_linear_attention_workspace_bytes(shape, SDM_LINEAR_FORWARD) bytes,
 *     256-byte aligned (not used where `kept` is given).
 * Arithmetic: products of the inputs and of float32 quantities (24 bits, to 2^-23) accumulate
 * in float32; the state stays float32; out is rounded once. Bitwise reproducible.
 * An infinity or NaN in a live token's inputs reaches the readings of that token and later ones
 * of its stream, of the heads that read it (from v or a state: its own column alone), and the
 * states after it; what an infinity reaches may be NaN. Padding tokens may hold anything.
 */
enum { SDM_LINEAR_FORWARD = 0, SDM_LINEAR_BACKWARD = 1, SDM_LINEAR_BACKWARD_KEPT = 2 };

/* 0 for shapes they reject. */
size_t sdm_linear_attention_workspace_bytes(const sdm_delta_shape *shape, int32_t what);
size_t sdm_linear_attention_kept_bytes(const sdm_delta_shape *shape);

int sdm_linear_attention_fwd(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                             const float *log_decay, int32_t decay_per_token, const float *state, float *state_out,
                             const int32_t *valid_tokens, void *out, void *kept, const sdm_exec *exec);

/*
 * The same token by token, for single tokens and a few at once: each state is read and
 * written once, whatever T. State, state_out, state_ids, slots: as for sdm_gated_delta_step.
 * out may be v where that is dense, but must not overlap an input or a state otherwise. No
 * workspace.
 */
int sdm_linear_attention_step(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                              const float *log_decay, int32_t decay_per_token, const float *state, float *state_out,
                              const int32_t *state_ids, int64_t slots, const int32_t *valid_tokens, void *out,
                              const sdm_exec *exec);

/*
 * The backward of sdm_linear_attention_fwd: for J = sum(grad_out * out) + sum(grad_state_out *
 * final state) the gradient of every input.
 *   state: the state the forward STARTED from (not read where `kept` is given).
 *   grad_out: device [P, T, Hv, V] in dtype, dense. grad_state_out: device float32
 *     [P, Hv, K, V], or NULL for zeros.
 *   kept: NULL (the forward's states are computed again), or what a forward with the same inputs left.
 *   grads (sdm_delta_grads, beta not used): dense, every element written (padding tokens:
 *     zeros): q, k and v in dtype, each sum over the sharing value heads in float32 and rounded
 *     once; log_decay float32 in log_decay's shape, or NULL; state float32, or NULL. None may
 *     overlap an input, except that grads->state may be grad_state_out.
 *   exec->workspace: sdm_linear_attention_workspace_bytes(shape, SDM_LINEAR_BACKWARD, or
 *     SDM_LINEAR_BACKWARD_KEPT with `kept`) bytes, 256-byte aligned.
 * The log-decays' gradient gathers differences over up to 256 tokens, in 64 bits; it is 0 where the
 * log-decay's exponential is 0 in float32.
 * Tokens are taken 32 at once here, and up to 256 for the log-decays: an infinity or NaN in a live
 * token's inputs or readings' gradient may reach gradients of as many tokens around those that
 * depend on it, never other streams or heads that do not share keys.
 */
int sdm_linear_attention_bwd(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                             const float *log_decay, int32_t decay_per_token, const float *state,
                             const int32_t *valid_tokens, const void *grad_out, const float *grad_state_out,
                             const void *kept, const sdm_delta_grads *grads, const sdm_exec *exec);

/*
 * Group norm with an activation over channels-last x [samples, rows, channels] in dtype, the
 * channels in `groups` groups of neighbours. Per sample and group, over its valid rows:
 *   y = act((x - mean) rstd weight + bias), rstd = 1 / sqrt(var + eps)
 *   act(z) = z, z sigmoid(z) or z Phi(z); float32 arithmetic, y rounded once.
 *   x: rows of `channels` dense elements, x_row elements apart, a sample's x_sample apart (a
 *     slice of a wider array needs no copy; element alignment).
 *   weight, bias: device [channels] in weight_dtype, or NULL (1 and 0). float32 rows take
 *     float32 parameters, bfloat16 rows either type.
 *   valid_rows: device int32 [samples], or NULL: rows at and past it are padding, which may hold
 *     anything; they do not count and give +0. A sample without a valid row has mean 0 and var 0.
 *   y: dense [samples, rows, channels], may be x where that is dense, but must not overlap an input
 *     otherwise; mean, rstd: device float32 [samples, groups], written.
 *   exec->workspace: sdm_group_norm_workspace_bytes(shape, 0) bytes, 256-byte aligned (where that is
 *     0, none).
 * At most 2^31 - 1 samples and rows of 2^20 channels. Samples whose rows a workgroup's registers do
 * not hold are cut into blocks of rows and tiles of channels: of these there are then less than
 * 2^24 in all samples (SDM_ERR_RANGE past that). Bitwise reproducible.
 */
enum { SDM_ACT_NONE = 0, SDM_ACT_SILU = 1, SDM_ACT_GELU = 2 };
typedef struct {
    int64_t samples;
    int64_t rows;
    int32_t channels;
    int32_t groups;
    int32_t dtype;
    int32_t weight_dtype;
    int32_t activation;   /* SDM_ACT_* */
    float eps;
} sdm_group_shape;

/* Workspace bytes of the forward (backward = 0) or the backward (1); 0 where none are needed, and
 * for shapes they reject. */
size_t sdm_group_norm_workspace_bytes(const sdm_group_shape *shape, int32_t backward);

int sdm_group_norm_fwd(const sdm_group_shape *shape, const void *x, int64_t x_sample, int64_t x_row, const void *weight,
                       const void *bias, const int32_t *valid_rows, void *y, float *mean, float *rstd,
                       const sdm_exec *exec);

/*
 * Its backward, from the mean and rstd that the forward wrote. grad_out, grad_x: dense
 * [samples, rows, channels] in dtype (padding rows of grad_x: zeros); grad_weight, grad_bias:
 * [channels] in weight_dtype; each gradient may be NULL (not wanted). grad_x may be grad_out, or x
 * where that is dense; none may overlap an input otherwise. Sums run in float32 in a fixed order.
 */
int sdm_group_norm_bwd(const sdm_group_shape *shape, const void *grad_out, const void *x, int64_t x_sample, int64_t x_row,
                       const void *weight, const void *bias, const int32_t *valid_rows, const float *mean,
                       const float *rstd, void *grad_x, void *grad_weight, void *grad_bias, const sdm_exec *exec);

#ifdef __cplusplus
}
#endif

#endif /* SDM_LINEAR_H */

/*
 * sdm_dense.h - C ABI of the dense operators beside the sparse memory op: the gated delta
 * rule and layer norm. Conventions, error codes, sdm_exec and sdm_last_error() are sdm.h's.
 */
#ifndef SDM_DENSE_H
#define SDM_DENSE_H

#include "sdm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The gated delta rule with a dense state: sdm_fwd's per-token definition with every row of
 * the state addressed by a dense key. Stream p and value head h own a float32 state S of
 * [head_dim, value_dim]; token t does
 *     S' = exp(g) S,  u = beta (v - k S'),  S = S' + k u,  out = scale q S
 * (k, q rows of head_dim, v, u, out rows of value_dim; g the log-decay, -inf to clear the
 * state). Value head h reads key head h / (value_heads / key_heads).
 */
typedef struct {
    int32_t streams;      /* P >= 1 */
    int32_t tokens;       /* T >= 0 */
    int32_t key_heads;    /* Hk >= 1 */
    int32_t value_heads;  /* Hv, a multiple of Hk; P * Hv < 2^24 */
    int32_t head_dim;     /* K in 1..256 */
    int32_t value_dim;    /* V in 1..65536; Hk * K and Hv * V below 2^24 */
    int32_t dtype;        /* sdm_dtype of q, k, v, out and their gradients */
    float scale;
} sdm_delta_shape;
/* Sequences (all but sdm_gated_delta_step) go by chunks of C = 64 tokens (bfloat16 with K <= 128)
 * or 32, with K padded to 64, 128 or 256 and V to a multiple of 8: (min(C, T) - 1) * Hk * K and
 * (min(C, T) - 1) * Hv * V, padded, are at most 2^31 - 2^16; P * Hv * ceil(V / 64) is below 2^23
 * and P * Hv * ceil(T / C) below 2^24. In sdm_gated_delta_step P * Hv * ceil(V / 16) is below 2^26.
 * SDM_ERR_RANGE past these limits. */

/* A device [P, T, heads, width] array whose rows of `width` elements are dense; strides in
 * elements, >= 0 (slices of one fused projection need no copy). Rows need their element's
 * alignment only. */
typedef struct {
    const void *data;
    int64_t stream;
    int64_t token;
    int64_t head;
} sdm_rows;

/*
 * The rule over whole sequences (chunked, on matrix instructions) and, from a start state,
 * the state after them.
 *   q, k: [P, T, Hk, K]; v: [P, T, Hv, V]. beta, log_decay: device float32 [P, T, Hv].
 *   state: device float32 [P, Hv, K, V], or NULL for zeros. state_out: the same shape, or
 *     NULL (the final state is not wanted); it may be `state` itself (the state advances in
 *     place), but must not overlap it otherwise.
 *   valid_tokens, out [P, T, Hv, V]: as for sdm_fwd.
 *   exec->workspace: sdm_gated_delta_workspace_bytes(shape, 0) bytes, 256-byte aligned.
 * Arithmetic: products of the inputs and of float32 quantities (24 bits, to 2^-23) accumulate in
 * float32; the state stays float32 throughout; out is rounded once. Bitwise reproducible.
 * Chunks of tokens are computed as one: an infinity or NaN in a live token's inputs may reach
 * readings of earlier tokens of its chunk (up to 63 before it), never other streams or heads that
 * do not read it, nor, from v or a state, other columns; what an infinity reaches may be NaN.
 * Padding tokens may hold anything.
 */
int sdm_gated_delta_fwd(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                        const float *beta, const float *log_decay, const float *state, float *state_out,
                        const int32_t *valid_tokens, void *out, const sdm_exec *exec);

/*
 * The same token by token, for single tokens and a few at once (generation, proposed
 * tokens): each state is read and written once, whatever T. No workspace.
 *   state, state_out: device float32 [slots, Hv, K, V]; state_out may be `state`, not NULL.
 *   state_ids: device int32 [P], the slot of each stream, all distinct; a stream whose id is
 *     outside [0, slots) is idle: it touches no state and its out rows are +0. NULL: stream
 *     p has slot p (slots >= P).
 * A slot that no stream names keeps its contents in state_out.
 */
int sdm_gated_delta_step(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                         const float *beta, const float *log_decay, const float *state, float *state_out,
                         const int32_t *state_ids, int64_t slots, const int32_t *valid_tokens, void *out,
                         const sdm_exec *exec);

/* Workspace bytes of sdm_gated_delta_fwd (backward = 0) or of the backward and of
 * sdm_gated_delta_fwd_keep (1); 0 for shapes they reject. */
size_t sdm_gated_delta_workspace_bytes(const sdm_delta_shape *shape, int32_t backward);

/*
 * The backward of sdm_gated_delta_fwd: for J = sum(grad_out * out) + sum(grad_state_out *
 * final state) the gradient of every input, at the given inputs (the forward is computed
 * again from them).
 *   grad_out: device [P, T, Hv, V] in dtype, dense. grad_state_out: device float32
 *   [P, Hv, K, V], or NULL for zeros.
 *   grads: device arrays, dense, every element written (padding tokens: zeros): q, k
 *   [P, T, Hk, K] and v [P, T, Hv, V] in dtype, each sum over the sharing value heads and
 *   over tokens in float32 and rounded once; beta, log_decay float32 [P, T, Hv]; state
 *   float32 [P, Hv, K, V], or NULL if not wanted. None may overlap an input, except that
 *   grads->state may be grad_state_out.
 *   exec->workspace: sdm_gated_delta_workspace_bytes(shape, 1) bytes, 256-byte aligned.
 */
typedef struct {
    void *q;
    void *k;
    void *v;
    float *beta;
    float *log_decay;
    float *state;
} sdm_delta_grads;

int sdm_gated_delta_bwd(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                        const float *beta, const float *log_decay, const float *state, const int32_t *valid_tokens,
                        const void *grad_out, const float *grad_state_out, const sdm_delta_grads *grads,
                        const sdm_exec *exec);

/*
 * The pair for training that computes the forward once: sdm_gated_delta_fwd_keep is
 * sdm_gated_delta_fwd on a workspace of the backward's size, in which it leaves what
 * sdm_gated_delta_bwd_kept, with the same inputs and that workspace unchanged, then does not
 * compute again. A token whose |beta| is below 1e-20 counts as one of 1e-20 in both.
 */
int sdm_gated_delta_fwd_keep(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                             const float *beta, const float *log_decay, const float *state, float *state_out,
                             const int32_t *valid_tokens, void *out, const sdm_exec *exec);
int sdm_gated_delta_bwd_kept(const sdm_delta_shape *shape, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v,
                             const float *beta, const float *log_decay, const float *state, const int32_t *valid_tokens,
                             const void *grad_out, const float *grad_state_out, const sdm_delta_grads *grads,
                             const sdm_exec *exec);

/*
 * Layer norm over the last axis of a dense device [rows, cols] array in dtype:
 *   y = (x - mean) rstd weight + bias, mean = sum(x) / cols,
 *   rstd = 1 / sqrt(sum((x - mean)^2) / cols + eps); float32 arithmetic, y rounded once.
 *   weight, bias: device [cols] in weight_dtype, or NULL (1 and 0). float32 rows take float32
 *   parameters, bfloat16 rows either type. mean, rstd: device float32 [rows], written.
 *   rows = 0 does nothing. exec->stream only.
 */
int sdm_layer_norm_fwd(int64_t rows, int32_t cols, const void *x, int32_t dtype, const void *weight, const void *bias,
                       int32_t weight_dtype, float eps, void *y, float *mean, float *rstd, const sdm_exec *exec);

/*
 * Its backward, from the mean and rstd that the forward wrote. grad_x [rows, cols] in dtype,
 * grad_weight and grad_bias [cols] in weight_dtype; each may be NULL (not wanted). The sums
 * over rows run in float32 in a fixed order (bitwise reproducible).
 *   exec->workspace: sdm_layer_norm_bwd_workspace_bytes(rows, cols, dtype) bytes, 256-byte
 *   aligned (not used where grad_weight and grad_bias are both NULL).
 */
size_t sdm_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t cols, int32_t dtype);
int sdm_layer_norm_bwd(int64_t rows, int32_t cols, const void *grad_out, const void *x, int32_t dtype,
                       const void *weight, int32_t weight_dtype, const float *mean, const float *rstd, void *grad_x,
                       void *grad_weight, void *grad_bias, const sdm_exec *exec);

#ifdef __cplusplus
}
#endif

#endif /* SDM_DENSE_H */

// Host entry points of the dense gated delta rule: argument checks, workspace layout, launches.
#include "delta.h"
#include "host.h"

using namespace sdm;

namespace {

// Everything but the pointers.
int check_delta(const sdm_delta_shape *s) {
    if (!s) return fail(SDM_ERR_NULL, "shape must not be NULL");
    if (s->dtype != SDM_F32 && s->dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "dtype must be SDM_F32 or SDM_BF16, got %d", s->dtype);
    if (s->streams < 1 || s->tokens < 0 || s->key_heads < 1 || s->value_heads < 1 || s->head_dim < 1 || s->value_dim < 1)
        return fail(SDM_ERR_SHAPE, "streams, heads and widths must be >= 1 and tokens >= 0, got %d, %d / %d, %d / %d, %d", s->streams,
                    s->key_heads, s->value_heads, s->head_dim, s->value_dim, s->tokens);
    if (s->value_heads % s->key_heads)
        return fail(SDM_ERR_SHAPE, "value_heads (%d) must be a multiple of key_heads (%d)", s->value_heads, s->key_heads);
    if (s->head_dim > 256 || s->value_dim > 65536)
        return fail(SDM_ERR_RANGE, "head_dim must be <= 256 and value_dim <= 65536, got %d and %d", s->head_dim, s->value_dim);
    const int64_t heads = int64_t(s->streams) * s->value_heads;
    if (heads >= 1 << 24) return fail(SDM_ERR_RANGE, "streams * value_heads (%lld) must be below 2^24", (long long)heads);
    if (s->tokens > (1 << 30) || heads * (int64_t(s->tokens) / 16 + 1) >= int64_t(0x7fffffff) ||
        heads * ((s->value_dim + 15) / 16) >= int64_t(0x7fffffff))
        return fail(SDM_ERR_RANGE, "%d tokens of %lld heads are too many", s->tokens, (long long)heads);
    return SDM_OK;
}

bool overlap(const void *a, const void *b, size_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + n && y < x + n;
}

int check_delta_inputs(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                       const float *log_decay, const float *state, const int32_t *valid, const sdm_exec *exec, DeltaArgs *a) {
    const int rc = check_delta(s);
    if (rc) return rc;
    if (!q || !k || !v || !exec) return fail(SDM_ERR_NULL, "q, k, v and exec must not be NULL");
    const size_t es = s->dtype == SDM_BF16 ? 2 : 4;
    const sdm_rows *rows[] = {q, k, v};
    const char *names[] = {"q", "k", "v"};
    for (int i = 0; i < 3; ++i) {
        if (s->tokens > 0 && !rows[i]->data) return fail(SDM_ERR_NULL, "%s must not be NULL", names[i]);
        if (!aligned(rows[i]->data, es)) return fail(SDM_ERR_ALIGN, "%s must be aligned to its element size", names[i]);
        if (rows[i]->stream < 0 || rows[i]->token < 0 || rows[i]->head < 0)
            return fail(SDM_ERR_SHAPE, "%s: strides must be >= 0", names[i]);
    }
    if (s->tokens > 0 && (!beta || !log_decay)) return fail(SDM_ERR_NULL, "beta and log_decay must not be NULL");
    const void *f[] = {beta, log_decay, state, valid};
    for (const void *x : f)
        if (!aligned(x, 4)) return fail(SDM_ERR_ALIGN, "float32 and int32 arrays must be 4-byte aligned");
    a->q = {q->data, q->stream, q->token, q->head};
    a->k = {k->data, k->stream, k->token, k->head};
    a->v = {v->data, v->stream, v->token, v->head};
    a->beta = beta; a->g = log_decay; a->state = state; a->valid = valid;
    a->P = s->streams; a->T = s->tokens; a->Hk = s->key_heads; a->Hv = s->value_heads;
    a->K = s->head_dim; a->V = s->value_dim; a->scale = s->scale;
    return SDM_OK;
}

// Lays the workspace out from `base` (NULL: only its size).
size_t layout(const sdm_delta_shape *s, bool backward, void *base, DeltaWs *ws) {
    const size_t C = size_t(delta_chunk(s->head_dim)), Nt = (size_t(s->tokens) + C - 1) / C;
    const size_t n = size_t(s->streams) * size_t(s->value_heads) * Nt;
    const size_t VP = (size_t(s->value_dim) + 15) / 16 * 16, KP = size_t(delta_kp(s->head_dim));
    char *p = static_cast<char *>(base);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *x = p ? p + at : nullptr;
        at += align256(bytes);
        return x;
    };
    DeltaWs w{};
    w.Nt = int32_t(Nt);
    w.backward = backward;
    w.mats = reinterpret_cast<unsigned char *>(take(n * delta_mats_bytes(s->head_dim, s->dtype == SDM_BF16, backward)));
    if (backward) {
        w.U = reinterpret_cast<float *>(take(n * C * VP * 4));
        w.Y = reinterpret_cast<float *>(take(n * C * VP * 4));
        w.S = reinterpret_cast<float *>(take(n * KP * VP * 4));
        w.dS = reinterpret_cast<float *>(take(n * KP * VP * 4));
    }
    if (ws) *ws = w;
    return at < 256 ? 256 : at;
}

int take_workspace(const sdm_delta_shape *s, bool backward, const sdm_exec *exec, DeltaWs *ws) {
    const size_t need = layout(s, backward, nullptr, nullptr);
    if (!exec->workspace || exec->workspace_bytes < need)
        return fail(SDM_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu bytes needed",
                    exec->workspace ? exec->workspace_bytes : size_t(0), need);
    if (!aligned(exec->workspace, 256)) return fail(SDM_ERR_ALIGN, "workspace must be 256-byte aligned");
    layout(s, backward, exec->workspace, ws);
    return SDM_OK;
}

}  // namespace

extern "C" {

size_t sdm_gated_delta_workspace_bytes(const sdm_delta_shape *s, int32_t backward) {
    if (check_delta(s) != SDM_OK) return 0;
    return layout(s, backward != 0, nullptr, nullptr);
}

int sdm_gated_delta_fwd(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                        const float *log_decay, const float *state, float *state_out, const int32_t *valid, void *out,
                        const sdm_exec *exec) {
    g_err[0] = 0;
    DeltaArgs a{};
    int rc = check_delta_inputs(s, q, k, v, beta, log_decay, state, valid, exec, &a);
    if (rc) return rc;
    if (s->tokens > 0 && !out) return fail(SDM_ERR_NULL, "out must not be NULL");
    if (!aligned(out, s->dtype == SDM_BF16 ? 2 : 4)) return fail(SDM_ERR_ALIGN, "out must be aligned to its element size");
    if (!aligned(state_out, 4)) return fail(SDM_ERR_ALIGN, "state_out must be 4-byte aligned");
    const size_t bytes = size_t(a.P) * a.Hv * a.K * a.V * 4;
    if (state && state_out && state != state_out && overlap(state, state_out, bytes))
        return fail(SDM_ERR_SHAPE, "state_out overlaps state without being it");
    DeltaWs ws{};
    if ((rc = take_workspace(s, false, exec, &ws))) return rc;
    int cus = 0;
    if ((rc = device_cus(&cus))) return rc;
    a.state_out = state_out;
    a.out = out;
    const hipError_t e = launch_delta_fwd(a, ws, s->dtype == SDM_BF16, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "gated delta launch");
}

int sdm_gated_delta_step(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                         const float *log_decay, const float *state, float *state_out, const int32_t *state_ids,
                         int64_t slots, const int32_t *valid, void *out, const sdm_exec *exec) {
    g_err[0] = 0;
    DeltaArgs a{};
    int rc = check_delta_inputs(s, q, k, v, beta, log_decay, state, valid, exec, &a);
    if (rc) return rc;
    if (slots < (state_ids ? 0 : s->streams))
        return fail(SDM_ERR_SHAPE, "%lld states for %d streams", (long long)slots, s->streams);
    if ((slots > 0 && (!state || !state_out)) || (s->tokens > 0 && !out))
        return fail(SDM_ERR_NULL, "state, state_out and out must not be NULL");
    if (!aligned(out, s->dtype == SDM_BF16 ? 2 : 4)) return fail(SDM_ERR_ALIGN, "out must be aligned to its element size");
    if (!aligned(state_out, 4) || !aligned(state_ids, 4)) return fail(SDM_ERR_ALIGN, "state_out and state_ids must be 4-byte aligned");
    const size_t bytes = size_t(slots) * a.Hv * a.K * a.V * 4;
    if (state != state_out && overlap(state, state_out, bytes))
        return fail(SDM_ERR_SHAPE, "state_out overlaps state without being it");
    int cus = 0;
    if ((rc = device_cus(&cus))) return rc;
    a.state_out = state_out;
    a.ids = state_ids;
    a.slots = slots;
    a.out = out;
    const hipError_t e = launch_delta_step(a, s->dtype == SDM_BF16, cus, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "gated delta step launch");
}

int sdm_gated_delta_bwd(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                        const float *log_decay, const float *state, const int32_t *valid, const void *grad_out,
                        const float *grad_state_out, const sdm_delta_grads *grads, const sdm_exec *exec) {
    g_err[0] = 0;
    DeltaArgs a{};
    int rc = check_delta_inputs(s, q, k, v, beta, log_decay, state, valid, exec, &a);
    if (rc) return rc;
    if (!grads) return fail(SDM_ERR_NULL, "grads must not be NULL");
    if (s->tokens > 0 && (!grad_out || !grads->q || !grads->k || !grads->v || !grads->beta || !grads->log_decay))
        return fail(SDM_ERR_NULL, "grad_out and the gradients of q, k, v, beta and log_decay must not be NULL");
    const size_t es = s->dtype == SDM_BF16 ? 2 : 4;
    const void *d[] = {grad_out, grads->q, grads->k, grads->v};
    for (const void *x : d)
        if (!aligned(x, es)) return fail(SDM_ERR_ALIGN, "grad_out and the gradients must be aligned to their element size");
    const void *f[] = {grad_state_out, grads->beta, grads->log_decay, grads->state};
    for (const void *x : f)
        if (!aligned(x, 4)) return fail(SDM_ERR_ALIGN, "float32 gradients must be 4-byte aligned");
    const size_t bytes = size_t(a.P) * a.Hv * a.K * a.V * 4;
    if (grads->state && ((state && overlap(state, grads->state, bytes)) ||
                         (grad_state_out && grad_state_out != grads->state && overlap(grad_state_out, grads->state, bytes))))
        return fail(SDM_ERR_SHAPE, "the state's gradient overlaps an input");
    DeltaWs ws{};
    if ((rc = take_workspace(s, true, exec, &ws))) return rc;
    int cus = 0;
    if ((rc = device_cus(&cus))) return rc;
    const DeltaGrads g{grad_out, grad_state_out, grads->q, grads->k, grads->v, grads->beta, grads->log_decay, grads->state};
    const hipError_t e = launch_delta_bwd(a, ws, g, s->dtype == SDM_BF16, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "gated delta backward launch");
}

}  // extern "C"

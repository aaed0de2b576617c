// Host entry points of the dense gated delta rule: argument checks, workspace layout, launches.
#include "delta.h"
#include "host.h"

using namespace sdm;

namespace {

// Everything but the pointers; `chunks`: for the kernels that take sequences chunk by chunk.
int check_delta(const sdm_delta_shape *s, bool chunks) {
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
    if (int64_t(s->key_heads) * s->head_dim >= kDeltaMaxStride || int64_t(s->value_heads) * s->value_dim >= kDeltaMaxStride)
        return fail(SDM_ERR_RANGE, "a token's rows must be below 2^24 elements: %d x %d and %d x %d", s->key_heads, s->head_dim,
                    s->value_heads, s->value_dim);
    if (s->tokens > (1 << 30) || heads * (int64_t(s->tokens) / 16 + 1) >= int64_t(0x7fffffff) ||
        heads * ((s->value_dim + 15) / 16) >= int64_t(0x7fffffff))
        return fail(SDM_ERR_RANGE, "%d tokens of %lld heads are too many", s->tokens, (long long)heads);
    // A launch of 2^32 threads or more would run a part of its workgroups, without an error.
    const int64_t threads = int64_t(1) << 32;
    if (!chunks) {
        if (heads * ((s->value_dim + 15) / 16) * 64 >= threads)
            return fail(SDM_ERR_RANGE, "%lld heads of value_dim %d are too many for a launch", (long long)heads, s->value_dim);
        return SDM_OK;
    }
    // 32-bit offsets in a chunk, from its first token to the end of its last one's row, of copies with padded widths too
    const int C = delta_chunk(s->head_dim, s->dtype == SDM_BF16), last = (s->tokens < C ? s->tokens : C) - 1;
    const int64_t keys = int64_t(s->key_heads) * delta_kp(s->head_dim), values = int64_t(s->value_heads) * ((s->value_dim + 7) / 8 * 8);
    if (last > 0 && last * (keys > values ? keys : values) > (int64_t(1) << 31) - 65536)
        return fail(SDM_ERR_RANGE, "%d tokens of %lld (keys) or %lld (values) padded elements pass 32-bit offsets", last + 1,
                    (long long)keys, (long long)values);
    if (heads * ((s->value_dim + 63) / 64) * 512 >= threads || heads * ((int64_t(s->tokens) + C - 1) / C) * 256 >= threads)
        return fail(SDM_ERR_RANGE, "%lld heads of value_dim %d and %d tokens are too many for a launch", (long long)heads, s->value_dim,
                    s->tokens);
    return SDM_OK;
}

bool overlap(const void *a, const void *b, size_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + n && y < x + n;
}

int check_delta_inputs(const sdm_delta_shape *s, bool chunks, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                       const float *log_decay, const float *state, const int32_t *valid, const sdm_exec *exec, DeltaArgs *a) {
    const int rc = check_delta(s, chunks);
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
    a->q = {q->data, q->stream, q->token, q->head, s->head_dim};
    a->k = {k->data, k->stream, k->token, k->head, s->head_dim};
    a->v = {v->data, v->stream, v->token, v->head, s->value_dim};
    a->beta = beta; a->g = log_decay; a->state = state; a->valid = valid;
    a->P = s->streams; a->T = s->tokens; a->Hk = s->key_heads; a->Hv = s->value_heads;
    a->K = s->head_dim; a->V = s->value_dim; a->scale = s->scale;
    return SDM_OK;
}

// The workspace, and in it the room for copies of q, k, v and the readings' gradient.
struct Layout {
    DeltaWs ws;
    void *q, *k, *v, *go;
    size_t bytes;
};

// From `base` on (NULL: only the size counts).
Layout layout(const sdm_delta_shape *s, bool backward, void *base) {
    const bool b16 = s->dtype == SDM_BF16;
    const size_t C = size_t(delta_chunk(s->head_dim, b16)), Nt = (size_t(s->tokens) + C - 1) / C;
    const size_t n = size_t(s->streams) * size_t(s->value_heads) * Nt, rows = size_t(s->streams) * size_t(s->tokens);
    const size_t VP = (size_t(s->value_dim) + 15) / 16 * 16, KP = size_t(delta_kp(s->head_dim));
    char *p = static_cast<char *>(base);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *x = p ? p + at : nullptr;
        at += align256(bytes);
        return x;
    };
    auto floats = [&](size_t count) { return reinterpret_cast<float *>(take(count * 4)); };
    Layout l{};
    l.ws.Nt = int32_t(Nt);
    l.ws.backward = backward;
    l.ws.mats = reinterpret_cast<unsigned char *>(take(n * delta_mats_bytes(s->head_dim, b16)));
    if (backward) {
        l.ws.U = floats(n * C * VP);
        l.ws.Y = floats(n * C * VP);
        l.ws.S = floats(n * KP * VP);
        l.ws.dS = floats(n * KP * VP);
    }
    const size_t heads = size_t(s->streams) * size_t(s->value_heads);
    l.ws.segs = backward ? 1 : delta_segments(int64_t(heads), (s->value_dim + 63) / 64, s->head_dim, int(Nt));
    l.ws.seg_chunks = l.ws.segs > 1 ? int32_t((Nt + size_t(l.ws.segs) - 1) / size_t(l.ws.segs)) : int32_t(Nt);
    if (l.ws.segs > 1) {
        l.ws.seg_state = floats(size_t(l.ws.segs) * heads * KP * VP);
        l.ws.seg_map = floats(size_t(l.ws.segs) * heads * KP * KP);
    }
    const size_t keys = rows * size_t(s->key_heads) * KP * (b16 ? 2 : 6);
    const size_t values = rows * size_t(s->value_heads) * ((size_t(s->value_dim) + 7) / 8 * 8) * (b16 ? 2 : 4);
    l.q = take(keys);
    l.k = take(keys);
    l.v = take(values);
    if (backward) l.go = take(values);
    l.bytes = at < 256 ? 256 : at;
    return l;
}

// Checks the workspace and makes the rows regular (go: NULL in the forward; kept: the copies of q, k and v are there).
int take_workspace(const sdm_delta_shape *s, bool backward, DeltaArgs *a, Rows *go, bool kept, const sdm_exec *exec, DeltaWs *ws) {
    const size_t need = layout(s, backward, nullptr).bytes;
    if (!exec->workspace || exec->workspace_bytes < need)
        return fail(SDM_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu bytes needed",
                    exec->workspace ? exec->workspace_bytes : size_t(0), need);
    if (!aligned(exec->workspace, 256)) return fail(SDM_ERR_ALIGN, "workspace must be 256-byte aligned");
    int cus = 0;
    const int rc = device_cus(&cus);
    if (rc) return rc;
    const Layout l = layout(s, backward, exec->workspace);
    *ws = l.ws;
    if (a->T == 0) return SDM_OK;
    const bool b16 = s->dtype == SDM_BF16;
    const hipStream_t st = static_cast<hipStream_t>(exec->stream);
    auto keys = [&](const Rows &r, KeyRows *k, void *to) {
        if (!delta_regular_keys(r, b16)) return launch_delta_copy_keys(r, k, to, a->P, a->T, a->Hk, b16, kept, st);
        *k = {static_cast<const bf16 *>(r.data), 0, r.sp, r.st, r.sh};
        return hipSuccess;
    };
    auto values = [&](Rows *r, void *to, bool there) {
        return delta_regular_values(*r, b16) ? hipSuccess : launch_delta_copy_values(r, to, a->P, a->T, a->Hv, b16, there, st);
    };
    hipError_t e = keys(a->q, &a->qq, l.q);
    if (e == hipSuccess) e = keys(a->k, &a->kk, l.k);
    if (e == hipSuccess) e = values(&a->v, l.v, kept);
    if (e == hipSuccess && go) e = values(go, l.go, false);
    return e == hipSuccess ? SDM_OK : hip_fail(e, "gated delta copy launch");
}

}  // namespace

extern "C" {

size_t sdm_gated_delta_workspace_bytes(const sdm_delta_shape *s, int32_t backward) {
    if (check_delta(s, true) != SDM_OK) return 0;
    return layout(s, backward != 0, nullptr).bytes;
}

static int delta_fwd(bool keep, const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                        const float *log_decay, const float *state, float *state_out, const int32_t *valid, void *out,
                        const sdm_exec *exec) {
    g_err[0] = 0;
    DeltaArgs a{};
    int rc = check_delta_inputs(s, true, q, k, v, beta, log_decay, state, valid, exec, &a);
    if (rc) return rc;
    if (s->tokens > 0 && !out) return fail(SDM_ERR_NULL, "out must not be NULL");
    if (!aligned(out, s->dtype == SDM_BF16 ? 2 : 4)) return fail(SDM_ERR_ALIGN, "out must be aligned to its element size");
    if (!aligned(state_out, 4)) return fail(SDM_ERR_ALIGN, "state_out must be 4-byte aligned");
    const size_t bytes = size_t(a.P) * a.Hv * a.K * a.V * 4;
    if (state && state_out && state != state_out && overlap(state, state_out, bytes))
        return fail(SDM_ERR_SHAPE, "state_out overlaps state without being it");
    DeltaWs ws{};
    if ((rc = take_workspace(s, keep, &a, nullptr, false, exec, &ws))) return rc;
    a.state_out = state_out;
    a.out = out;
    const hipError_t e = launch_delta_fwd(a, ws, s->dtype == SDM_BF16, true, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "gated delta launch");
}

int sdm_gated_delta_fwd(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                        const float *log_decay, const float *state, float *state_out, const int32_t *valid, void *out,
                        const sdm_exec *exec) {
    return delta_fwd(false, s, q, k, v, beta, log_decay, state, state_out, valid, out, exec);
}

int sdm_gated_delta_fwd_keep(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                             const float *log_decay, const float *state, float *state_out, const int32_t *valid, void *out,
                             const sdm_exec *exec) {
    return delta_fwd(true, s, q, k, v, beta, log_decay, state, state_out, valid, out, exec);
}

int sdm_gated_delta_step(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                         const float *log_decay, const float *state, float *state_out, const int32_t *state_ids,
                         int64_t slots, const int32_t *valid, void *out, const sdm_exec *exec) {
    g_err[0] = 0;
    DeltaArgs a{};
    int rc = check_delta_inputs(s, false, q, k, v, beta, log_decay, state, valid, exec, &a);
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

static int delta_bwd(bool kept, const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                        const float *log_decay, const float *state, const int32_t *valid, const void *grad_out,
                        const float *grad_state_out, const sdm_delta_grads *grads, const sdm_exec *exec) {
    g_err[0] = 0;
    DeltaArgs a{};
    int rc = check_delta_inputs(s, true, q, k, v, beta, log_decay, state, valid, exec, &a);
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
    Rows go{grad_out, int64_t(a.T) * a.Hv * a.V, int64_t(a.Hv) * a.V, a.V, a.V};
    if ((rc = take_workspace(s, true, &a, &go, kept, exec, &ws))) return rc;
    const DeltaGrads g{go, grad_state_out, grads->q, grads->k, grads->v, grads->beta, grads->log_decay, grads->state};
    const hipError_t e = launch_delta_bwd(a, ws, g, s->dtype == SDM_BF16, kept, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "gated delta backward launch");
}

int sdm_gated_delta_bwd(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                        const float *log_decay, const float *state, const int32_t *valid, const void *grad_out,
                        const float *grad_state_out, const sdm_delta_grads *grads, const sdm_exec *exec) {
    return delta_bwd(false, s, q, k, v, beta, log_decay, state, valid, grad_out, grad_state_out, grads, exec);
}

int sdm_gated_delta_bwd_kept(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *beta,
                             const float *log_decay, const float *state, const int32_t *valid, const void *grad_out,
                             const float *grad_state_out, const sdm_delta_grads *grads, const sdm_exec *exec) {
    return delta_bwd(true, s, q, k, v, beta, log_decay, state, valid, grad_out, grad_state_out, grads, exec);
}

}  // extern "C"

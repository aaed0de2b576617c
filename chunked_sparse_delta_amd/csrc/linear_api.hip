// Host entry points of linear attention with a decay: argument checks, workspace layout, launches.
#include <mutex>

#include "linear.h"
#include "host.h"

using namespace sdm;

namespace {

// Everything but the pointers; `step`: for the token by token form.
int check_shape(const sdm_delta_shape *s, bool step) {
    if (!s) return fail(SDM_ERR_NULL, "shape must not be NULL");
    if (s->dtype != SDM_F32 && s->dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "dtype must be SDM_F32 or SDM_BF16, got %d", s->dtype);
    if (s->streams < 1 || s->tokens < 0 || s->key_heads < 1 || s->value_heads < 1 || s->head_dim < 1 || s->value_dim < 1)
        return fail(SDM_ERR_SHAPE, "streams, heads and widths must be >= 1 and tokens >= 0, got %d, %d / %d, %d / %d, %d", s->streams,
                    s->key_heads, s->value_heads, s->head_dim, s->value_dim, s->tokens);
    if (s->value_heads % s->key_heads)
        return fail(SDM_ERR_SHAPE, "value_heads (%d) must be a multiple of key_heads (%d)", s->value_heads, s->key_heads);
    const int most = step ? 65536 : 256;
    if (s->head_dim > 256 || s->value_dim > most)
        return fail(SDM_ERR_RANGE, "head_dim must be <= 256 and value_dim <= %d, got %d and %d", most, s->head_dim, s->value_dim);
    if (s->tokens > 1 << 30) return fail(SDM_ERR_RANGE, "%d tokens are too many", s->tokens);
    const int64_t heads = int64_t(s->streams) * s->value_heads, groups = int64_t(1) << 24;   // of 256 threads: 2^32 to a launch
    if (heads >= groups) return fail(SDM_ERR_RANGE, "streams * value_heads (%lld) must be below 2^24", (long long)heads);
    if (step) {
        if (int64_t(s->key_heads) * s->head_dim >= groups || int64_t(s->value_heads) * s->value_dim >= groups)
            return fail(SDM_ERR_RANGE, "a token's rows must be below 2^24 elements: %d x %d and %d x %d", s->key_heads, s->head_dim,
                        s->value_heads, s->value_dim);
        if (heads * ((s->value_dim + 15) / 16) >= groups * 4)
            return fail(SDM_ERR_RANGE, "%lld heads of value_dim %d are too many for a launch", (long long)heads, s->value_dim);
        return SDM_OK;
    }
    const int widest = s->head_dim > s->value_dim ? s->head_dim : s->value_dim;
    if (heads * ((s->head_dim * s->value_dim + 255) / 256) >= groups || heads * (s->tokens / 64 + 4) * ((widest + 63) / 64) >= groups / 2)
        return fail(SDM_ERR_RANGE, "%lld states of %d x %d and %d tokens are too many for a launch", (long long)heads, s->head_dim,
                    s->value_dim, s->tokens);
    return SDM_OK;
}

size_t state_bytes(const sdm_delta_shape *s, int64_t slots) {
    return size_t(slots) * size_t(s->value_heads) * size_t(s->head_dim) * size_t(s->value_dim) * 4;
}

int check_inputs(const sdm_delta_shape *s, bool step, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *log_decay,
                 int32_t per_token, const float *state, const int32_t *valid, const sdm_exec *exec, LinArgs *a) {
    const int rc = check_shape(s, step);
    if (rc) return rc;
    if (!q || !k || !v || !exec) return fail(SDM_ERR_NULL, "q, k, v and exec must not be NULL");
    if (per_token != 0 && per_token != 1) return fail(SDM_ERR_SHAPE, "decay_per_token must be 0 or 1, got %d", per_token);
    const size_t es = s->dtype == SDM_BF16 ? 2 : 4;
    const sdm_rows *rows[] = {q, k, v};
    const char *names[] = {"q", "k", "v"};
    for (int i = 0; i < 3; ++i) {
        if (s->tokens > 0 && !rows[i]->data) return fail(SDM_ERR_NULL, "%s must not be NULL", names[i]);
        if (!aligned(rows[i]->data, es)) return fail(SDM_ERR_ALIGN, "%s must be aligned to its element size", names[i]);
        if (rows[i]->stream < 0 || rows[i]->token < 0 || rows[i]->head < 0)
            return fail(SDM_ERR_SHAPE, "%s: strides must be >= 0", names[i]);
    }
    if (s->tokens > 0 && !log_decay) return fail(SDM_ERR_NULL, "log_decay must not be NULL");
    const void *f[] = {log_decay, state, valid};
    for (const void *x : f)
        if (!aligned(x, 4)) return fail(SDM_ERR_ALIGN, "float32 and int32 arrays must be 4-byte aligned");
    a->q = {q->data, q->stream, q->token, q->head, s->head_dim};
    a->k = {k->data, k->stream, k->token, k->head, s->head_dim};
    a->v = {v->data, v->stream, v->token, v->head, s->value_dim};
    a->gates = {log_decay, per_token ? int64_t(s->tokens) * s->value_heads : 0, per_token ? s->value_heads : 0};
    a->state = state; a->valid = valid;
    a->P = s->streams; a->T = s->tokens; a->Hk = s->key_heads; a->Hv = s->value_heads;
    a->K = s->head_dim; a->V = s->value_dim; a->scale = s->scale;
    return SDM_OK;
}

Extent extent(const sdm_delta_shape *s, const Rows &r, int heads) {
    return {r.data, {{s->streams, r.sp}, {s->tokens, r.st}, {heads, r.sh}}, r.width, s->dtype == SDM_BF16 ? 2 : 4};
}
size_t readings_bytes(const sdm_delta_shape *s) {
    return size_t(s->streams) * size_t(s->tokens) * size_t(s->value_heads) * size_t(s->value_dim) * (s->dtype == SDM_BF16 ? 2 : 4);
}
// Whether the n bytes of a result at p (null: not wanted) meet q, k, v, the log-decays or the counts. over_v: a dense v's own place is
// allowed.
bool meets_inputs(const sdm_delta_shape *s, const LinArgs &a, const void *p, size_t n, bool over_v) {
    if (!p) return false;
    const Extent v = extent(s, a.v, a.Hv);
    const size_t gates = size_t(a.Hv) * (a.gates.st ? size_t(a.P) * size_t(a.T) : 1) * 4;
    return extent(s, a.q, a.Hk).meets(p, n) || extent(s, a.k, a.Hk).meets(p, n) || (!(over_v && p == v.data && v.dense()) && v.meets(p, n)) ||
           (a.gates.g && overlap(p, n, a.gates.g, gates)) || (a.valid && overlap(p, n, a.valid, size_t(a.P) * 4));
}
// The forward's and the step's results: states of `bytes` at a.state (may be null) and a.state_out, readings at a.out.
int check_apart(const sdm_delta_shape *s, const LinArgs &a, size_t bytes, bool over_v) {
    const size_t n = readings_bytes(s);
    if (a.state && a.state_out && a.state != a.state_out && overlap(a.state, bytes, a.state_out, bytes))
        return fail(SDM_ERR_SHAPE, "state_out overlaps state without being it");
    if (meets_inputs(s, a, a.out, n, over_v) || (a.state && overlap(a.out, n, a.state, bytes)) || (a.state_out && overlap(a.out, n, a.state_out, bytes)))
        return fail(SDM_ERR_SHAPE, "out overlaps an input or a state%s", over_v ? " (it may be a dense v)" : "");
    if (meets_inputs(s, a, a.state_out, bytes, false)) return fail(SDM_ERR_SHAPE, "the state overlaps another input");
    return SDM_OK;
}

// The device's setup, and that of the sequences' kernels, which may take more LDS than by default: once a device, by the first call of
// theirs. (As a part of the device's setup it cost the first call of every other entry point 5 ms beside its 34.)
int prepare_once() {
    static std::mutex mu;
    static bool ready[64];      // device_cus refuses devices past these
    int cus = 0, dev = 0;
    const int rc = device_cus(&cus);
    if (rc) return rc;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev]) {
        if ((e = linear_prepare()) != hipSuccess) return hip_fail(e, "hipFuncSetAttribute (linear attention)");
        ready[dev] = true;
    }
    return SDM_OK;
}

// Takes arrays from a buffer in order (from NULL: only the size counts).
struct Taker {
    char *base;
    size_t at = 0;
    template <typename T> T *take(size_t count) {
        T *x = base ? reinterpret_cast<T *>(base + at) : nullptr;
        at += align256(count * sizeof(T));
        return x;
    }
    size_t bytes() const { return at < 256 ? 256 : at; }
};

void take_states(const sdm_delta_shape *s, LinWs *ws, Taker &t) {
    const size_t heads = size_t(s->streams) * size_t(s->value_heads), KV = size_t(s->head_dim) * size_t(s->value_dim);
    ws->S = t.take<float>(heads * (size_t(ws->segs) + 1) * KV);
    ws->decay = t.take<float>(heads * size_t(ws->segs));
}
LinWs segments(const sdm_delta_shape *s) {
    LinWs ws{};
    ws.tokens = lin_seg_tokens(s->dtype == SDM_BF16, s->tokens);
    ws.segs = s->tokens > ws.tokens ? (s->tokens + ws.tokens - 1) / ws.tokens : 1;
    return ws;
}
// what: SDM_LINEAR_*, or -1: `kept`.
size_t layout(const sdm_delta_shape *s, int what, LinWs *ws, void *base) {
    Taker t{static_cast<char *>(base)};
    if (what == -1 || what == SDM_LINEAR_BACKWARD || (what == SDM_LINEAR_FORWARD && ws->segs > 1)) take_states(s, ws, t);
    if (what == SDM_LINEAR_BACKWARD || what == SDM_LINEAR_BACKWARD_KEPT) {
        const size_t heads = size_t(s->streams) * size_t(s->value_heads), segs = size_t(ws->segs);
        const size_t gates = size_t(lin_slices(s->head_dim)) * heads * size_t(s->tokens);
        ws->dS = t.take<float>(heads * segs * size_t(s->head_dim) * size_t(s->value_dim));
        ws->dots = t.take<float>(heads * (segs + 1) * size_t(lin_dot_parts(s->head_dim, s->value_dim)));
        ws->rows = t.take<float>(gates);
        ws->cols = t.take<float>(gates);
        ws->sums = t.take<double>(heads * segs);
        ws->rest = t.take<float>(s->value_heads > s->key_heads ? 2 * lin_rest_floats(s->streams, s->key_heads, s->head_dim, ws->segs, ws->tokens) : 0);
    }
    return t.bytes();
}
int take_workspace(const sdm_delta_shape *s, int what, const sdm_exec *exec, LinWs *ws) {
    const size_t need = layout(s, what, ws, nullptr);
    if (!exec->workspace || exec->workspace_bytes < need)
        return fail(SDM_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu bytes needed",
                    exec->workspace ? exec->workspace_bytes : size_t(0), need);
    if (!aligned(exec->workspace, 256)) return fail(SDM_ERR_ALIGN, "workspace must be 256-byte aligned");
    layout(s, what, ws, exec->workspace);
    return SDM_OK;
}

}  // namespace

extern "C" {

size_t sdm_linear_attention_workspace_bytes(const sdm_delta_shape *s, int32_t what) {
    if (check_shape(s, false) != SDM_OK || what < SDM_LINEAR_FORWARD || what > SDM_LINEAR_BACKWARD_KEPT) return 0;
    LinWs ws = segments(s);
    return layout(s, what, &ws, nullptr);
}

size_t sdm_linear_attention_kept_bytes(const sdm_delta_shape *s) {
    if (check_shape(s, false) != SDM_OK) return 0;
    LinWs ws = segments(s);
    return layout(s, -1, &ws, nullptr);
}

int sdm_linear_attention_fwd(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *log_decay,
                             int32_t per_token, const float *state, float *state_out, const int32_t *valid, void *out, void *kept,
                             const sdm_exec *exec) {
    g_err[0] = 0;
    LinArgs a{};
    int rc = check_inputs(s, false, q, k, v, log_decay, per_token, state, valid, exec, &a);
    if (rc) return rc;
    if (s->tokens > 0 && !out) return fail(SDM_ERR_NULL, "out must not be NULL");
    if (!aligned(out, s->dtype == SDM_BF16 ? 2 : 4)) return fail(SDM_ERR_ALIGN, "out must be aligned to its element size");
    if (!aligned(state_out, 4)) return fail(SDM_ERR_ALIGN, "state_out must be 4-byte aligned");
    if (!aligned(kept, 256)) return fail(SDM_ERR_ALIGN, "kept must be 256-byte aligned");
    a.state_out = state_out;
    a.out = out;
    if ((rc = check_apart(s, a, state_bytes(s, s->streams), false))) return rc;
    LinWs ws = segments(s);
    if (kept) layout(s, -1, &ws, kept);
    else if ((rc = take_workspace(s, SDM_LINEAR_FORWARD, exec, &ws))) return rc;
    if ((rc = prepare_once())) return rc;
    const hipError_t e = launch_linear_fwd(a, ws, s->dtype == SDM_BF16, kept != nullptr, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "linear attention launch");
}

int sdm_linear_attention_step(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *log_decay,
                              int32_t per_token, const float *state, float *state_out, const int32_t *state_ids, int64_t slots,
                              const int32_t *valid, void *out, const sdm_exec *exec) {
    g_err[0] = 0;
    LinArgs a{};
    int rc = check_inputs(s, true, q, k, v, log_decay, per_token, state, valid, exec, &a);
    if (rc) return rc;
    if (slots < (state_ids ? 0 : s->streams))
        return fail(SDM_ERR_SHAPE, "%lld states for %d streams", (long long)slots, s->streams);
    if ((slots > 0 && (!state || !state_out)) || (s->tokens > 0 && !out))
        return fail(SDM_ERR_NULL, "state, state_out and out must not be NULL");
    if (!aligned(out, s->dtype == SDM_BF16 ? 2 : 4)) return fail(SDM_ERR_ALIGN, "out must be aligned to its element size");
    if (!aligned(state_out, 4) || !aligned(state_ids, 4)) return fail(SDM_ERR_ALIGN, "state_out and state_ids must be 4-byte aligned");
    a.state_out = state_out;
    a.out = out;
    const size_t bytes = state_bytes(s, slots);
    if ((rc = check_apart(s, a, bytes, true))) return rc;
    if (state_ids && (overlap(out, readings_bytes(s), state_ids, size_t(a.P) * 4) || overlap(state_out, bytes, state_ids, size_t(a.P) * 4)))
        return fail(SDM_ERR_SHAPE, "out or state_out overlaps state_ids");
    int cus = 0;
    if ((rc = device_cus(&cus))) return rc;
    DeltaArgs d{};
    d.q = a.q; d.k = a.k; d.v = a.v;
    d.g = log_decay; d.g_stream = a.gates.sp; d.g_token = a.gates.st;
    d.state = state; d.state_out = state_out; d.valid = valid; d.ids = state_ids; d.slots = slots; d.out = out;
    d.P = a.P; d.T = a.T; d.Hk = a.Hk; d.Hv = a.Hv; d.K = a.K; d.V = a.V; d.scale = a.scale;
    const hipError_t e = launch_linear_step(d, s->dtype == SDM_BF16, cus, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "linear attention step launch");
}

int sdm_linear_attention_bwd(const sdm_delta_shape *s, const sdm_rows *q, const sdm_rows *k, const sdm_rows *v, const float *log_decay,
                             int32_t per_token, const float *state, const int32_t *valid, const void *grad_out,
                             const float *grad_state_out, const void *kept, const sdm_delta_grads *grads, const sdm_exec *exec) {
    g_err[0] = 0;
    LinArgs a{};
    int rc = check_inputs(s, false, q, k, v, log_decay, per_token, state, valid, exec, &a);
    if (rc) return rc;
    if (!grads) return fail(SDM_ERR_NULL, "grads must not be NULL");
    if (s->tokens > 0 && (!grad_out || !grads->q || !grads->k || !grads->v))
        return fail(SDM_ERR_NULL, "grad_out and the gradients of q, k and v must not be NULL");
    const size_t es = s->dtype == SDM_BF16 ? 2 : 4;
    const void *d[] = {grad_out, grads->q, grads->k, grads->v};
    for (const void *x : d)
        if (!aligned(x, es)) return fail(SDM_ERR_ALIGN, "grad_out and the gradients must be aligned to their element size");
    const void *f[] = {grad_state_out, grads->log_decay, grads->state};
    for (const void *x : f)
        if (!aligned(x, 4)) return fail(SDM_ERR_ALIGN, "float32 gradients must be 4-byte aligned");
    if (!aligned(kept, 256)) return fail(SDM_ERR_ALIGN, "kept must be 256-byte aligned");
    const size_t bytes = state_bytes(s, s->streams), readings = readings_bytes(s), keys = size_t(a.P) * a.T * a.Hk * a.K * es;
    const struct {
        const void *p;
        size_t n;
    } results[] = {{grads->q, keys}, {grads->k, keys}, {grads->v, readings},
                   {grads->log_decay, size_t(a.Hv) * (per_token ? size_t(a.P) * size_t(a.T) : 1) * 4}, {grads->state, bytes}};
    for (const auto &r : results) {
        if (!r.p) continue;
        const bool own = r.p == grads->state && grads->state == grad_state_out;
        if (meets_inputs(s, a, r.p, r.n, false) || (state && overlap(r.p, r.n, state, bytes)) || (grad_out && overlap(r.p, r.n, grad_out, readings)) ||
            (grad_state_out && !own && overlap(r.p, r.n, grad_state_out, bytes)))
            return fail(SDM_ERR_SHAPE, "a gradient overlaps an input (the state's may be grad_state_out)");
    }
    LinWs ws = segments(s);
    if (kept) layout(s, -1, &ws, const_cast<void *>(kept));
    if ((rc = take_workspace(s, kept ? SDM_LINEAR_BACKWARD_KEPT : SDM_LINEAR_BACKWARD, exec, &ws))) return rc;
    if ((rc = prepare_once())) return rc;
    const LinGrads g{{grad_out, int64_t(a.T) * a.Hv * a.V, int64_t(a.Hv) * a.V, a.V, a.V}, grad_state_out,
                     grads->q, grads->k, grads->v, grads->log_decay, grads->state};
    const hipError_t e = launch_linear_bwd(a, ws, g, s->dtype == SDM_BF16, kept != nullptr, static_cast<hipStream_t>(exec->stream));
    return e == hipSuccess ? SDM_OK : hip_fail(e, "linear attention backward launch");
}

}  // extern "C"

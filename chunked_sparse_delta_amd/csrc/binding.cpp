// Linear attention and group norm on torch tensors: checks of the arguments, allocation, and autograd, around the C ABI of
// include/sdm_linear.h. Host code only; in C++ because a call of a few microseconds' work, and a training step of tens, notice what
// the same in Python costs (a backward in Python alone took about 60 us beside its launches).
#include <torch/extension.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/variable.h>

#include "sdm_linear.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// libsdm's functions, handed over by the package, which has loaded it.
struct Api {
    decltype(&sdm_linear_attention_fwd) la_fwd;
    decltype(&sdm_linear_attention_step) la_step;
    decltype(&sdm_linear_attention_bwd) la_bwd;
    decltype(&sdm_linear_attention_workspace_bytes) la_bytes;
    decltype(&sdm_linear_attention_kept_bytes) la_kept;
    decltype(&sdm_group_norm_fwd) gn_fwd;
    decltype(&sdm_group_norm_bwd) gn_bwd;
    decltype(&sdm_group_norm_workspace_bytes) gn_bytes;
    decltype(&sdm_last_error) last_error;
} api;

struct SdmFailure : std::runtime_error {
    int code;
    SdmFailure(int c, const char *msg) : std::runtime_error(msg), code(c) {}
};
void check_rc(int rc) {
    if (rc) throw SdmFailure(rc, api.last_error());
}

template <typename... A> [[noreturn]] void type_error(const A &...a) { throw py::type_error(c10::str(a...)); }
template <typename... A> [[noreturn]] void value_error(const A &...a) { throw py::value_error(c10::str(a...)); }

std::string name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}
int dtype_code(at::ScalarType t) { return t == at::kFloat ? SDM_F32 : t == at::kBFloat16 ? SDM_BF16 : -1; }

const Tensor *given(const OptTensor &t) { return t && t->defined() ? &*t : nullptr; }
template <typename T> T *ptr(const OptTensor &t) { return given(t) ? static_cast<T *>(t->data_ptr()) : nullptr; }

// Calls run on the current device: the tensors have to be there.
int on(const Tensor &t) {
    if (!t.is_cuda()) value_error("expected GPU tensors, got ", t.device());
    const int index = c10::hip::current_device();
    if (t.get_device() != index) value_error("the tensors are on ", t.device(), ", the current device is cuda:", index);
    return index;
}

void need(const Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) {
    if (t.scalar_type() != dtype) type_error(name, ": expected ", name_of(dtype), ", got ", name_of(t.scalar_type()));
    if (t.sizes() != shape) value_error(name, ": expected shape ", shape, ", got ", t.sizes());
    if (t.device() != dev) value_error(name, " is on ", t.device(), ", expected ", dev);
    if (!t.is_contiguous()) value_error(name, " must be contiguous");
}
void need(const OptTensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) {
    if (given(t)) need(*t, name, shape, dtype, dev);
}

int32_t small(int64_t n, const char *what) {
    if (n > INT32_MAX) value_error(what, " (", n, ") is past 2^31 - 1");
    return int32_t(n);
}

Tensor make(at::IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) { return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev)); }
Tensor scratch(size_t bytes, const at::Device &dev) { return make({int64_t(bytes < 256 ? 256 : bytes)}, at::kByte, dev); }

sdm_exec exec_of(int index, const OptTensor &workspace) {
    sdm_exec e{};
    e.stream = c10::hip::getCurrentHIPStream(index).stream();
    if (const Tensor *w = given(workspace)) {
        if (!w->is_cuda() || w->get_device() != index || !w->is_contiguous()) value_error("workspace must be a contiguous tensor on cuda:", index);
        e.workspace = w->data_ptr();
        e.workspace_bytes = w->nbytes();
    }
    return e;
}

// The caller's tensors that a call has written through their pointers: with their versions raised, a backward that saved one of them
// is refused, as after any other write in place. (Inference tensors have no version.)
void wrote(std::initializer_list<const OptTensor *> tensors) {
    for (const OptTensor *t : tensors)
        if (given(*t) && !(*t)->is_inference()) torch::autograd::impl::bump_version(**t);
}

// Python's once_differentiable: a gradient of these gradients is an error, not nothing.
variable_list once(variable_list grads) {
    if (!at::GradMode::is_enabled()) return grads;
    variable_list fake;
    for (const Tensor &g : grads) fake.push_back(g.defined() ? g.detach().requires_grad_(true) : g);
    auto fn = std::make_shared<torch::autograd::DelayedError>("trying to differentiate twice a function that can be differentiated once",
                                                              int(fake.size()));
    return (*fn)(std::move(fake));
}

// ---- linear attention ------------------------------------------------------------------------------------------------

struct Attention {
    sdm_delta_shape shape;
    sdm_rows q, k, v;
    const float *g;
    int32_t per_token;
    int index;
    at::Device dev;
    std::array<int64_t, 4> state;     // [P, Hv, K, V]
};

sdm_rows rows_of(const Tensor &t) { return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)}; }

sdm_rows view(const Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) {
    if (t.scalar_type() != dtype) type_error(name, ": expected ", name_of(dtype), ", got ", name_of(t.scalar_type()));
    if (t.sizes() != shape) value_error(name, ": expected shape ", shape, ", got ", t.sizes());
    if (t.device() != dev) value_error(name, " is on ", t.device(), ", v on ", dev);
    if (t.stride(3) != 1 && shape[3] > 1) value_error(name, ": the last axis must be dense, its stride is ", t.stride(3));
    return rows_of(t);
}

Attention attention(const OptTensor &k_, const OptTensor &v_, const OptTensor &g_, const OptTensor &q_, std::optional<double> scale,
                    const OptTensor &valid) {
    if (!given(k_) || !given(v_) || !given(g_) || !given(q_)) type_error("k, v, log_decay and q must be torch tensors");
    const Tensor &k = *k_, &v = *v_, &g = *g_, &q = *q_;
    const at::ScalarType dtype = v.scalar_type();
    const int code = dtype_code(dtype);
    if (code < 0) type_error("v must be float32 or bfloat16, got ", name_of(dtype));
    if (v.dim() != 4 || k.dim() != 4) value_error("k and v must be [P, T, heads, width], got ", k.sizes(), " and ", v.sizes());
    const int index = on(v);
    const at::Device dev = v.device();
    const int64_t P = v.size(0), T = v.size(1), Hv = v.size(2), V = v.size(3), Hk = k.size(2), K = k.size(3);
    if (Hk < 1 || Hv % Hk) value_error("the value heads (", Hv, ") must be a multiple of the key heads (", Hk, ")");
    const std::array<int64_t, 4> keys{P, T, Hk, K};
    const bool per_token = g.dim() != 1;
    if (per_token) need(g, "log_decay", {P, T, Hv}, at::kFloat, dev);
    else need(g, "log_decay", {Hv}, at::kFloat, dev);
    need(valid, "valid_tokens", {P}, at::kInt, dev);
    return {{small(P, "streams"), small(T, "tokens"), small(Hk, "key heads"), small(Hv, "value heads"), small(K, "head_dim"), small(V, "value_dim"), code,
             float(scale ? *scale : 1.0 / std::sqrt(double(K)))},
            view(q, "q", keys, dtype, dev), view(k, "k", keys, dtype, dev), view(v, "v", v.sizes(), dtype, dev),
            static_cast<const float *>(g.data_ptr()), per_token, index, dev, {P, Hv, K, V}};
}

Tensor dense_out(const OptTensor &out, const Tensor &v) {
    if (!given(out)) return make(v.sizes(), v.scalar_type(), v.device());     // dense whatever v's strides are
    need(*out, "out", v.sizes(), v.scalar_type(), v.device());
    return *out;
}

void check_kept(const Attention &a, const OptTensor &kept) {
    if (!given(kept)) return;
    const size_t least = api.la_kept(&a.shape);
    if (kept->device() != a.dev || !kept->is_contiguous() || kept->nbytes() < least)
        value_error("kept must be a contiguous tensor of ", least, " bytes on ", a.dev);
}

void la_values(const Attention &a, const OptTensor &state, const OptTensor &state_out, const OptTensor &valid, const Tensor &out, const OptTensor &kept,
               const OptTensor &workspace) {
    OptTensor ws = workspace;
    if (!given(ws) && !given(kept)) ws = scratch(api.la_bytes(&a.shape, SDM_LINEAR_FORWARD), a.dev);
    const sdm_exec e = exec_of(a.index, ws);
    check_rc(api.la_fwd(&a.shape, &a.q, &a.k, &a.v, a.g, a.per_token, ptr<float>(state), ptr<float>(state_out), ptr<int32_t>(valid), out.data_ptr(),
                        ptr<void>(kept), &e));
}

Tensor la_fwd(const OptTensor &state, const OptTensor &k, const OptTensor &v, const OptTensor &g, const OptTensor &q, std::optional<double> scale,
              const OptTensor &valid, const OptTensor &state_out, const OptTensor &out_, const OptTensor &workspace, const OptTensor &kept) {
    const Attention a = attention(k, v, g, q, scale, valid);
    need(state, "state", a.state, at::kFloat, a.dev);
    need(state_out, "state_out", a.state, at::kFloat, a.dev);
    check_kept(a, kept);
    const Tensor out = dense_out(out_, *v);
    const OptTensor &final = given(state_out) ? state_out : state;
    la_values(a, state, final, valid, out, kept, workspace);
    wrote({&final, &out_, &kept});
    return out;
}

Tensor la_step(const OptTensor &state, const OptTensor &k, const OptTensor &v, const OptTensor &g, const OptTensor &q, const OptTensor &ids,
               std::optional<double> scale, const OptTensor &valid, const OptTensor &state_out, const OptTensor &out_) {
    const Attention a = attention(k, v, g, q, scale, valid);
    if (!given(state) || state->dim() != 4) value_error("state must be a [slots, Hv, K, V] tensor");
    const std::array<int64_t, 4> pool{state->size(0), a.state[1], a.state[2], a.state[3]};
    need(*state, "state", pool, at::kFloat, a.dev);
    need(state_out, "state_out", pool, at::kFloat, a.dev);
    need(ids, "state_ids", {a.state[0]}, at::kInt, a.dev);
    const Tensor out = dense_out(out_, *v);
    const sdm_exec e = exec_of(a.index, std::nullopt);
    const OptTensor &final = given(state_out) ? state_out : state;
    check_rc(api.la_step(&a.shape, &a.q, &a.k, &a.v, a.g, a.per_token, ptr<float>(state), ptr<float>(final), ptr<int32_t>(ids), pool[0],
                         ptr<int32_t>(valid), out.data_ptr(), &e));
    wrote({&final, &out_});
    return out;
}

struct AttentionGrads {
    Tensor state, k, v, g, q;
};
AttentionGrads la_grads(const Attention &a, const OptTensor &state, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &q, const Tensor &go,
                        const OptTensor &gs, const OptTensor &valid, const OptTensor &kept, const OptTensor &workspace, bool want_state, bool want_g) {
    AttentionGrads r;
    r.k = make(k.sizes(), k.scalar_type(), a.dev);
    r.v = make(v.sizes(), v.scalar_type(), a.dev);
    r.q = make(q.sizes(), q.scalar_type(), a.dev);
    if (want_state) r.state = make(a.state, at::kFloat, a.dev);
    if (want_g) r.g = make(g.sizes(), at::kFloat, a.dev);
    OptTensor ws = workspace;
    if (!given(ws)) ws = scratch(api.la_bytes(&a.shape, given(kept) ? SDM_LINEAR_BACKWARD_KEPT : SDM_LINEAR_BACKWARD), a.dev);
    const sdm_exec e = exec_of(a.index, ws);
    const sdm_delta_grads grads{r.q.data_ptr(), r.k.data_ptr(), r.v.data_ptr(), nullptr, ptr<float>(r.g), ptr<float>(r.state)};
    check_rc(api.la_bwd(&a.shape, &a.q, &a.k, &a.v, a.g, a.per_token, ptr<float>(state), ptr<int32_t>(valid), go.data_ptr(), ptr<float>(gs),
                        ptr<void>(kept), &grads, &e));
    return r;
}

py::dict la_bwd(const OptTensor &state, const OptTensor &k, const OptTensor &v, const OptTensor &g, const OptTensor &q, const Tensor &go,
                const OptTensor &gs, std::optional<double> scale, const OptTensor &valid, const OptTensor &workspace, const OptTensor &kept,
                const std::vector<std::string> &names) {
    const Attention a = attention(k, v, g, q, scale, valid);
    need(go, "grad_out", v->sizes(), v->scalar_type(), a.dev);
    need(state, "state", a.state, at::kFloat, a.dev);
    need(gs, "grad_state", a.state, at::kFloat, a.dev);
    bool want_state = false, want_g = false;
    for (const std::string &n : names) {
        if (n == "state") want_state = true;
        else if (n == "log_decay") want_g = true;
        else if (n != "k" && n != "v" && n != "q") value_error("need names state, k, v, log_decay and q, got ", n);
    }
    check_kept(a, kept);
    const AttentionGrads r = la_grads(a, state, *k, *v, *g, *q, go, gs, valid, kept, workspace, want_state, want_g);
    py::dict d;
    if (want_state) d["state"] = r.state;
    d["k"] = r.k;
    d["v"] = r.v;
    if (want_g) d["log_decay"] = r.g;
    d["q"] = r.q;
    return d;
}

struct LinearAttention : torch::autograd::Function<LinearAttention> {
    static variable_list forward(AutogradContext *ctx, const OptTensor &state, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &q,
                                 std::optional<double> scale, const OptTensor &valid, bool keep) {
        const Attention a = attention(k, v, g, q, scale, valid);
        need(state, "state", a.state, at::kFloat, a.dev);
        const Tensor final = make(a.state, at::kFloat, a.dev), out = make(v.sizes(), v.scalar_type(), a.dev);
        const bool wants[5] = {given(state) && state->requires_grad(), k.requires_grad(), v.requires_grad(), g.requires_grad(), q.requires_grad()};
        OptTensor kept;
        if (keep && (wants[0] || wants[1] || wants[2] || wants[3] || wants[4])) kept = scratch(api.la_kept(&a.shape), a.dev);
        la_values(a, state, final, valid, out, kept, std::nullopt);
        auto some = [](const OptTensor &t) { return given(t) ? *t : Tensor(); };
        // (the start state is not read where `kept` is there: the caller may advance it before the backward)
        ctx->save_for_backward({given(kept) ? Tensor() : some(state), k, v, g, q, some(valid), some(kept)});
        if (scale) ctx->saved_data["scale"] = *scale;
        for (int i = 0; i < 5; ++i) ctx->saved_data[std::string("want") + char('0' + i)] = wants[i];
        ctx->set_materialize_grads(false);
        return {out, final};
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        if (!grads[0].defined() && !grads[1].defined()) return variable_list(8);
        const variable_list s = ctx->get_saved_variables();
        const Tensor &state = s[0], &k = s[1], &v = s[2], &g = s[3], &q = s[4], &valid = s[5], &kept = s[6];
        const auto scale = ctx->saved_data.find("scale");
        const Attention a = attention(k, v, g, q, scale == ctx->saved_data.end() ? std::nullopt : std::optional<double>(scale->second.toDouble()), valid);
        const Tensor go = grads[0].defined() ? grads[0].detach().contiguous() : at::zeros(v.sizes(), v.options().requires_grad(false));
        OptTensor gs;
        if (grads[1].defined()) gs = grads[1].detach().contiguous();
        auto want = [&](int i) { return ctx->saved_data[std::string("want") + char('0' + i)].toBool(); };
        const AttentionGrads r = la_grads(a, state, k, v, g, q, go, gs, valid, kept, std::nullopt, want(0), want(3));
        return once({r.state, want(1) ? r.k : Tensor(), want(2) ? r.v : Tensor(), r.g, want(4) ? r.q : Tensor(), Tensor(), Tensor(), Tensor()});
    }
};

py::tuple linear_attention(const OptTensor &state, const OptTensor &k, const OptTensor &v, const OptTensor &g, const OptTensor &q, std::optional<double> scale,
                           const OptTensor &valid, bool recompute) {
    if (!given(k) || !given(v) || !given(g) || !given(q)) type_error("k, v, log_decay and q must be torch tensors");
    const variable_list r = LinearAttention::apply(state, *k, *v, *g, *q, scale, valid, !recompute && at::GradMode::is_enabled());
    return py::make_tuple(r[0], r[1]);
}

// ---- group norm ------------------------------------------------------------------------------------------------------

struct Norm {
    sdm_group_shape shape;
    const void *x;
    int64_t sample, row;
    at::ScalarType wdtype;
    int index;
    at::Device dev;
};

Norm norm_of(const Tensor &x, int64_t groups, const OptTensor &weight, const OptTensor &bias, int activation, double eps, const OptTensor &valid) {
    const int code = dtype_code(x.scalar_type());
    if (code < 0) type_error("x must be float32 or bfloat16, got ", name_of(x.scalar_type()));
    if (x.dim() < 2 || x.size(-1) < 1) value_error("x must be [N, ..., channels], got ", x.sizes());
    const int index = on(x);
    const at::Device dev = x.device();
    const int64_t N = x.size(0), C = x.size(-1), last = x.dim() - 1;
    if (groups < 1 || C % groups) value_error("the channels (", C, ") must be a multiple of the groups (", groups, ")");
    // the axes between the first and the last as one of L rows, `row` elements apart
    int64_t L = 1, row = C;
    bool begun = false;
    for (int64_t d = last - 1; d >= 1; --d) {
        if (x.size(d) == 1) continue;
        if (begun && x.numel() > 0 && x.stride(d) != row * L) value_error("x: its axes between the first and the last must count as one, strides ", x.strides());
        if (!begun) row = x.stride(d);
        begun = true;
        L *= x.size(d);
    }
    if (x.stride(last) != 1 && C > 1) value_error("x: the last axis must be dense, its stride is ", x.stride(last));
    const Tensor *w = given(weight) ? given(weight) : given(bias);
    const at::ScalarType wdtype = w ? w->scalar_type() : x.scalar_type();
    if (dtype_code(wdtype) < 0) type_error(given(weight) ? "weight" : "bias", ": expected float32 or bfloat16, got ", name_of(wdtype));
    need(weight, "weight", {C}, wdtype, dev);
    need(bias, "bias", {C}, wdtype, dev);
    need(valid, "valid_rows", {N}, at::kInt, dev);
    return {{N, L, small(C, "channels"), small(groups, "groups"), code, dtype_code(wdtype), activation, float(eps)}, x.data_ptr(), x.stride(0), row, wdtype,
            index, dev};
}

OptTensor norm_scratch(const Norm &a, bool backward, const OptTensor &workspace) {
    if (given(workspace)) return workspace;
    const size_t bytes = api.gn_bytes(&a.shape, backward);
    return bytes ? OptTensor(scratch(bytes, a.dev)) : std::nullopt;
}

struct NormValues {
    Tensor y, mean, rstd;
};
NormValues gn_values(const Norm &a, const Tensor &x, const OptTensor &weight, const OptTensor &bias, const OptTensor &valid, const OptTensor &out,
                     const OptTensor &workspace) {
    const std::array<int64_t, 2> size{a.shape.samples, a.shape.groups};
    NormValues r{given(out) ? *out : make(x.sizes(), x.scalar_type(), a.dev), make(size, at::kFloat, a.dev), make(size, at::kFloat, a.dev)};
    const sdm_exec e = exec_of(a.index, norm_scratch(a, false, workspace));
    check_rc(api.gn_fwd(&a.shape, a.x, a.sample, a.row, ptr<void>(weight), ptr<void>(bias), ptr<int32_t>(valid), r.y.data_ptr(), ptr<float>(r.mean),
                        ptr<float>(r.rstd), &e));
    return r;
}

py::tuple gn_fwd(const Tensor &x, int64_t groups, const OptTensor &weight, const OptTensor &bias, int activation, double eps, const OptTensor &valid,
                 const OptTensor &out, const OptTensor &workspace) {
    const Norm a = norm_of(x, groups, weight, bias, activation, eps, valid);
    need(out, "out", x.sizes(), x.scalar_type(), a.dev);
    const NormValues r = gn_values(a, x, weight, bias, valid, out, workspace);
    wrote({&out});
    return py::make_tuple(r.y, r.mean, r.rstd);
}

struct NormGrads {
    Tensor x, weight, bias;
};
NormGrads gn_grads(const Norm &a, const Tensor &go, const Tensor &x, const Tensor &mean, const Tensor &rstd, const OptTensor &weight, const OptTensor &bias,
                   const OptTensor &valid, const OptTensor &workspace, bool want_x, bool want_weight, bool want_bias) {
    NormGrads r;
    if (want_x) r.x = make(x.sizes(), x.scalar_type(), a.dev);
    if (want_weight) r.weight = make({a.shape.channels}, a.wdtype, a.dev);
    if (want_bias) r.bias = make({a.shape.channels}, a.wdtype, a.dev);
    const sdm_exec e = exec_of(a.index, norm_scratch(a, true, workspace));
    check_rc(api.gn_bwd(&a.shape, go.data_ptr(), a.x, a.sample, a.row, ptr<void>(weight), ptr<void>(bias), ptr<int32_t>(valid), ptr<float>(mean),
                        ptr<float>(rstd), ptr<void>(r.x), ptr<void>(r.weight), ptr<void>(r.bias), &e));
    return r;
}

py::dict gn_bwd(const Tensor &go, const Tensor &x, int64_t groups, const Tensor &mean, const Tensor &rstd, const OptTensor &weight, const OptTensor &bias,
                int activation, double eps, const OptTensor &valid, const std::vector<std::string> &names, const OptTensor &workspace) {
    const Norm a = norm_of(x, groups, weight, bias, activation, eps, valid);
    need(go, "grad_out", x.sizes(), x.scalar_type(), a.dev);
    need(mean, "mean", {a.shape.samples, groups}, at::kFloat, a.dev);
    need(rstd, "rstd", {a.shape.samples, groups}, at::kFloat, a.dev);
    bool want[3] = {};
    for (const std::string &n : names) {
        if (n == "x") want[0] = true;
        else if (n == "weight") want[1] = true;
        else if (n == "bias") want[2] = true;
        else value_error("need names x, weight and bias, got ", n);
    }
    const NormGrads r = gn_grads(a, go, x, mean, rstd, weight, bias, valid, workspace, want[0], want[1], want[2]);
    py::dict d;
    if (want[0]) d["x"] = r.x;
    if (want[1]) d["weight"] = r.weight;
    if (want[2]) d["bias"] = r.bias;
    return d;
}

struct GroupNorm : torch::autograd::Function<GroupNorm> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, int64_t groups, const OptTensor &weight, const OptTensor &bias, int64_t activation, double eps,
                          const OptTensor &valid) {
        const Norm a = norm_of(x, groups, weight, bias, int(activation), eps, valid);
        const NormValues r = gn_values(a, x, weight, bias, valid, std::nullopt, std::nullopt);
        auto some = [](const OptTensor &t) { return given(t) ? *t : Tensor(); };
        ctx->save_for_backward({x, some(weight), some(bias), some(valid), r.mean, r.rstd});
        ctx->saved_data["groups"] = groups;
        ctx->saved_data["activation"] = activation;
        ctx->saved_data["eps"] = eps;
        ctx->saved_data["wants"] = int64_t(x.requires_grad()) | int64_t(given(weight) && weight->requires_grad()) << 1 |
                                   int64_t(given(bias) && bias->requires_grad()) << 2;
        return r.y;
    }
    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        const variable_list s = ctx->get_saved_variables();
        const Tensor &x = s[0], &weight = s[1], &bias = s[2], &valid = s[3];
        const Norm a = norm_of(x, ctx->saved_data["groups"].toInt(), weight, bias, int(ctx->saved_data["activation"].toInt()), ctx->saved_data["eps"].toDouble(),
                               valid);
        const int64_t wants = ctx->saved_data["wants"].toInt();
        const NormGrads r = gn_grads(a, grads[0].detach().contiguous(), x, s[4], s[5], weight, bias, valid, std::nullopt, wants & 1, wants & 2, wants & 4);
        return once({r.x, Tensor(), r.weight, r.bias, Tensor(), Tensor(), Tensor()});
    }
};

Tensor group_norm(const Tensor &x, int64_t groups, const OptTensor &weight, const OptTensor &bias, int64_t activation, double eps, const OptTensor &valid) {
    return GroupNorm::apply(x, groups, weight, bias, activation, eps, valid);
}

void bind(const py::dict &addresses, const py::object &error) {
    auto take = [&](auto &f, const char *name) { f = reinterpret_cast<std::decay_t<decltype(f)>>(addresses[name].cast<uintptr_t>()); };
    take(api.la_fwd, "sdm_linear_attention_fwd");
    take(api.la_step, "sdm_linear_attention_step");
    take(api.la_bwd, "sdm_linear_attention_bwd");
    take(api.la_bytes, "sdm_linear_attention_workspace_bytes");
    take(api.la_kept, "sdm_linear_attention_kept_bytes");
    take(api.gn_fwd, "sdm_group_norm_fwd");
    take(api.gn_bwd, "sdm_group_norm_bwd");
    take(api.gn_bytes, "sdm_group_norm_workspace_bytes");
    take(api.last_error, "sdm_last_error");
    static PyObject *raise = error.inc_ref().ptr();      // SdmError, for the process's life
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const SdmFailure &e) {
            const py::object x = py::reinterpret_borrow<py::object>(raise)(e.code, std::string(e.what()));
            PyErr_SetObject(raise, x.ptr());
        }
    });
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    m.def("bind", &bind);
    m.def("linear_attention_fwd", &la_fwd);
    m.def("linear_attention_step", &la_step);
    m.def("linear_attention_bwd", &la_bwd);
    m.def("linear_attention", &linear_attention);
    m.def("group_norm_fwd", &gn_fwd);
    m.def("group_norm_bwd", &gn_bwd);
    m.def("group_norm", &group_norm);
}

"""The dense gated delta rule (sequences, training, single tokens) and layer norm (forward, training), as cases to
measure: the inputs of each, one pass through it, the work that a pass cannot do without, and its values in 64 bits.

Where ``own`` is false a pass computes the operator in elementary torch operations in float32, rounded once at the end;
where it is true it calls chunked_sparse_delta_amd.

The gated delta rule, per stream and value head, with a state S of [head_dim, value_dim] (scale = head_dim ** -0.5):
    S' = exp(g_t) S;  u_t = beta_t (v_t - k_t S');  S = S' + k_t u_t;  o_t = scale q_t S
Value head h reads key head h // (value heads / key heads). Tokens at and past a stream's valid count are padding: they
leave the state alone and read 0.
Layer norm, per row: y = (x - mean) / sqrt(var + eps) * weight + bias.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64     # tokens of a chunk of the plain form
EPS = 1e-5


def listed():
    def delta(name, kind, P, T, Hk, Hv, K, V, dtype, ragged=False):
        return {"name": name, "kind": kind, "P": P, "T": T, "Hk": Hk, "Hv": Hv, "K": K, "V": V, "dtype": dtype,
                "ragged": ragged}

    def norm(name, kind, rows, N, dtype):
        return {"name": name, "kind": kind, "rows": rows, "N": N, "dtype": dtype}

    return [
        # one stream generating: the latency of one layer's state update
        delta("step_one_stream", "step", 1, 1, 16, 16, 128, 128, "bf16"),
        # a serving batch generating one token each, keys shared by pairs of value heads
        delta("step_batch", "step", 64, 1, 16, 32, 128, 128, "bf16"),
        # a few proposed tokens per stream checked at once, float32, widths off the powers of two
        delta("step_few_tokens_odd", "step", 7, 3, 5, 10, 72, 200, "f32"),
        # a short prompt on a small layer
        delta("fwd_short", "fwd", 1, 200, 4, 4, 64, 64, "bf16"),
        # the streams, tokens and width of the memory op's first benchmark workload, 8 heads
        delta("fwd_width64", "fwd", 8, 2048, 8, 8, 64, 64, "bf16"),
        # a batch of prompts of unequal lengths
        delta("fwd_ragged", "fwd", 4, 4096, 16, 16, 128, 128, "bf16", True),
        # one long document, keys shared: few states, a long sequential axis
        delta("fwd_long", "fwd", 1, 16384, 8, 16, 128, 128, "bf16"),
        # a training step of an odd float32 layer
        delta("train_odd", "train", 3, 301, 3, 6, 40, 72, "f32", True),
        # a training step of an ordinary layer, keys shared
        delta("train", "train", 4, 2048, 8, 16, 128, 128, "bf16"),
        # the norm before such a layer: one token of a batch of streams
        norm("norm_decode", "norm_fwd", 64, 4096, "bf16"),
        # the same in training, an ordinary batch of tokens
        norm("norm_train", "norm_train", 16384, 4096, "bf16"),
        # ... and rows of an odd width in float32
        norm("norm_train_odd", "norm_train", 1001, 1537, "f32"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["step", "fwd", "train", "norm_fwd", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind.startswith("norm"):
        N = _log(rng, 64, 8192)
        return {"kind": kind, "rows": _log(rng, 1, (1 << 26) // N), "N": N, "dtype": dtype}
    Hk, group = _log(rng, 1, 16), rng.choice([1, 1, 2, 4])
    K, V = (rng.choice([64, 128]),) * 2 if rng.random() < 0.5 else (_log(rng, 16, 256), _log(rng, 16, 256))
    heads = Hk * group
    if kind == "step":
        P = _log(rng, 1, max(1, min(128, (1 << 25) // (heads * K * V))))
        T = rng.choice([1, 1, 1, 2, 5, 8])
    else:
        P = _log(rng, 1, max(1, min(8, (1 << 21) // (heads * K * V))))
        most = (1 << 32 if kind == "fwd" else 1 << 31) // (P * heads * K * V)   # tokens
        T = _log(rng, 16, min(16384 if kind == "fwd" else 2048, most))
    return {"kind": kind, "P": P, "T": T, "Hk": Hk, "Hv": heads, "K": K, "V": V, "dtype": dtype,
            "ragged": rng.random() < 0.5}


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"].startswith("norm"):
        n, N, rows = case["rows"] * case["N"], case["N"], case["rows"]
        if case["kind"] == "norm_fwd":    # x in, y out
            return {"bytes": 2 * es * n + 2 * es * N + 8 * rows, "flops": 8 * n}
        # x and grad_out in, y and grad_x out
        return {"bytes": 4 * es * n + 4 * es * N + 8 * rows, "flops": 20 * n}
    P, T, Hk, Hv, K, V = (case[k] for k in ("P", "T", "Hk", "Hv", "K", "V"))
    live = P * T if not case["ragged"] else P * (T + T // 2) // 2    # the mean of the drawn counts
    tokens = live * (es * (2 * Hk * K + Hv * V) + 8 * Hv) + P * T * es * Hv * V     # inputs, and o
    state = 2 * 4 * P * Hv * K * V
    flops = live * Hv * 6 * K * V     # k S', k u and q S: a product and a sum each
    if case["kind"] == "train":       # the inputs again, grad_o, and the gradients out; the gradients' own products
        return {"bytes": tokens + state + live * (2 * es * (2 * Hk * K + Hv * V) + 16 * Hv) + P * T * es * Hv * V
                + 3 * 4 * P * Hv * K * V, "flops": 3 * flops}
    return {"bytes": tokens + state, "flops": flops}


def prepare(case, seed):
    dev, dt = torch.device("cuda:0"), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["kind"].startswith("norm"):
        rows, N = case["rows"], case["N"]
        s = {"case": case, "x": (2.0 * randn(rows, N) + randn(rows, 1)).to(dt), "weight": (1.0 + 0.2 * randn(N)).to(dt),
             "bias": (0.2 * randn(N)).to(dt)}
        if case["kind"] == "norm_train":
            s["grad_out"] = randn(rows, N).to(dt)
            for n in ("x", "weight", "bias"):
                s[n].requires_grad_()
        return s
    P, T, Hk, Hv, K, V = (case[k] for k in ("P", "T", "Hk", "Hv", "K", "V"))

    def unit(*shape):     # what a convolution's activation and a normalisation leave of a projection
        x = torch.nn.functional.silu(randn(*shape))
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = {"case": case, "q": unit(P, T, Hk, K), "k": unit(P, T, Hk, K), "v": randn(P, T, Hv, V).to(dt),
         "beta": torch.sigmoid(randn(P, T, Hv)), "state": 0.5 * randn(P, Hv, K, V), "valid": None}
    rate = 0.02 + torch.rand((Hv,), generator=gen, device=dev)
    s["log_decay"] = -rate * torch.nn.functional.softplus(randn(P, T, Hv) - 1.0)
    if case["ragged"]:
        s["valid"] = torch.randint(T // 2, T + 1, (P,), generator=gen, device=dev, dtype=torch.int32)
    if case["kind"] == "train":
        s["grad_out"], s["grad_state"] = randn(P, T, Hv, V).to(dt), 0.1 * randn(P, Hv, K, V)
        for n in ("state", "k", "v", "beta", "log_decay", "q"):
            s[n].requires_grad_()
    else:
        s["state_out"] = torch.empty_like(s["state"])
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _inputs32(state, k, v, beta, log_decay, q, valid):
    """The inputs in float32, heads before tokens, the keys once per value head, padding tokens with beta and g 0."""
    group = v.shape[2] // k.shape[2]
    scale = k.shape[-1] ** -0.5
    k, q, v = (x.float().transpose(1, 2) for x in (k, q, v))
    k, q = (x.repeat_interleave(group, 1) for x in (k, q))
    beta, g = beta.transpose(1, 2), log_decay.transpose(1, 2)
    live = None
    if valid is not None:
        live = (torch.arange(v.shape[2], device=v.device) < valid[:, None])[:, None]
        beta, g = (torch.where(live, x, torch.zeros_like(x)) for x in (beta, g))
    return state, k, v, beta, g, q * scale, live


def _plain_chunks(state, k, v, beta, log_decay, q, valid):
    """Chunk by chunk: with G the running sum of g in a chunk and A = tril(exp(G_i - G_j) k_i k_j, -1),
    U = (1 + beta A)^-1 beta (V - exp(G) K S); O = exp(G) Q S + tril(exp(G_i - G_j) q_i k_j) U;
    S = exp(G_C) S + (exp(G_C - G) K)^T U."""
    dtype = v.dtype
    S, k, v, beta, g, q, live = _inputs32(state, k, v, beta, log_decay, q, valid)
    P, H, T, K = k.shape
    C = min(CHUNK, 1 << (T - 1).bit_length())
    Nt = -(-T // C)
    pad = Nt * C - T

    def chunks(x):
        if pad:
            x = torch.cat([x, x.new_zeros(P, H, pad, *x.shape[3:])], 2)
        return x.reshape(P, H, Nt, C, *x.shape[3:])

    k, v, beta, g, q = (chunks(x) for x in (k, v, beta, g, q))
    G = g.cumsum(-1)
    at = torch.arange(C, device=k.device)
    lower = at[:, None] >= at
    D = torch.where(lower, G[..., :, None] - G[..., None, :], -math.inf).exp()
    L = beta[..., None] * torch.where(at[:, None] > at, D * (k @ k.transpose(-1, -2)), 0.0)
    QK = D * (q @ k.transpose(-1, -2))
    X = torch.eye(C, device=k.device).expand_as(L)
    s = 1
    while s < C:     # the inverses of the diagonal blocks of size s, to those of size 2 s
        join = (at[:, None] // s % 2 == 1) & (at[:, None] // s - 1 == at // s)
        X = X - X @ (torch.where(join, L, 0.0) @ X)
        s *= 2
    fresh = X @ (beta[..., None] * v)
    W = X @ ((beta * G.exp())[..., None] * k)
    late = (G[..., -1:] - G).exp()[..., None] * k
    early = G.exp()[..., None] * q
    last = G[..., -1].exp()[..., None, None]
    outs = []
    for n in range(Nt):
        U = fresh[:, :, n] - W[:, :, n] @ S
        outs.append(early[:, :, n] @ S + QK[:, :, n] @ U)
        S = last[:, :, n] * S + late[:, :, n].transpose(-1, -2) @ U
    out = torch.cat(outs, 2)[:, :, :T]
    if live is not None:
        out = torch.where(live[..., None], out, 0.0)
    return out.transpose(1, 2).to(dtype), S


def _plain_tokens(state, k, v, beta, log_decay, q, valid):
    """Token by token, as the rule is defined."""
    dtype = v.dtype
    S, k, v, beta, g, q, live = _inputs32(state, k, v, beta, log_decay, q, valid)
    decay = g.exp()
    outs = []
    for t in range(k.shape[2]):
        S = decay[:, :, t, None, None] * S
        u = beta[:, :, t, None] * (v[:, :, t] - (k[:, :, t, :, None] * S).sum(-2))
        S = S + k[:, :, t, :, None] * u[:, :, None]
        outs.append((q[:, :, t, :, None] * S).sum(-2))
    out = torch.stack(outs, 1)
    if live is not None:
        out = torch.where(live[:, 0, :, None, None], out, 0.0)
    return out.to(dtype), S


def _plain_norm(x, weight, bias):
    dtype = x.dtype
    x = x.float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return (d * rstd * weight.float() + bias.float()).to(dtype), mean[:, 0], rstd[:, 0]


# ---- one pass --------------------------------------------------------------------------------------------------------

RULE = ("state", "k", "v", "beta", "log_decay", "q")
NORM = ("x", "weight", "bias")


def run(s):
    kind = s["case"]["kind"]
    if own:
        return _run_own(s, kind)
    if kind == "norm_fwd":
        y, mean, rstd = _plain_norm(s["x"], s["weight"], s["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_train":
        y, _, _ = _plain_norm(s["x"], s["weight"], s["bias"])
        grads = torch.autograd.grad(y, [s[n] for n in NORM], s["grad_out"])
        return {"y": y.detach(), **{"grad_" + n: g for n, g in zip(NORM, grads)}}
    args = [s[n] for n in RULE] + [s["valid"]]
    if kind == "step":
        out, state = _plain_tokens(*args)
        return {"out": out, "state": state}
    out, state = _plain_chunks(*args)
    if kind == "fwd":
        return {"out": out, "state": state}
    grads = torch.autograd.grad([out, state], [s[n] for n in RULE], [s["grad_out"], s["grad_state"]])
    return {"out": out.detach(), "state": state.detach(), **{"grad_" + n: g for n, g in zip(RULE, grads)}}


def _run_own(s, kind):
    import chunked_sparse_delta_amd as sdm
    if kind == "norm_fwd":
        y, mean, rstd = sdm.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_train":
        y = sdm.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        grads = torch.autograd.grad(y, [s[n] for n in NORM], s["grad_out"])
        return {"y": y.detach(), **{"grad_" + n: g for n, g in zip(NORM, grads)}}
    args = [s[n] for n in RULE]
    if kind == "train":
        out, state = sdm.gated_delta_rule(*args, valid_tokens=s["valid"])
        grads = torch.autograd.grad([out, state], args, [s["grad_out"], s["grad_state"]])
        return {"out": out.detach(), "state": state.detach(), **{"grad_" + n: g for n, g in zip(RULE, grads)}}
    call = sdm.gated_delta_step if kind == "step" else sdm.gated_delta_fwd
    return {"out": call(*args, valid_tokens=s["valid"], state_out=s["state_out"]), "state": s["state_out"]}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["kind"].startswith("norm"):
            return _exact_norm(s, case["kind"] == "norm_train")
        return _exact_rule(s, case["kind"] == "train")


def _exact_norm(s, train):
    x, w, b = (s[n].detach().double() for n in NORM)
    mean = x.sum(1) / x.shape[1]
    var = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
    rstd = 1.0 / torch.sqrt(var + EPS)
    hat = (x - mean[:, None]) * rstd[:, None]
    y = hat * w + b
    if not train:
        return {"y": y, "mean": mean, "rstd": rstd}
    dy = s["grad_out"].double()
    dh = dy * w
    dx = rstd[:, None] * (dh - dh.mean(1, keepdim=True) - hat * (dh * hat).mean(1, keepdim=True))
    return {"y": y, "grad_x": dx, "grad_weight": (dy * hat).sum(0), "grad_bias": dy.sum(0)}


def _exact_rule(s, train):
    """The rule token by token and, for training, its adjoint token by token backwards, the states of a stretch of
    tokens computed again from the one kept at its start."""
    S, k, v, beta, g, q = (s[n].detach().double() for n in RULE)
    P, T, Hk, K = k.shape
    Hv, V = v.shape[2:]
    n, scale, stretch = Hv // Hk, K ** -0.5, 64
    valid = s["valid"] if s["valid"] is not None else torch.full((P,), T, device=k.device)
    a = g.exp()

    def forward(S, t):
        kt, on = k[:, t].repeat_interleave(n, 1), (t < valid)[:, None, None]
        Sd = a[:, t, :, None, None] * S
        e = v[:, t] - torch.matmul(kt[:, :, None], Sd)[:, :, 0]
        new = Sd + kt[..., None] * (beta[:, t, :, None] * e)[:, :, None]
        return torch.where(on[..., None], new, S), Sd, e

    out = torch.zeros(P, T, Hv, V, dtype=torch.float64, device=k.device)
    kept = []
    for t in range(T):
        if train and t % stretch == 0:
            kept.append(S)
        S, _, _ = forward(S, t)
        o = scale * torch.matmul(q[:, t].repeat_interleave(n, 1)[:, :, None], S)[:, :, 0]
        out[:, t] = torch.where((t < valid)[:, None, None], o, 0.0)
    got = {"out": out, "state": S}
    if not train:
        return got
    do, dS = s["grad_out"].double(), s["grad_state"].double()
    dq, dk, dv, dbeta, dg = (torch.zeros_like(x) for x in (q, k, v, beta, g))
    for c in reversed(range(len(kept))):
        at, S, seen = range(c * stretch, min(T, (c + 1) * stretch)), kept[c], []
        for t in at:
            new, Sd, e = forward(S, t)
            seen.append((Sd, e, new))
            S = new
        for t in reversed(at):
            Sd, e, new = seen.pop()
            on = (t < valid)[:, None, None]
            kt, qt = (x[:, t].repeat_interleave(n, 1) for x in (k, q))
            dot, b = torch.where(on, scale * do[:, t], 0.0), beta[:, t, :, None]
            dqt = torch.matmul(new, dot[..., None])[..., 0]
            dSt = dS + qt[..., None] * dot[:, :, None]
            du = torch.matmul(kt[:, :, None], dSt)[:, :, 0]
            dkt = torch.matmul(dSt, (b * e)[..., None])[..., 0] - torch.matmul(Sd, (b * du)[..., None])[..., 0]
            dSd = dSt - kt[..., None] * (b * du)[:, :, None]
            dq[:, t], dk[:, t] = (torch.where(on, x.reshape(P, Hk, n, K).sum(2), 0.0) for x in (dqt, dkt))
            dv[:, t] = torch.where(on, b * du, 0.0)
            dbeta[:, t] = torch.where(on[..., 0], (du * e).sum(-1), 0.0)
            dg[:, t] = torch.where(on[..., 0], (dSd * Sd).sum((-1, -2)), 0.0)
            dS = torch.where(on[..., None], a[:, t, :, None, None] * dSd, dS)
    return got | {"grad_state": dS, "grad_k": dk, "grad_v": dv, "grad_beta": dbeta, "grad_log_decay": dg, "grad_q": dq}

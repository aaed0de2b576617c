"""Linear attention with a decay for each head (sequences, training, single tokens) and group norm with an activation
(forward, training), as cases to measure: the inputs of each, one pass through it, the work that a pass cannot do
without, and its values in 64 bits.

Where ``own`` is false a pass computes the operator in elementary torch operations in float32, rounded once at the end;
where it is true it calls chunked_sparse_delta_amd.

Linear attention, per stream and value head, with a state S of [head_dim, value_dim] (scale = head_dim ** -0.5):
    S = exp(g_t) S + k_t v_t;  o_t = scale q_t S
Value head h reads key head h // (value heads / key heads). The log-decay g is one number for each head, or one for each
token and head. Tokens at and past a stream's valid count are padding: they leave the state alone and read 0.

Group norm of x [samples, rows, channels] (channels last), the channels in groups of neighbours: per sample and group, over
its rows and channels,
    y = act((x - mean) / sqrt(var + eps) * weight + bias),  act(z) = z, z sigmoid(z) (silu) or z Phi(z) (gelu)
with a weight and a bias for each channel. Rows at and past a sample's valid count are padding: they do not count and
give 0.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64     # tokens of a chunk of the plain form
EPS = 1e-5


def listed():
    def attn(name, kind, P, T, Hk, Hv, K, V, dtype, decay, ragged=False):
        return {"name": name, "kind": kind, "P": P, "T": T, "Hk": Hk, "Hv": Hv, "K": K, "V": V, "dtype": dtype,
                "decay": decay, "ragged": ragged}

    def norm(name, kind, N, L, C, G, dtype, act, ragged=False):
        return {"name": name, "kind": kind, "N": N, "L": L, "C": C, "G": G, "dtype": dtype, "act": act, "ragged": ragged}

    return [
        # one stream generating: the latency of one layer's state update
        attn("step_one_stream", "step", 1, 1, 16, 16, 128, 128, "bf16", "head"),
        # a serving batch generating one token each, keys shared by pairs of value heads
        attn("step_batch", "step", 64, 1, 16, 32, 128, 128, "bf16", "token"),
        # a short prompt on a small layer
        attn("fwd_short", "fwd", 1, 200, 4, 4, 64, 64, "bf16", "head"),
        # a batch of prompts of unequal lengths
        attn("fwd_ragged", "fwd", 4, 4096, 16, 16, 128, 128, "bf16", "token", True),
        # one long document, keys shared: few states, a long sequential axis
        attn("fwd_long", "fwd", 1, 16384, 8, 16, 128, 128, "bf16", "head"),
        # a float32 layer with widths off the powers of two
        attn("fwd_odd", "fwd", 2, 1500, 5, 10, 72, 200, "f32", "token"),
        # a training step of an odd float32 layer, its decays learned for each head
        attn("train_odd", "train", 3, 301, 3, 6, 40, 72, "f32", "head", True),
        # a training step of an ordinary layer, keys shared, decays made from the tokens
        attn("train", "train", 4, 2048, 8, 16, 128, 128, "bf16", "token"),
        # the readings' norm of each head: one token of a batch of streams
        norm("norm_decode", "norm_fwd", 64, 1, 4096, 32, "bf16", "silu"),
        # the same in training, an ordinary batch of tokens
        norm("norm_train_tokens", "norm_train", 8192, 1, 4096, 32, "bf16", "silu"),
        # features over positions, large enough for the whole device only
        norm("norm_train_positions", "norm_train", 8, 4096, 512, 32, "bf16", "silu"),
        # ... of unequal lengths in float32, ten channels to a group
        norm("norm_train_odd", "norm_train", 5, 1001, 320, 32, "f32", "gelu", True),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["step", "fwd", "train", "norm_fwd", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind.startswith("norm"):
        G, D = rng.choice([1, 2, 4, 8, 16, 32, 32, 48]), _log(rng, 4, 256)
        most = (1 << 24) // (G * D)
        L = 1 if rng.random() < 0.3 else _log(rng, 2, min(8192, most))
        return {"kind": kind, "N": _log(rng, 1, max(1, min(16384, most // L))), "L": L, "C": G * D, "G": G, "dtype": dtype,
                "act": rng.choice(["none", "silu", "silu", "gelu"]), "ragged": L > 1 and rng.random() < 0.3}
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
            "decay": rng.choice(["head", "token"]), "ragged": rng.random() < 0.5}


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"].startswith("norm"):
        N, L, C, G = (case[k] for k in ("N", "L", "C", "G"))
        whole, live = N * L * C, N * L * C if not case["ragged"] else N * (L + 1) // 2 * C
        small = 2 * es * C + 8 * N * G
        if case["kind"] == "norm_fwd":    # x in, y out
            return {"bytes": es * (live + whole) + small, "flops": 12 * live}
        # x and grad_out in, y and grad_x out
        return {"bytes": 2 * es * (live + whole) + 2 * small, "flops": 30 * live}
    P, T, Hk, Hv, K, V = (case[k] for k in ("P", "T", "Hk", "Hv", "K", "V"))
    live = P * T if not case["ragged"] else P * (T + T // 2) // 2    # the mean of the drawn counts
    gates = 4 * (live * Hv if case["decay"] == "token" else Hv)
    rows = live * es * (2 * Hk * K + Hv * V)
    o = P * T * es * Hv * V
    state = 2 * 4 * P * Hv * K * V
    flops = live * Hv * 4 * K * V     # k v and q S: a product and a sum each
    if case["kind"] == "train":       # the inputs again, grad_o, and the gradients out; the gradients' own products
        return {"bytes": 3 * rows + 3 * gates + 2 * o + state + 3 * 4 * P * Hv * K * V, "flops": 3 * flops}
    return {"bytes": rows + gates + o + state, "flops": flops}


def prepare(case, seed):
    dev, dt = torch.device("cuda:0"), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def counts(n, lo, hi):
        return torch.randint(lo, hi + 1, (n,), generator=gen, device=dev, dtype=torch.int32) if case["ragged"] else None

    if case["kind"].startswith("norm"):
        N, L, C = (case[k] for k in ("N", "L", "C"))
        s = {"case": case, "x": (2.0 * randn(N, L, C) + randn(N, 1, C)).to(dt), "weight": (1.0 + 0.2 * randn(C)).to(dt),
             "bias": (0.2 * randn(C)).to(dt), "valid": counts(N, 1, L)}
        if case["kind"] == "norm_train":
            s["grad_out"] = randn(N, L, C).to(dt)
            for n in NORM:
                s[n].requires_grad_()
        return s
    P, T, Hk, Hv, K, V = (case[k] for k in ("P", "T", "Hk", "Hv", "K", "V"))
    s = {"case": case, "q": torch.nn.functional.silu(randn(P, T, Hk, K)).to(dt),
         "k": torch.nn.functional.silu(randn(P, T, Hk, K)).to(dt), "v": randn(P, T, Hv, V).to(dt),
         "state": 0.5 * randn(P, Hv, K, V), "valid": counts(P, T // 2, T)}
    if case["decay"] == "head":    # memories from two tokens to hundreds
        s["log_decay"] = torch.log1p(-torch.exp2(-1.0 - 8.0 * torch.rand((Hv,), generator=gen, device=dev)))
    else:
        rate = 0.02 + torch.rand((Hv,), generator=gen, device=dev)
        s["log_decay"] = -rate * torch.nn.functional.softplus(randn(P, T, Hv) - 1.0)
    if case["kind"] == "train":
        s["grad_out"], s["grad_state"] = randn(P, T, Hv, V).to(dt), 0.1 * randn(P, Hv, K, V)
        for n in ATTN:
            s[n].requires_grad_()
    else:
        s["state_out"] = torch.empty_like(s["state"])
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _inputs32(state, k, v, log_decay, q, valid):
    """The inputs in float32, heads before tokens, the keys once per value head, padding tokens with k and g 0."""
    P, T, Hv = v.shape[:3]
    group = Hv // k.shape[2]
    scale = k.shape[-1] ** -0.5
    k, q, v = (x.float().transpose(1, 2) for x in (k, q, v))
    k, q = (x.repeat_interleave(group, 1) for x in (k, q))
    g = log_decay.expand(P, T, Hv).transpose(1, 2)
    live = None
    if valid is not None:
        live = (torch.arange(T, device=v.device) < valid[:, None])[:, None]
        g = torch.where(live, g, 0.0)
        k = torch.where(live[..., None], k, 0.0)
    return state, k, v, g, q * scale, live


def _plain_chunks(state, k, v, log_decay, q, valid):
    """Chunk by chunk, G the running sum of g in a chunk: O = exp(G) Q S + tril(exp(G_i - G_j) q_i k_j) V;
    S = exp(G_C) S + (exp(G_C - G) K)^T V."""
    dtype = v.dtype
    S, k, v, g, q, live = _inputs32(state, k, v, log_decay, q, valid)
    P, H, T, K = k.shape
    C = min(CHUNK, 1 << (T - 1).bit_length())
    Nt = -(-T // C)
    pad = Nt * C - T

    def chunks(x):
        if pad:
            x = torch.cat([x, x.new_zeros(P, H, pad, *x.shape[3:])], 2)
        return x.reshape(P, H, Nt, C, *x.shape[3:])

    k, v, g, q = (chunks(x) for x in (k, v, g, q))
    G = g.cumsum(-1)
    at = torch.arange(C, device=k.device)
    D = torch.where(at[:, None] >= at, G[..., :, None] - G[..., None, :], -math.inf).exp()
    inside = (D * (q @ k.transpose(-1, -2))) @ v
    fresh = ((G[..., -1:] - G).exp()[..., None] * k).transpose(-1, -2) @ v
    last = G[..., -1].exp()[..., None, None]
    starts = []
    for n in range(Nt):
        starts.append(S)
        S = last[:, :, n] * S + fresh[:, :, n]
    out = (inside + (G.exp()[..., None] * q) @ torch.stack(starts, 2)).reshape(P, H, Nt * C, -1)[:, :, :T]
    if live is not None:
        out = torch.where(live[..., None], out, 0.0)
    return out.transpose(1, 2).to(dtype), S


def _plain_tokens(state, k, v, log_decay, q, valid):
    """Token by token, as it is defined."""
    dtype = v.dtype
    S, k, v, g, q, live = _inputs32(state, k, v, log_decay, q, valid)
    decay = g.exp()
    outs = []
    for t in range(k.shape[2]):
        S = decay[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None]
        outs.append((q[:, :, t, :, None] * S).sum(-2))
    out = torch.stack(outs, 1)
    if live is not None:
        out = torch.where(live[:, 0, :, None, None], out, 0.0)
    return out.to(dtype), S


def _plain_norm(x, weight, bias, G, act, valid):
    dtype, (N, L, C) = x.dtype, x.shape
    x = x.float().reshape(N, L, G, C // G)
    if valid is None:
        mean = x.mean((1, 3), keepdim=True)
        d = x - mean
        var = d.square().mean((1, 3), keepdim=True)
    else:
        live = (torch.arange(L, device=x.device) < valid[:, None])[:, :, None, None]
        count = (valid.clamp(min=1) * (C // G)).float()[:, None, None, None]
        mean = torch.where(live, x, 0.0).sum((1, 3), keepdim=True) / count
        d = torch.where(live, x - mean, 0.0)
        var = d.square().sum((1, 3), keepdim=True) / count
    rstd = (var + EPS).rsqrt()
    z = (d * rstd).reshape(N, L, C) * weight.float() + bias.float()
    if act == "silu":
        z = z * torch.sigmoid(z)
    elif act == "gelu":
        z = 0.5 * z * torch.erfc(-math.sqrt(0.5) * z)
    if valid is not None:
        z = torch.where(live[:, :, 0], z, 0.0)
    return z.to(dtype), mean[:, 0, :, 0], rstd[:, 0, :, 0]


# ---- one pass --------------------------------------------------------------------------------------------------------

ATTN = ("state", "k", "v", "log_decay", "q")
NORM = ("x", "weight", "bias")


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        return _run_own(s, case, kind)
    if kind.startswith("norm"):
        y, mean, rstd = _plain_norm(*(s[n] for n in NORM), case["G"], case["act"], s["valid"])
        if kind == "norm_fwd":
            return {"y": y, "mean": mean, "rstd": rstd}
        grads = torch.autograd.grad(y, [s[n] for n in NORM], s["grad_out"])
        return {"y": y.detach(), **{"grad_" + n: g for n, g in zip(NORM, grads)}}
    args = [s[n] for n in ATTN] + [s["valid"]]
    if kind == "step":
        out, state = _plain_tokens(*args)
        return {"out": out, "state": state}
    out, state = _plain_chunks(*args)
    if kind == "fwd":
        return {"out": out, "state": state}
    grads = torch.autograd.grad([out, state], [s[n] for n in ATTN], [s["grad_out"], s["grad_state"]])
    return {"out": out.detach(), "state": state.detach(), **{"grad_" + n: g for n, g in zip(ATTN, grads)}}


def _run_own(s, case, kind):
    import chunked_sparse_delta_amd as sdm
    if kind.startswith("norm"):
        how = {"activation": None if case["act"] == "none" else case["act"], "eps": EPS, "valid_rows": s["valid"]}
        if kind == "norm_fwd":
            y, mean, rstd = sdm.group_norm_fwd(s["x"], case["G"], s["weight"], s["bias"], **how)
            return {"y": y, "mean": mean, "rstd": rstd}
        y = sdm.group_norm(s["x"], case["G"], s["weight"], s["bias"], **how)
        grads = torch.autograd.grad(y, [s[n] for n in NORM], s["grad_out"])
        return {"y": y.detach(), **{"grad_" + n: g for n, g in zip(NORM, grads)}}
    args = [s[n] for n in ATTN]
    if kind == "train":
        out, state = sdm.linear_attention(*args, valid_tokens=s["valid"])
        grads = torch.autograd.grad([out, state], args, [s["grad_out"], s["grad_state"]])
        return {"out": out.detach(), "state": state.detach(), **{"grad_" + n: g for n, g in zip(ATTN, grads)}}
    call = sdm.linear_attention_step if kind == "step" else sdm.linear_attention_fwd
    return {"out": call(*args, valid_tokens=s["valid"], state_out=s["state_out"]), "state": s["state_out"]}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["kind"].startswith("norm"):
            return _exact_norm(s, case)
        return _exact_attn(s, case["kind"] == "train")


def _exact_norm(s, case):
    """Sample by sample over the valid rows alone; gradients by the formula."""
    G, act = case["G"], case["act"]
    N, L, C = s["x"].shape
    D = C // G
    valid = s["valid"].tolist() if s["valid"] is not None else [L] * N
    full = min(valid) == L
    x, w, b = (s[n].detach().double() for n in NORM)
    w, b = w.view(G, D), b.view(G, D)
    train = case["kind"] == "norm_train"
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    mean, rstd = (torch.zeros(N, G, dtype=torch.float64, device=x.device) for _ in range(2))
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    root2, rootpi = math.sqrt(2.0), math.sqrt(2.0 * math.pi)
    # samples of equal length go together, a bounded number of elements at a time
    step = max(1, (1 << 24) // (L * C)) if full else 1
    for n in range(0, N, step):
        at, rows = slice(n, n + step), L if full else valid[n]
        xs = x[at, :rows].reshape(-1, rows, G, D)
        m = xs.sum((1, 3)) / (rows * D)
        d = xs - m[:, None, :, None]
        r = 1.0 / torch.sqrt((d * d).sum((1, 3)) / (rows * D) + EPS)
        hat = d * r[:, None, :, None]
        z = hat * w + b
        if act == "silu":
            sig = 1.0 / (1.0 + torch.exp(-z))
            a, da = z * sig, sig * (1.0 + z * (1.0 - sig))
        elif act == "gelu":
            phi = 0.5 * torch.special.erfc(-z / root2)
            a, da = z * phi, phi + z * torch.exp(-0.5 * z * z) / rootpi
        else:
            a, da = z, torch.ones_like(z)
        mean[at], rstd[at] = m, r
        y[at, :rows] = a.reshape(-1, rows, C)
        if train:
            dz = s["grad_out"][at, :rows].double().reshape(-1, rows, G, D) * da
            dw += (dz * hat).sum((0, 1))
            db += dz.sum((0, 1))
            h = dz * w
            m1, m2 = (t.sum((1, 3), keepdim=True) / (rows * D) for t in (h, h * hat))
            dx[at, :rows] = (r[:, None, :, None] * (h - m1 - hat * m2)).reshape(-1, rows, C)
    if not train:
        return {"y": y, "mean": mean, "rstd": rstd}
    return {"y": y, "grad_x": dx, "grad_weight": dw.flatten(), "grad_bias": db.flatten()}


def _exact_attn(s, train):
    """Token by token and, for training, its adjoint token by token backwards, the states of a stretch of tokens computed
    again from the one kept at its start."""
    S, k, v, g, q = (s[n].detach().double() for n in ATTN)
    P, T, Hk, K = k.shape
    Hv, V = v.shape[2:]
    n, scale, stretch = Hv // Hk, K ** -0.5, 32
    valid = s["valid"] if s["valid"] is not None else torch.full((P,), T, device=k.device)
    a = g.exp().expand(P, T, Hv)
    group = torch.arange(Hv, device=k.device) // n

    def forward(S, t):
        new = a[:, t, :, None, None] * S + k[:, t, group, :, None] * v[:, t, :, None]
        return torch.where((t < valid)[:, None, None, None], new, S)

    out = torch.zeros(P, T, Hv, V, dtype=torch.float64, device=k.device)
    kept = []
    for t in range(T):
        if train and t % stretch == 0:
            kept.append(S)
        S = forward(S, t)
        o = scale * torch.matmul(q[:, t, group, None], S)[:, :, 0]
        out[:, t] = torch.where((t < valid)[:, None, None], o, 0.0)
    got = {"out": out, "state": S}
    if not train:
        return got
    do, dS = s["grad_out"].double(), s["grad_state"].double()
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    dg = torch.zeros(P, T, Hv, dtype=torch.float64, device=k.device)
    for c in reversed(range(len(kept))):
        at, S, seen = range(c * stretch, min(T, (c + 1) * stretch)), kept[c], []
        for t in at:
            seen.append(S)
            S = forward(S, t)
        for t in reversed(at):
            before = seen.pop()
            on = (t < valid)[:, None, None]
            dot = torch.where(on, scale * do[:, t], 0.0)
            dq[:, t] = torch.matmul(S, dot[..., None])[..., 0].view(P, Hk, n, K).sum(2) * on
            now = dS + q[:, t, group, :, None] * dot[:, :, None]
            dk[:, t] = torch.matmul(now, v[:, t, :, :, None])[..., 0].view(P, Hk, n, K).sum(2) * on
            dv[:, t] = torch.matmul(k[:, t, group, None], now)[:, :, 0] * on
            back = a[:, t, :, None, None] * now
            dg[:, t] = (back * before).sum((-1, -2)) * on[..., 0]
            dS, S = torch.where(on[..., None], back, dS), before
    if g.dim() == 1:
        dg = dg.sum((0, 1))
    return got | {"grad_state": dS, "grad_k": dk, "grad_v": dv, "grad_log_decay": dg, "grad_q": dq}

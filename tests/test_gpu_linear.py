"""Linear attention with a decay on the GPU against its definition in 64 bits (oracle/linear.py).

Bars. A result is a sum of products, and the same sum over the inputs' absolute values, from the oracle too, is the sum A
of its terms' sizes. A term carries its operands' products to 2^-23, decays (an exponential and a rounded exponent that is
at most about 20 where the term counts: 20 * 2^-24 + 2^-22) and up to about 40 additions in float32 (16 products of depth
32, the state's, the scan over segments), 2^-24 each: 64 * 2^-23 A in all. On top a rounded result is off by half a step,
2^-8 of a bfloat16 value, 2^-24 of a float32 one.
A log-decay's gradient sums up to 512 shares of tokens that partly cancel (and a head's one those of every token), each
off by at most 64 * 2^-23 of its terms; independent, they leave 64 * 2^-23 * sqrt(512) = 1.7e-4 of a share; the bar is that,
normwise, against the gradient itself, whose size is that of a share or more.
"""

import math

import pytest
import torch

from oracle import linear as oracle

pytestmark = pytest.mark.gpu
C = 64 * 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
NAMES = ("state", "k", "v", "log_decay", "q")


def make(P, T, Hk, Hv, K, V, dtype, decay="token", ragged=None, seed=0, state=True):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=gen)

    x = {"q": randn(P, T, Hk, K).to(dtype), "k": randn(P, T, Hk, K).to(dtype), "v": randn(P, T, Hv, V).to(dtype),
         "state": randn(P, Hv, K, V) if state else None}
    rate = 0.01 + torch.rand(Hv, generator=gen)
    x["log_decay"] = -0.3 * rate if decay == "head" else -rate * torch.nn.functional.softplus(randn(P, T, Hv) - 1)
    x["valid"] = None if ragged is None else torch.tensor(ragged, dtype=torch.int32)
    return x


def want(x, scale=None, absolute=False):
    f = [None if x[n] is None else x[n].double() for n in NAMES]
    if absolute:
        f = [t if t is None or n == "log_decay" else t.abs() for n, t in zip(NAMES, f)]
    state, k, v, g, q = f
    scale = k.shape[-1] ** -0.5 if scale is None else scale
    return oracle.linear_attention(state, k, v, g, q, abs(scale) if absolute else scale, x["valid"])


def on(x, gpu):
    return {n: None if t is None else t.to(gpu) for n, t in x.items()}


def close(got, ref, size, dtype):
    got = got.double().cpu()
    assert got.shape == ref.shape
    bar = C * size + HALF[dtype] * (ref.abs() + C * size)
    worst = ((got - ref).abs() - bar).max() if got.numel() else torch.tensor(0.0)
    assert bool(((got - ref).abs() <= bar).all()), f"over the bar by {worst:.3g}"


def run(gpu, x, **kw):
    import chunked_sparse_delta_amd as sdm
    d = on(x, gpu)
    final = torch.full((x["v"].shape[0], x["v"].shape[2], x["k"].shape[3], x["v"].shape[3]), math.nan, device=gpu)
    out = sdm.linear_attention_fwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], valid_tokens=d["valid"], state_out=final, **kw)
    torch.cuda.synchronize()
    return out, final


SHAPES = [
    # P, T, Hk, Hv, K, V, dtype, decay
    (1, 1, 1, 1, 1, 1, "f32", "token"), (2, 2, 1, 2, 3, 5, "bf16", "head"), (1, 31, 2, 2, 16, 16, "bf16", "token"),
    (1, 32, 1, 1, 64, 64, "bf16", "token"), (1, 33, 1, 1, 64, 64, "f32", "head"), (2, 63, 2, 4, 40, 72, "f32", "token"),
    (1, 64, 2, 2, 128, 128, "bf16", "head"), (1, 65, 1, 2, 128, 128, "f32", "token"), (1, 127, 1, 1, 65, 129, "bf16", "token"),
    (1, 128, 1, 1, 100, 36, "bf16", "token"), (2, 129, 2, 2, 129, 65, "f32", "head"), (1, 255, 1, 1, 256, 256, "bf16", "token"),
    (1, 256, 1, 1, 256, 250, "f32", "token"), (1, 257, 2, 2, 128, 128, "bf16", "token"), (1, 300, 3, 6, 72, 200, "f32", "token"),
    (1, 513, 1, 2, 200, 128, "bf16", "head"), (2, 600, 1, 1, 64, 64, "f32", "head"), (1, 1111, 2, 4, 33, 17, "bf16", "token"),
    (1, 2300, 1, 1, 16, 8, "f32", "head"),
]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,decay", SHAPES)
def test_forward(gpu, P, T, Hk, Hv, K, V, dtype, decay):
    dt = DT[dtype]
    x = make(P, T, Hk, Hv, K, V, dt, decay, seed=T)
    out, final = run(gpu, x)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("state", [True, False])
def test_ragged_padding_may_hold_anything(gpu, dtype, state):
    """Streams of no, one, some and all valid tokens (a count past the end counts as all); NaN and infinities in padding."""
    dt, counts = DT[dtype], [0, 1, 130, 300, 555, 256]
    x = make(6, 300, 2, 4, 48, 80, dt, ragged=counts, seed=3, state=state)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    for p, n in enumerate(counts):
        for name in ("q", "k", "v", "log_decay"):
            x[name][p, min(n, 300):] = math.nan if name != "v" else math.inf
    out, final = run(gpu, x)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)
    for p, n in enumerate(counts):
        assert not out[p, min(n, 300):].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_at_their_ends(gpu, dtype):
    """Decays of 0, -inf (which clears the state), -1e30 and -80 among ordinary ones; sums of 64 bits keep what follows exact."""
    dt = DT[dtype]
    x = make(1, 400, 1, 2, 64, 64, dt, seed=5)
    g = x["log_decay"]
    g[:, 50:90] = 0.0
    g[0, 100, 0], g[0, 256, 1], g[0, 301, 0], g[0, 17, 1] = -math.inf, -math.inf, -1e30, -80.0
    out, final = run(gpu, x)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)


def test_scale_and_in_place(gpu):
    import chunked_sparse_delta_amd as sdm
    for T in (40, 700):
        x = make(2, T, 1, 2, 32, 48, torch.float32, seed=T)
        for scale in (0.0, -0.7, 3.0):
            d = on(x, gpu)
            out = sdm.linear_attention_fwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], scale=scale)
            (o, s), (ao, as_) = want(x, scale), want(x, scale, True)
            close(out, o, ao, torch.float32)
            close(d["state"], s, as_, torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strided_views(gpu, dtype, offset):
    """q, k and v as slices of one projection at odd element offsets: the same bits as dense copies."""
    import chunked_sparse_delta_amd as sdm
    P, T, Hk, Hv, K, V = 2, 150, 2, 4, 33, 50
    gen = torch.Generator().manual_seed(offset)
    width = offset + 2 * Hk * K + Hv * V + 3
    fused = torch.randn((P, T, width), generator=gen).to(DT[dtype]).to(gpu)
    q, k, v = (fused[..., a:a + h * w].unflatten(-1, (h, w)) for a, h, w in (
        (offset, Hk, K), (offset + Hk * K, Hk, K), (offset + 2 * Hk * K, Hv, V)))
    g = -torch.rand((Hv,), generator=gen).to(gpu)
    outs = []
    for a in ((k, v, q), tuple(t.contiguous() for t in (k, v, q))):
        final = torch.empty((P, Hv, K, V), device=gpu)
        outs.append((sdm.linear_attention_fwd(None, a[0], a[1], g, a[2], state_out=final), final))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    x = {"q": q.cpu(), "k": k.cpu(), "v": v.cpu(), "log_decay": g.cpu(), "state": None, "valid": None}
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(outs[0][0], o, ao, DT[dtype])
    close(outs[0][1], s, as_, torch.float32)


def test_no_tokens(gpu):
    import chunked_sparse_delta_amd as sdm
    x = on(make(2, 0, 1, 2, 8, 12, torch.float32), gpu)
    for kept in (None, torch.empty(sdm.linear_attention_kept_bytes(2, 0, 1, 2, 8, 12, torch.float32), dtype=torch.uint8, device=gpu)):
        final = torch.full_like(x["state"], math.nan)
        out = sdm.linear_attention_fwd(x["state"], x["k"], x["v"], x["log_decay"], x["q"], state_out=final, kept=kept)
        assert out.shape == (2, 0, 2, 12) and torch.equal(final, x["state"])
    gs = torch.randn_like(x["state"])
    g = sdm.linear_attention_bwd(x["state"], x["k"], x["v"], x["log_decay"], x["q"], out, grad_state=gs)
    assert torch.equal(g["state"], gs) and g["log_decay"].shape == (2, 0, 2)


# ---- single tokens ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,decay", [
    (1, 1, 1, 1, 1, 1, "f32", "token"), (3, 1, 2, 4, 128, 128, "bf16", "head"), (2, 5, 1, 3, 72, 200, "f32", "token"),
    (4, 2, 2, 2, 64, 64, "bf16", "token"), (1, 8, 1, 1, 256, 37, "bf16", "head"), (64, 1, 4, 8, 64, 96, "f32", "head")])
def test_step(gpu, P, T, Hk, Hv, K, V, dtype, decay):
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    x = make(P, T, Hk, Hv, K, V, dt, decay, seed=P + T)
    d = on(x, gpu)
    new = torch.full_like(d["state"], math.nan)
    out = sdm.linear_attention_step(d["state"], d["k"], d["v"], d["log_decay"], d["q"], state_out=new)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(out, o, ao, dt)
    close(new, s, as_, torch.float32)
    assert torch.equal(d["state"].cpu(), x["state"])
    again = sdm.linear_attention_step(d["state"], d["k"], d["v"], d["log_decay"], d["q"])
    assert torch.equal(again, out) and torch.equal(d["state"], new)


def test_step_pool(gpu):
    """Streams on slots of a pool, one idle, one without a valid token; slots that nobody names stay."""
    import chunked_sparse_delta_amd as sdm
    x = make(4, 2, 1, 2, 16, 24, torch.bfloat16, "head", seed=9)
    d = on(x, gpu)
    pool = torch.randn((7, 2, 16, 24), generator=torch.Generator().manual_seed(1))
    ids, valid = torch.tensor([5, -1, 2, 0], dtype=torch.int32), torch.tensor([2, 2, 0, 1], dtype=torch.int32)
    x["state"], x["valid"] = pool[ids.long().clamp(min=0)], torch.where(ids < 0, 0, valid).int()
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    got = pool.to(gpu)
    out = sdm.linear_attention_step(got, d["k"], d["v"], d["log_decay"], d["q"], state_ids=ids.to(gpu), valid_tokens=valid.to(gpu))
    close(out, o, ao, torch.bfloat16)
    for p, i in enumerate(ids.tolist()):
        if i >= 0:
            close(got[i], s[p], as_[p], torch.float32)
    for i in (1, 2, 3, 4, 6):
        assert torch.equal(got[i].cpu(), pool[i])


def test_prompt_then_steps(gpu):
    """A prompt, then its continuation token by token on the same states, is the whole sequence."""
    import chunked_sparse_delta_amd as sdm
    x = make(2, 300, 2, 4, 64, 64, torch.float32, seed=4)
    d = on(x, gpu)
    state = d["state"].clone()
    outs = [sdm.linear_attention_fwd(state, d["k"][:, :270], d["v"][:, :270], d["log_decay"][:, :270].contiguous(), d["q"][:, :270])]
    for t in range(270, 300):
        at = slice(t, t + 1)
        outs.append(sdm.linear_attention_step(state, d["k"][:, at], d["v"][:, at], d["log_decay"][:, at].contiguous(), d["q"][:, at]))
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(torch.cat(outs, 1), o, ao, torch.float32)
    close(state, s, as_, torch.float32)


# ---- gradients -------------------------------------------------------------------------------------------------------

def grads_of(x, go, gs, scale=None, absolute=False):
    """The formula's gradients by autograd through the oracle, or the sums of their terms' sizes."""
    f = {n: None if x[n] is None else x[n].double() for n in NAMES}
    if absolute:
        f = {n: t if t is None or n == "log_decay" else t.abs() for n, t in f.items()}
        go, gs = go.abs(), None if gs is None else gs.abs()
    leaves = {n: t.requires_grad_() for n, t in f.items() if t is not None}
    scale = f["k"].shape[-1] ** -0.5 if scale is None else scale
    out, final = oracle.linear_attention(f["state"], f["k"], f["v"], f["log_decay"], f["q"], abs(scale) if absolute else scale, x["valid"])
    total = (out * go.double()).sum() + (0 if gs is None else (final * gs.double()).sum())
    got = torch.autograd.grad(total, list(leaves.values()), allow_unused=True)
    return {n: torch.zeros_like(t) if g is None else g for (n, t), g in zip(leaves.items(), got)}


def check_grads(got, x, go, gs, dt, scale=None):
    ref, size = grads_of(x, go, gs, scale), grads_of(x, go, gs, scale, True)
    for n in ref:
        if n == "log_decay":
            d = (got[n].double().cpu() - ref[n]).norm()
            assert d <= C * math.sqrt(512) * ref[n].norm() + 1e-30, f"log_decay off by {d / ref[n].norm():.3g}"
        else:
            try:
                close(got[n], ref[n], size[n], torch.float32 if n == "state" else dt)
            except AssertionError as e:
                raise AssertionError(f"{n}: {e}") from None


GRADS = [
    (1, 1, 1, 1, 1, 1, "f32", "token"), (2, 3, 1, 2, 5, 3, "bf16", "head"), (1, 32, 1, 1, 64, 64, "bf16", "token"),
    (1, 33, 2, 4, 40, 72, "f32", "token"), (1, 100, 1, 2, 128, 128, "bf16", "token"), (1, 130, 1, 1, 129, 65, "f32", "head"),
    (1, 256, 1, 3, 64, 130, "bf16", "head"), (1, 257, 2, 2, 128, 128, "f32", "token"), (1, 300, 1, 2, 200, 256, "bf16", "token"),
    (1, 280, 1, 2, 256, 200, "f32", "token"), (2, 540, 1, 1, 32, 16, "f32", "head"),
]


@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,decay", GRADS)
@pytest.mark.parametrize("kept", [True, False])
def test_backward(gpu, P, T, Hk, Hv, K, V, dtype, decay, kept):
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    x = make(P, T, Hk, Hv, K, V, dt, decay, seed=T + 1)
    gen = torch.Generator().manual_seed(T)
    go, gs = torch.randn((P, T, Hv, V), generator=gen).to(dt), torch.randn((P, Hv, K, V), generator=gen)
    d = on(x, gpu)
    buf = None
    if kept:
        buf = torch.empty(sdm.linear_attention_kept_bytes(P, T, Hk, Hv, K, V, dt), dtype=torch.uint8, device=gpu)
        sdm.linear_attention_fwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], state_out=torch.empty_like(d["state"]), kept=buf)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu), kept=buf)
    check_grads(got, x, go, gs, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_backward_ragged(gpu, dtype, decay):
    """Streams of no, one and some valid tokens; NaN in padding, in the readings' gradient there too; zero gradients there."""
    import chunked_sparse_delta_amd as sdm
    dt, counts = DT[dtype], [0, 1, 97, 290, 256]
    x = make(5, 290, 1, 2, 48, 40, dt, decay, ragged=counts, seed=8)
    gen = torch.Generator().manual_seed(2)
    go, gs = torch.randn((5, 290, 2, 40), generator=gen).to(dt), torch.randn((5, 2, 48, 40), generator=gen)
    clean, clean_go = {n: None if t is None else t.clone() for n, t in x.items()}, go.clone()
    for p, n in enumerate(counts):
        go[p, n:] = math.nan
        for name in ("q", "k", "v") + (("log_decay",) if decay == "token" else ()):
            x[name][p, n:] = math.nan
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu),
                                   valid_tokens=d["valid"])
    check_grads(got, clean, clean_go, gs, dt)
    for p, n in enumerate(counts):
        for name in ("q", "k", "v") + (("log_decay",) if decay == "token" else ()):
            assert not got[name][p, n:].any(), name


def test_backward_against_differences(gpu):
    """Central differences of the library's own forward along random directions, float32: the step 2^-6 leaves a third-order
    term for the log-decays alone (everything else is at most quadratic): 1e-3 of the result covers it, and the forward's
    rounding over the step."""
    import chunked_sparse_delta_amd as sdm
    x = on(make(2, 90, 1, 2, 24, 20, torch.float32, seed=11), gpu)
    gen = torch.Generator().manual_seed(5)
    go, gs = (torch.randn(s, generator=gen).to(gpu) for s in ((2, 90, 2, 20), (2, 2, 24, 20)))
    g = sdm.linear_attention_bwd(x["state"], x["k"], x["v"], x["log_decay"], x["q"], go, grad_state=gs)

    def value(y):
        final = torch.empty_like(y["state"])
        out = sdm.linear_attention_fwd(y["state"], y["k"], y["v"], y["log_decay"], y["q"], state_out=final)
        return (out.double() * go).sum() + (final.double() * gs).sum()

    for n in NAMES:
        direction = torch.randn(x[n].shape, generator=gen).to(gpu)
        if n == "log_decay":
            direction = direction * 0.1
        h = 2.0 ** -6
        plus, minus = ({**x, n: x[n] + s * h * direction} for s in (1, -1))
        slope = (value(plus) - value(minus)) / (2 * h)
        exact = (g[n].double() * direction).sum()
        scale = (g[n].double() * direction).norm() * 4
        assert (slope - exact).abs() <= 1e-3 * scale + 1e-3 * exact.abs(), n


@pytest.mark.parametrize("recompute", [False, True])
def test_autograd(gpu, recompute):
    """Gradients reach every input; broadcast and partial uses; a grad of the final state alone; heads that share keys."""
    import chunked_sparse_delta_amd as sdm
    x = make(1, 70, 1, 2, 16, 24, torch.float32, "head", seed=6)
    gen = torch.Generator().manual_seed(6)
    go, gs = torch.randn((1, 70, 2, 24), generator=gen), torch.randn((1, 2, 16, 24), generator=gen)
    for use in ("both", "out", "state"):
        d = {n: t.to(gpu).requires_grad_() for n, t in x.items() if t is not None}
        out, final = sdm.linear_attention(*(d[n] for n in NAMES), recompute=recompute)
        loss = (out * go.to(gpu)).sum() * (use != "state") + (final * gs.to(gpu)).sum() * (use != "out")
        got = dict(zip(NAMES, torch.autograd.grad(loss, [d[n] for n in NAMES])))
        check_grads(got, x, go * (use != "state"), gs * (use != "out"), torch.float32)
    # the output's gradient as an expanded view; only some inputs want one
    d = on(x, gpu)
    d["v"].requires_grad_()
    out, _ = sdm.linear_attention(None, d["k"], d["v"], d["log_decay"], d["q"], recompute=recompute)
    g, = torch.autograd.grad(out.sum(), [d["v"]])
    x["state"] = None
    check_grads({"v": g, **{n: t for n, t in grads_of(x, torch.ones(1, 70, 2, 24), None).items() if n != "v"}}, x,
                torch.ones(1, 70, 2, 24), None, torch.float32)
    with pytest.raises(RuntimeError):     # no second derivative
        d["v"].grad = None
        out, _ = sdm.linear_attention(None, d["k"], d["v"], d["log_decay"], d["q"])
        g, = torch.autograd.grad(out.square().sum(), [d["v"]], create_graph=True)
        g.sum().backward()


# ---- the same bits, streams, graphs ----------------------------------------------------------------------------------

def test_reruns_and_streams(gpu):
    """The same bits from run to run, on another stream, with given or own workspaces; streams of a batch do not matter to
    each other."""
    import chunked_sparse_delta_amd as sdm
    x = on(make(3, 700, 2, 4, 64, 64, torch.bfloat16, seed=2), gpu)
    args = (x["k"], x["v"], x["log_decay"], x["q"])
    first = torch.empty_like(x["state"])
    out = sdm.linear_attention_fwd(x["state"], *args, state_out=first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(first)
    again = sdm.linear_attention_fwd(x["state"], *args, state_out=other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, again) and torch.equal(first, other)
    one = [t[1:2].contiguous() for t in (x["state"], *args)]
    alone = sdm.linear_attention_fwd(*one)
    assert torch.equal(alone[0], out[1]) and torch.equal(one[0][0], first[1])
    go = torch.randn_like(out)
    a, b = (sdm.linear_attention_bwd(x["state"], *args, go) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_graph(gpu):
    """Forward, backward and steps captured together; every replay against the eager result, with eager work between."""
    import chunked_sparse_delta_amd as sdm
    x = on(make(2, 600, 1, 2, 64, 64, torch.bfloat16, seed=13), gpu)
    go = torch.randn((2, 600, 2, 64), device=gpu).to(torch.bfloat16)
    args = (x["k"], x["v"], x["log_decay"], x["q"])
    ws = [torch.empty(sdm.linear_attention_workspace_bytes(2, 600, 1, 2, 64, 64, torch.bfloat16, w), dtype=torch.uint8, device=gpu)
          for w in ("forward", "backward")]
    final = torch.empty_like(x["state"])
    out = torch.empty_like(go)
    step_state = x["state"].clone()
    token = [t[:, :1].contiguous() for t in args]

    def work():
        sdm.linear_attention_fwd(x["state"], *args, state_out=final, out=out, workspace=ws[0])
        g = sdm.linear_attention_bwd(x["state"], *args, go, workspace=ws[1])
        return g, sdm.linear_attention_step(step_state, *token)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, stepped = work()
    start = step_state.clone()
    for i in range(3):
        x["v"].copy_(torch.randn_like(x["v"], dtype=torch.float32))
        step_state.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone(), final.clone(), step_state.clone(), stepped.clone()] + [t.clone() for t in captured.values()]
        step_state.copy_(start)
        g, s = work()
        torch.cuda.synchronize()
        eager = [out, final, step_state, s] + list(g.values())
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), i


def test_refusals(gpu):
    """Shapes, types and devices that do not go together are refused before anything runs."""
    import chunked_sparse_delta_amd as sdm
    x = on(make(1, 5, 1, 2, 8, 12, torch.float32), gpu)
    state, k, v, g, q = (x[n] for n in NAMES)
    bad = [
        ((state, k, v, g[..., :1], q), ValueError), ((state, k, v, g.double(), q), TypeError), ((state, k, v, g, q[:, :4]), ValueError),
        ((state, k, v.bfloat16(), g, q), TypeError), ((state[:, :1], k, v, g, q), ValueError), ((state, k.cpu(), v, g, q), ValueError),
        ((state, k[..., ::2], v, g, q[..., ::2]), ValueError), ((state.bfloat16(), k, v, g, q), TypeError),
        ((state, k, v[:, :, :1], g, torch.cat([q, q], 2)), ValueError)]
    for args, error in bad:
        for call in (sdm.linear_attention_fwd, sdm.linear_attention_step, sdm.linear_attention):
            with pytest.raises(error):
                call(*args)
    with pytest.raises(ValueError):
        sdm.linear_attention_fwd(state, k, v, g, q, kept=torch.empty(16, dtype=torch.uint8, device=gpu))
    with pytest.raises(ValueError):
        sdm.linear_attention_bwd(state, k, v, g, q, v, need=("beta",))
    with pytest.raises(ValueError):
        sdm.linear_attention_bwd(state, k, v, g, q, v[:, :4])
    with pytest.raises(sdm.SdmError):
        sdm.linear_attention_fwd(state, k, v, g, q, state_out=state, workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    with pytest.raises(sdm.SdmError):       # value_dim past 256 for sequences
        wide = torch.zeros(1, 5, 2, 300, device=gpu)
        sdm.linear_attention_fwd(None, k, wide, g, q)
    assert torch.equal(state.cpu(), make(1, 5, 1, 2, 8, 12, torch.float32)["state"])


def test_retained_graph(gpu):
    """The backward may run twice on what the forward kept: it only reads it."""
    import chunked_sparse_delta_amd as sdm
    x = {n: None if t is None else t.to(gpu).requires_grad_() for n, t in make(1, 600, 1, 2, 32, 32, torch.float32).items()}
    out, final = sdm.linear_attention(*(x[n] for n in NAMES))
    loss = out.square().sum() + final.sum()
    a, b = (torch.autograd.grad(loss, [x[n] for n in NAMES], retain_graph=True) for _ in range(2))
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("dtype,T", [(torch.float32, t) for t in (127, 128, 129, 192, 193)] + [(torch.bfloat16, t) for t in (255, 256, 257, 384, 385)])
def test_lengths_around_segments(gpu, dtype, T):
    """One token less and more than the lengths at which segments' number and length change, forward and backward."""
    import chunked_sparse_delta_amd as sdm
    x = make(1, T, 1, 2, 24, 40, dtype, seed=T)
    out, final = want(x)
    size, fsize = want(x, absolute=True)
    d = on(x, gpu)
    state = torch.empty_like(d["state"])
    close(sdm.linear_attention_fwd(*(d[n] for n in NAMES), state_out=state), out, size, dtype)
    close(state, final, fsize, torch.float32)
    gen = torch.Generator().manual_seed(T)
    go, gs = torch.randn((1, T, 2, 40), generator=gen).to(dtype), torch.randn((1, 2, 24, 40), generator=gen)
    got = sdm.linear_attention_bwd(*(d[n] for n in NAMES), go.to(gpu), grad_state=gs.to(gpu))
    check_grads(got, x, go, gs, dtype)


def test_no_grad_keeps_nothing(gpu):
    """Without autograd: the same bits, no graph, and no memory for a backward."""
    import chunked_sparse_delta_amd as sdm
    x = make(4, 100, 8, 8, 128, 128, torch.float32, seed=3)
    x = {n: None if t is None else t.to(gpu).requires_grad_() for n, t in x.items()}
    args = [x[n] for n in NAMES]
    first = [t.detach() for t in sdm.linear_attention(*args)]
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with torch.no_grad():
        got = sdm.linear_attention(*args)
    used = torch.cuda.max_memory_allocated() - before
    assert all(torch.equal(a, b) and not b.requires_grad for a, b in zip(first, got))
    kept = sdm.linear_attention_kept_bytes(4, 100, 8, 8, 128, 128, torch.float32)
    assert used < sum(t.nbytes for t in got) + kept // 2


def test_graph_of_a_training_step(gpu):
    """Linear attention, each head's norm with its activation, and all gradients through autograd, captured together: every replay
    against the eager result."""
    import chunked_sparse_delta_amd as sdm
    x = on(make(2, 300, 2, 4, 64, 64, torch.bfloat16, seed=21), gpu)
    weight = torch.randn(256, device=gpu)
    go = torch.randn(600, 256, device=gpu).to(torch.bfloat16)
    leaves = [x[n].requires_grad_() for n in NAMES] + [weight.requires_grad_()]

    def work():
        out, final = sdm.linear_attention(*leaves[:5])
        y = sdm.group_norm(out.flatten(2).flatten(0, 1), 4, weight, activation="silu")
        return [y.detach(), final.detach(), *torch.autograd.grad(y, leaves, go)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for i in range(3):
        with torch.no_grad():
            x["v"].copy_(torch.randn(x["v"].shape, device=gpu))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, work())), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_terms_that_cancel(gpu, dtype):
    """Readings and gradients whose terms cancel keep float32's bits: every sixteenth value, 2^12 times the others, meets its
    negative one token later with the same key, so that the small ones alone are left."""
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    x = make(1, 128, 1, 1, 64, 64, dt, seed=21)
    x["log_decay"] = torch.zeros(1, 128, 1)
    big = 4096.0 * torch.randn(1, 8, 1, 64, generator=torch.Generator().manual_seed(0))
    x["v"][:, 0::16], x["v"][:, 1::16] = big.to(dt), -big.to(dt)
    x["k"][:, 1::16] = x["k"][:, 0::16]
    out, final = run(gpu, x)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)
    # the bar on what is left, where 16 bits of the large terms would not do: 2^-17 of them is past it
    assert (final.double().cpu() - s).abs().max() <= 2.0 ** -19 * as_.max()


def test_reach_of_an_infinity(gpu):
    """An infinity in a live token's v stays in its column, its stream and its head, and reaches at most the 31 tokens before it
    and those after."""
    x = make(2, 300, 2, 2, 32, 40, torch.bfloat16, seed=17)
    clean, _ = run(gpu, x)
    x["v"][1, 170, 1, 7] = math.inf
    out, final = run(gpu, x)
    same = out == clean
    hit = ~same
    assert not hit[0].any() and not hit[1, :, 0].any() and not hit[1, :139].any()
    hit[1, :, 1, 7] = False
    assert not hit.any()
    assert not torch.isfinite(out[1, 170:, 1, 7]).any() and not torch.isfinite(final[1, 1, :, 7]).any()

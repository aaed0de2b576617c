"""The dense gated delta rule on the GPU (sequences, single tokens, backward) against the token loop in 64 bits
(oracle/dense.py) and its gradients.

Bars, as the 2-norm of the error over that of the result, per output:
  float32 results: 2e-5. An element is a sum of at most head_dim + chunk = 320 products in float32, whose worst relative
    error is 320 * 2^-24 = 1.9e-5 of the terms' size, and errors of different terms do not line up.
  bfloat16 results: 2^-8: the last rounding (at most 2^-9) and as much again for quantities that only reach a bfloat16
    result and are rounded to bfloat16 on the way.
"""

import pytest
import torch

from oracle import dense as oracle

pytestmark = pytest.mark.gpu

BAR = {torch.float32: 2e-5, torch.bfloat16: 2.0 ** -8}
NAMES = ("state", "k", "v", "beta", "log_decay", "q")


def make(P, T, Hk, Hv, K, V, dtype, seed=0, state=True, decay=0.3):
    gen = torch.Generator().manual_seed(seed * 7919 + P + 3 * T + 5 * Hv + 7 * K + 11 * V)

    def randn(*s):
        return torch.randn(s, generator=gen)

    def unit(*s):
        x = randn(*s) + 0.2
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    return dict(state=randn(P, Hv, K, V) if state else None, k=unit(P, T, Hk, K), v=randn(P, T, Hv, V).to(dtype),
                beta=torch.sigmoid(randn(P, T, Hv)), log_decay=-decay * torch.rand((P, T, Hv), generator=gen),
                q=unit(P, T, Hk, K))


def gpu_of(x, dev):
    return {n: None if t is None else t.to(dev) for n, t in x.items()}


def f64_of(x, grad=False):
    return {n: None if t is None else t.double().requires_grad_(grad) for n, t in x.items()}


def close(got, want, what, dtype=None):
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, what
    bar = BAR[dtype or torch.float32]
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), what
    err, norm = (got - want)[fine].norm().item(), want[fine].norm().item()
    assert err <= bar * norm, f"{what}: {err / max(norm, 1e-300):.2e} of the result, bar {bar:.1e}"


# P, T, Hk, Hv, K, V, dtype, valid
CASES = [
    (1, 1, 1, 1, 1, 1, "f32", None), (2, 1, 1, 1, 16, 16, "f32", None), (1, 2, 1, 2, 7, 3, "f32", None),
    (1, 15, 2, 2, 40, 17, "f32", None), (2, 16, 1, 3, 64, 64, "bf16", None), (1, 17, 2, 4, 72, 40, "bf16", None),
    (3, 63, 1, 2, 33, 65, "f32", (0, 1, 63)), (2, 64, 2, 2, 128, 130, "bf16", (64, 33)),
    (1, 65, 1, 1, 128, 16, "f32", None), (2, 130, 2, 4, 96, 72, "bf16", (130, 65)),
    (1, 200, 1, 1, 200, 33, "f32", None), (2, 97, 1, 2, 256, 256, "bf16", (96, 31)),
    (1, 300, 3, 3, 48, 48, "bf16", None), (4, 129, 2, 2, 64, 200, "f32", (129, 128, 64, 0)),
    (1, 1100, 1, 2, 128, 64, "bf16", None),
]
IDS = [f"P{c[0]}-T{c[1]}-H{c[2]}of{c[3]}-K{c[4]}-V{c[5]}-{c[6]}{'' if c[7] is None else '-ragged'}" for c in CASES]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("form", ["fwd", "step"])
@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,valid", CASES, ids=IDS)
def test_forward_matches_oracle(gpu, P, T, Hk, Hv, K, V, dtype, valid, form):
    import chunked_sparse_delta_amd as sdm
    x = make(P, T, Hk, Hv, K, V, DT[dtype])
    y = f64_of(x)
    want, final = oracle.gated_delta(*(y[n] for n in NAMES), K ** -0.5, valid)
    g = gpu_of(x, gpu)
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    start = g["state"].clone()
    other = torch.full_like(start, float("nan"))
    call = sdm.gated_delta_fwd if form == "fwd" else sdm.gated_delta_step
    out = call(*(g[n] for n in NAMES), valid_tokens=vt, state_out=other)
    assert torch.equal(g["state"], start)
    close(out, want, "readings", DT[dtype])
    close(other, final, "state")
    for p in range(P):
        if valid is not None:
            assert (out[p, valid[p]:] == 0).all()
            assert valid[p] > 0 or torch.equal(other[p], start[p])
    again = call(*(g[n] for n in NAMES), valid_tokens=vt)      # in place, the same bits
    assert torch.equal(again, out) and torch.equal(g["state"], other)


@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,valid", CASES, ids=IDS)
def test_backward_matches_oracle(gpu, P, T, Hk, Hv, K, V, dtype, valid):
    import chunked_sparse_delta_amd as sdm
    x = make(P, T, Hk, Hv, K, V, DT[dtype], seed=1)
    gen = torch.Generator().manual_seed(5)
    go = torch.randn((P, T, Hv, V), generator=gen).to(DT[dtype])
    gs = 0.3 * torch.randn((P, Hv, K, V), generator=gen)
    y = f64_of(x, grad=True)
    out, final = oracle.gated_delta(*(y[n] for n in NAMES), K ** -0.5, valid)
    ((out * go.double()).sum() + (final * gs.double()).sum()).backward()
    g = gpu_of(x, gpu)
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    got = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go.to(gpu), grad_state=gs.to(gpu), valid_tokens=vt)
    for n in NAMES:
        assert got[n].dtype == (DT[dtype] if n in "kvq" else torch.float32)
        close(got[n], y[n].grad, n, got[n].dtype)
    again = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go.to(gpu), grad_state=gs.to(gpu), valid_tokens=vt)
    for n in NAMES:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,valid", CASES, ids=IDS)
def test_kept_forward(gpu, P, T, Hk, Hv, K, V, dtype, valid):
    """A forward that keeps what it computed gives the readings to the bar and the backward's own gradients, twice over."""
    import chunked_sparse_delta_amd as sdm
    g = gpu_of(make(P, T, Hk, Hv, K, V, DT[dtype], seed=6), gpu)
    go = torch.randn((P, T, Hv, V), generator=torch.Generator().manual_seed(5)).to(DT[dtype]).to(gpu)
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    ws = torch.full((sdm.gated_delta_workspace_bytes(P, T, Hk, Hv, K, V, DT[dtype], True),), 0xFF, dtype=torch.uint8, device=gpu)
    a, b = torch.empty_like(g["state"]), torch.empty_like(g["state"])
    out = sdm.gated_delta_fwd(*(g[n] for n in NAMES), valid_tokens=vt, state_out=a, workspace=ws, keep=True)
    plain = sdm.gated_delta_fwd(*(g[n] for n in NAMES), valid_tokens=vt, state_out=b)
    close(out, plain.double().cpu(), "readings", DT[dtype])
    close(a, b.double().cpu(), "state")
    want = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go, valid_tokens=vt)
    for _ in range(2):
        got = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go, valid_tokens=vt, kept=ws)
        for n in NAMES:
            assert torch.equal(got[n], want[n]), n


# Few states and many chunks: the forward walks segments of such sequences at once and joins them. A segment's start state is
# one more sum of head_dim products of float32 quantities: within the float32 bar's derivation.
LONG = [
    (1, 1500, 1, 1, 64, 64, "f32", None), (1, 2111, 1, 2, 40, 20, "bf16", None), (2, 1100, 1, 1, 200, 33, "bf16", (1100, 517)),
    (3, 1024, 1, 1, 128, 64, "bf16", (0, 70, 1024)), (2, 700, 1, 1, 128, 128, "f32", (33, 699)),
]


@pytest.mark.parametrize("decay", [0.3, 0.0])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,valid", LONG)
def test_long_sequences_of_few_states(gpu, P, T, Hk, Hv, K, V, dtype, valid, state, decay):
    import chunked_sparse_delta_amd as sdm
    x = make(P, T, Hk, Hv, K, V, DT[dtype], seed=9, state=state, decay=decay)
    y, g = f64_of(x), gpu_of(x, gpu)
    start = y["state"] if state else torch.zeros((P, Hv, K, V), dtype=torch.float64)
    want, final = oracle.gated_delta(start, *(y[n] for n in NAMES[1:]), K ** -0.5, valid)
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    end = torch.full((P, Hv, K, V), float("nan"), device=gpu)
    out = sdm.gated_delta_fwd(*(g[n] for n in NAMES), valid_tokens=vt, state_out=end)
    close(out, want, "readings", DT[dtype])
    close(end, final, "state")
    for p in range(P):
        if valid is not None:
            assert (out[p, valid[p]:] == 0).all()


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(gpu, seed):
    """Every entry point on drawn sizes, types, valid counts, and rows at odd element offsets."""
    import random
    import chunked_sparse_delta_amd as sdm
    rng = random.Random(seed)
    Hk, dt = rng.randint(1, 4), rng.choice([torch.float32, torch.bfloat16])
    P, T, Hv, K, V = rng.randint(1, 4), rng.randint(1, 200), Hk * rng.randint(1, 3), rng.randint(1, 256), rng.randint(1, 150)
    valid = [rng.randint(0, T) for _ in range(P)] if rng.random() < 0.5 else None
    x = make(P, T, Hk, Hv, K, V, dt, seed=seed)
    go = torch.randn((P, T, Hv, V), generator=torch.Generator().manual_seed(seed)).to(dt)
    y, g = f64_of(x, grad=True), gpu_of(x, gpu)
    if rng.random() < 0.5:
        for n in "kvq":     # one element past an aligned address, a token stride that no vector divides
            t = g[n]
            flat = torch.full((t.shape[0], t.shape[1], t[0, 0].numel() + 3), float("nan"), dtype=dt, device=gpu)
            g[n] = flat[..., 1:1 + t[0, 0].numel()].unflatten(2, t.shape[2:]).copy_(t)
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    out, final = oracle.gated_delta(*(y[n] for n in NAMES), K ** -0.5, valid)
    for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        end = torch.empty_like(g["state"])
        close(call(*(g[n] for n in NAMES), valid_tokens=vt, state_out=end), out, "readings", dt)
        close(end, final, "state")
    (out * go.double()).sum().backward()
    got = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go.to(gpu), valid_tokens=vt)
    for n in NAMES:
        close(got[n], y[n].grad, n, got[n].dtype)


def test_rows_past_32_bits(gpu):
    """Streams and heads of q, k and v, and slots of a state pool, further apart than 2^32 elements."""
    import chunked_sparse_delta_amd as sdm
    P, T, H, K, V = 2, 70, 2, 64, 64
    x = make(P, T, H, H, K, V, torch.bfloat16)
    g = gpu_of(x, gpu)
    far = 2 ** 32 + 8
    room = torch.empty(far + 2 ** 21, dtype=torch.bfloat16, device=gpu)
    for n, at, stride in (("q", 0, (far, 2 * K, K)), ("k", 2 ** 19, (2 ** 20, K, far)), ("v", 3 * 2 ** 18, (far, V, 2 ** 16))):
        g[n + "far"] = room.as_strided((P, T, H, K), (*stride, 1), at).copy_(g[n])
    for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        a, b = torch.empty_like(g["state"]), torch.empty_like(g["state"])
        one = call(g["state"], g["k"], g["v"], g["beta"], g["log_decay"], g["q"], state_out=a)
        two = call(g["state"], g["kfar"], g["vfar"], g["beta"], g["log_decay"], g["qfar"], state_out=b)
        assert torch.equal(one, two) and torch.equal(a, b)
    del room, g["qfar"], g["kfar"], g["vfar"]
    slots = 2 ** 32 // (H * K * V) + 2
    pool = torch.empty((slots, H, K, V), device=gpu)
    ids = torch.tensor([slots - 1, 0], dtype=torch.int32, device=gpu)
    pool[slots - 1], pool[0] = g["state"][0], g["state"][1]
    start = g["state"].clone()
    out = sdm.gated_delta_step(pool, *(g[n] for n in NAMES[1:]), state_ids=ids)
    want = sdm.gated_delta_step(start, *(g[n] for n in NAMES[1:]))
    assert torch.equal(out, want) and torch.equal(pool[slots - 1], start[0]) and torch.equal(pool[0], start[1])


def test_graph(gpu):
    """Captured calls replay with the eager calls' bits, other work in between."""
    import chunked_sparse_delta_amd as sdm
    for P, T, K, V, dt in ((1, 600, 64, 64, torch.float32), (2, 130, 40, 24, torch.bfloat16)):
        g = gpu_of(make(P, T, 1, 2, K, V, dt), gpu)
        go = torch.randn((P, T, 2, V), device=gpu).to(dt)
        x = torch.randn((T, 2 * V), device=gpu).to(dt)
        w = torch.randn(2 * V, device=gpu).to(dt)

        def work():
            end = torch.empty_like(g["state"])
            y, mean, rstd = sdm.layer_norm_fwd(x, w)
            return [sdm.gated_delta_fwd(*(g[n] for n in NAMES), state_out=end), end, y,
                    *sdm.layer_norm_bwd(y, x, mean, rstd, w).values(),
                    sdm.gated_delta_step(*(g[n] for n in NAMES), state_out=torch.empty_like(end)),
                    *sdm.gated_delta_bwd(*(g[n] for n in NAMES), go).values()]

        work()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work()
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            got = work()
        for seed in range(3):
            torch.cuda.synchronize()
            new = gpu_of(make(P, T, 1, 2, K, V, dt, seed=seed), gpu)
            for n in NAMES:
                g[n].copy_(new[n])
            want = work()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_state_and_no_tokens(gpu):
    """state=None starts from zeros; T = 0 copies the state and gives an empty result; gradients of no tokens."""
    import chunked_sparse_delta_amd as sdm
    x = make(2, 70, 1, 2, 32, 24, torch.float32, state=False)
    y = f64_of(x)
    want, final = oracle.gated_delta(*(y[n] for n in NAMES), 0.25)
    g = gpu_of(x, gpu)
    end = torch.empty(2, 2, 32, 24, device=gpu)
    close(sdm.gated_delta_fwd(*(g[n] for n in NAMES), scale=0.25, state_out=end), want, "readings")
    close(end, final, "state")
    close(sdm.gated_delta_fwd(*(g[n] for n in NAMES), scale=0.25), want, "readings")
    e = {n: None if t is None else t[:, :0].contiguous() for n, t in g.items()}
    start, moved = torch.randn(2, 2, 32, 24, device=gpu), torch.zeros(2, 2, 32, 24, device=gpu)
    for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        moved.zero_()
        out = call(start, *(e[n] for n in NAMES[1:]), state_out=moved)
        assert out.shape == (2, 0, 2, 24) and torch.equal(moved, start)
    got = sdm.gated_delta_bwd(start, *(e[n] for n in NAMES[1:]), e["v"], grad_state=moved)
    assert torch.equal(got["state"], moved) and got["k"].shape == (2, 0, 1, 32)


def test_rows_of_a_projection_and_head_major(gpu):
    """q, k, v as slices of one projection, and as transposes of head-major tensors: the same bits as their copies."""
    import chunked_sparse_delta_amd as sdm
    P, T, Hk, Hv, K, V = 2, 83, 2, 4, 40, 24
    x = make(P, T, Hk, Hv, K, V, torch.bfloat16)
    g = gpu_of(x, gpu)
    proj = torch.cat([g["q"].flatten(2), g["k"].flatten(2), g["v"].flatten(2), g["v"].flatten(2)[..., :1]], 2)
    a, b = Hk * K, 2 * Hk * K
    views = dict(q=proj[..., :a].unflatten(2, (Hk, K)), k=proj[..., a:b].unflatten(2, (Hk, K)),
                 v=proj[..., b:b + Hv * V].unflatten(2, (Hv, V)))
    heads = {n: g[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"}
    go = torch.randn(P, T, Hv, V, device=gpu).bfloat16()
    base = None
    for form in (g, g | views, g | heads):
        assert form is g or not form["v"].is_contiguous()
        res = []
        for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
            end = torch.empty_like(g["state"])
            res += [call(*(form[n] for n in NAMES), state_out=end), end]
        res += list(sdm.gated_delta_bwd(*(form[n] for n in NAMES), go).values())
        base = base or res
        assert all(torch.equal(p, q) for p, q in zip(res, base))


def test_state_pool(gpu):
    """Streams on named slots of a pool: idle streams (ids outside it) read 0, other slots keep their bits."""
    import chunked_sparse_delta_amd as sdm
    P, T, Hk, Hv, K, V = 5, 2, 1, 2, 72, 36
    x = make(P, T, Hk, Hv, K, V, torch.float32)
    g = gpu_of(x, gpu)
    pool = torch.randn(9, Hv, K, V, device=gpu)
    ids = torch.tensor([7, -1, 0, 9, 3], dtype=torch.int32, device=gpu)
    before = pool.clone()
    out = sdm.gated_delta_step(pool, *(g[n] for n in NAMES[1:]), state_ids=ids)
    y = f64_of(x)
    for p, i in enumerate(ids.tolist()):
        if not 0 <= i < 9:
            assert (out[p] == 0).all()
            continue
        want, final = oracle.gated_delta(before[i:i + 1].double().cpu(), *(y[n][p:p + 1] for n in NAMES[1:]), K ** -0.5)
        close(out[p:p + 1], want, f"readings of stream {p}")
        close(pool[i:i + 1], final, f"slot {i}")
    for i in (1, 2, 4, 5, 6, 8):
        assert torch.equal(pool[i], before[i])


def test_padding_may_hold_anything(gpu):
    """NaN and infinities in padding tokens change nothing, forward or backward."""
    import chunked_sparse_delta_amd as sdm
    P, T = 3, 90
    x = make(P, T, 1, 2, 48, 40, torch.float32)
    g = gpu_of(x, gpu)
    valid = torch.tensor([40, 0, 64], dtype=torch.int32, device=gpu)
    go = torch.randn(P, T, 2, 40, device=gpu)
    dirty = {n: t.clone() for n, t in g.items()}
    dgo = go.clone()
    for p, n in enumerate(valid.tolist()):
        for t in [*(dirty[m] for m in NAMES[1:]), dgo]:
            t[p, n:] = float("nan") if p else float("inf")
    for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        a, b = torch.empty_like(g["state"]), torch.empty_like(g["state"])
        assert torch.equal(call(*(g[n] for n in NAMES), valid_tokens=valid, state_out=a),
                           call(*(dirty[n] for n in NAMES), valid_tokens=valid, state_out=b))
        assert torch.equal(a, b)
    c = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go, valid_tokens=valid)
    d = sdm.gated_delta_bwd(*(dirty[n] for n in NAMES), dgo, valid_tokens=valid)
    for n in NAMES:
        assert torch.equal(c[n], d[n]), n


@pytest.mark.parametrize("kind", ["clear", "steep", "grow", "beta0", "beta_big"])
def test_gates_at_their_ends(gpu, kind):
    """Log-decays of -inf (the state is cleared), of tens per token, above 0; beta of 0, and above 1."""
    import chunked_sparse_delta_amd as sdm
    P, T, Hk, Hv, K, V = 1, 150, 1, 2, 64, 48
    x = make(P, T, Hk, Hv, K, V, torch.float32, seed=3)
    if kind == "clear":
        x["log_decay"][:, ::37] = -float("inf")
        x["log_decay"][:, 60:66] = -float("inf")
    elif kind == "steep":
        x["log_decay"] = x["log_decay"] * 300.0
    elif kind == "grow":
        x["log_decay"] = -x["log_decay"] * 0.1
    elif kind == "beta0":
        x["beta"][:, ::3] = 0.0
        x["beta"][:, 64:] = 0.0
    else:
        x["beta"] = x["beta"] + 0.8
    y = f64_of(x, grad=True)
    want, final = oracle.gated_delta(*(y[n] for n in NAMES), K ** -0.5)
    go = torch.randn((P, T, Hv, V), generator=torch.Generator().manual_seed(1))
    (want * go.double()).sum().backward()
    g = gpu_of(x, gpu)
    for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        end = torch.empty_like(g["state"])
        close(call(*(g[n] for n in NAMES), state_out=end), want, "readings")
        close(end, final, "state")
    got = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go.to(gpu))
    for n in NAMES:
        # exp(-inf) has the gradient 0 times inf in the oracle's exp: the rule's derivative there is 0
        ref = torch.nan_to_num(y[n].grad, nan=0.0) if n == "log_decay" else y[n].grad
        close(got[n], ref, n)


def test_differences(gpu):
    """The gradient along random directions against central differences of the GPU forward (64-bit sums). The step h = 1e-2 of
    inputs of order 1: the curvature's term is about h^2 = 1e-4 of the value, rounding 2^-24 / h = 6e-6 of its terms."""
    import chunked_sparse_delta_amd as sdm
    P, T, Hk, Hv, K, V, h = 2, 100, 1, 2, 32, 48, 1e-2
    g = gpu_of(make(P, T, Hk, Hv, K, V, torch.float32, seed=9), gpu)
    gen = torch.Generator(device=gpu).manual_seed(2)
    go = torch.randn((P, T, Hv, V), generator=gen, device=gpu)
    gs = torch.randn((P, Hv, K, V), generator=gen, device=gpu)
    got = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go, grad_state=gs)

    def J(x):
        end = torch.empty_like(x["state"])
        out = sdm.gated_delta_fwd(*(x[n] for n in NAMES), state_out=end)
        return ((out.double() * go.double()).sum() + (end.double() * gs.double()).sum()).item()

    for n in NAMES:
        # along the gradient itself, so that the directional derivative is its norm and nothing cancels
        u = got[n] / got[n].norm()
        want = (got[n].double() * u.double()).sum().item()
        d = (J(g | {n: g[n] + h * u}) - J(g | {n: g[n] - h * u})) / (2 * h)
        assert abs(d - want) <= 1e-2 * abs(want), (n, d, want)


def test_autograd(gpu):
    """gated_delta_rule: the gradients of gated_delta_bwd, for the inputs that ask, through a view and a later sum."""
    import chunked_sparse_delta_amd as sdm
    g = gpu_of(make(2, 50, 1, 2, 32, 24, torch.float32), gpu)
    for t in g.values():
        t.requires_grad_()
    for recompute in (False, True):
        out, state = sdm.gated_delta_rule(*(g[n] for n in NAMES), recompute=recompute)
        loss = (out.transpose(1, 2) ** 2).sum() + state.sum()
        grads = torch.autograd.grad(loss, [g[n] for n in NAMES])
        with torch.no_grad():
            end = torch.empty_like(state)
            assert torch.equal(out, sdm.gated_delta_fwd(*(g[n] for n in NAMES), state_out=end)) and torch.equal(state, end)
            want = sdm.gated_delta_bwd(*(g[n] for n in NAMES), 2 * out, grad_state=torch.ones_like(state))
        for n, t in zip(NAMES, grads):
            assert torch.equal(t, want[n]), n
    out, _ = sdm.gated_delta_rule(None, *(g[n].detach() for n in NAMES[1:5]), g["q"])
    out.sum().backward()
    assert g["q"].grad is not None and g["k"].grad is None


def test_streams(gpu):
    """The calls run on the stream they are given, in its order."""
    import chunked_sparse_delta_amd as sdm
    g = gpu_of(make(2, 200, 2, 2, 64, 64, torch.bfloat16), gpu)
    base = g["state"].clone()
    want = sdm.gated_delta_fwd(base, *(g[n] for n in NAMES[1:]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = sdm.gated_delta_fwd(g["state"], *(g[n] for n in NAMES[1:]), stream=side)
    tail = sdm.gated_delta_step(g["state"], *(g[n][:, :1].contiguous() for n in NAMES[1:]), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    assert torch.equal(tail, sdm.gated_delta_step(base, *(g[n][:, :1].contiguous() for n in NAMES[1:])))
    assert torch.equal(base, g["state"])


@pytest.mark.parametrize("call", ["fwd", "step", "bwd", "norm_fwd", "norm_bwd"])
def test_memory_of_another_stream(gpu, call):
    """A call on a stream of its own does not get, for its outputs or its workspace, memory that the current stream's work
    still writes."""
    import chunked_sparse_delta_amd as sdm
    P, T, K, V = 2, 150, 64, 64
    g = gpu_of(make(P, T, 1, 2, K, V, torch.float32), gpu)
    x, w = torch.randn(300, 640, device=gpu), torch.randn(640, device=gpu)
    _, mean, rstd = sdm.layer_norm_fwd(x, w)
    side = torch.cuda.Stream()

    def run(**kw):
        args = [g[n] for n in NAMES]
        if call == "norm_fwd":
            return list(sdm.layer_norm_fwd(x, w, **kw))
        if call == "norm_bwd":
            return list(sdm.layer_norm_bwd(x, x, mean, rstd, w, **kw).values())
        if call == "bwd":
            return list(sdm.gated_delta_bwd(*args, g["v"], **kw).values())
        end = torch.zeros_like(g["state"])
        torch.cuda.synchronize()
        return [(sdm.gated_delta_fwd if call == "fwd" else sdm.gated_delta_step)(*args, state_out=end, **kw), end]

    want = run()
    torch.cuda.synchronize()
    sizes = [4096, 2 ** 15, 2 ** 17, 2 ** 18, 2 ** 19, 2 ** 20, 2 ** 22]
    old = [torch.empty(n // 4, device=gpu) for n in sizes for _ in range(6)]
    end = torch.zeros_like(g["state"])
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for t in old:
        t.fill_(7.0)
    del old, t
    if call in ("fwd", "step"):
        got = [(sdm.gated_delta_fwd if call == "fwd" else sdm.gated_delta_step)(*(g[n] for n in NAMES), state_out=end,
                                                                                stream=side), end]
    else:
        got = run(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_second_gradient(gpu):
    """Gradients of the gradients are refused, not silently left out."""
    import chunked_sparse_delta_amd as sdm
    g = gpu_of(make(1, 5, 1, 1, 8, 8, torch.float32), gpu)
    for t in g.values():
        t.requires_grad_()
    out, _ = sdm.gated_delta_rule(*(g[n] for n in NAMES))
    y = sdm.layer_norm(g["v"].detach().requires_grad_())
    for z, t in ((out, g["k"]), (y, y.grad_fn.next_functions[0][0].variable)):
        (first,) = torch.autograd.grad((z ** 2).sum(), t, create_graph=True)
        with pytest.raises(RuntimeError):
            first.sum().backward()


def test_split_sequences(gpu):
    """A sequence cut anywhere, its state handed on, and single tokens after a prompt: the whole sequence's results."""
    import chunked_sparse_delta_amd as sdm
    g = gpu_of(make(1, 140, 1, 2, 64, 32, torch.float32, seed=4), gpu)
    whole, end = g["state"].clone(), None
    want = sdm.gated_delta_fwd(whole, *(g[n] for n in NAMES[1:]))
    state, outs = g["state"].clone(), []
    for a, b, call in ((0, 77, sdm.gated_delta_fwd), (77, 78, sdm.gated_delta_step), (78, 81, sdm.gated_delta_step),
                       (81, 140, sdm.gated_delta_fwd)):
        outs.append(call(state, *(g[n][:, a:b].contiguous() for n in NAMES[1:])))
    close(torch.cat(outs, 1), want.double().cpu(), "readings")
    close(state, whole.double().cpu(), "state")


def test_refusals(gpu):
    import chunked_sparse_delta_amd as sdm
    good = gpu_of(make(2, 8, 1, 2, 32, 24, torch.float32), gpu)

    def call(fn=sdm.gated_delta_fwd, **change):
        x = good | {n: t for n, t in change.items() if n in NAMES}
        return fn(*(x[n] for n in NAMES), **{n: t for n, t in change.items() if n not in NAMES})

    for change, err in [
        (dict(v=good["v"].half()), TypeError), (dict(k=good["k"].bfloat16()), TypeError),
        (dict(q=good["q"][:, :4]), ValueError), (dict(v=good["v"].transpose(2, 3).contiguous().transpose(2, 3)), ValueError),
        (dict(beta=good["beta"].double()), TypeError), (dict(beta=good["beta"].transpose(1, 2)), ValueError),
        (dict(log_decay=good["log_decay"][..., :1]), ValueError), (dict(state=good["state"].bfloat16()), TypeError),
        (dict(state=good["state"][:1]), ValueError), (dict(v=good["v"].cpu()), ValueError),
        (dict(valid_tokens=torch.zeros(2, dtype=torch.int64, device=gpu)), TypeError),
        (dict(out=torch.empty(2, 8, 2, 23, device=gpu)), ValueError),
        (dict(state_out=torch.empty(2, 2, 32, 25, device=gpu)), ValueError),
        (dict(v=good["v"].repeat(1, 1, 2, 1)[:, :, :3], k=good["k"].repeat(1, 1, 2, 1)), ValueError),
    ]:
        with pytest.raises(err):
            call(**change)
    with pytest.raises(sdm.SdmError) as e:
        call(workspace=torch.empty(256, dtype=torch.uint8, device=gpu))
    assert e.value.code == -6
    big = gpu_of(make(1, 4, 1, 1, 257, 8, torch.float32), gpu)
    for fn in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        with pytest.raises(sdm.SdmError) as e:
            fn(*(big[n] for n in NAMES))
        assert e.value.code == -3
    flat = torch.empty(2 * good["state"].numel(), device=gpu)
    half = flat[1:1 + good["state"].numel()].view_as(good["state"])
    with pytest.raises(sdm.SdmError) as e:
        call(state=flat[:good["state"].numel()].view_as(good["state"]), state_out=half)
    assert e.value.code == -2
    with pytest.raises(sdm.SdmError):
        sdm.gated_delta_step(good["state"][:1].clone(), *(good[n] for n in NAMES[1:]))    # 1 state, 2 streams
    with pytest.raises(TypeError):
        call(sdm.gated_delta_step, state_ids=torch.zeros(2, dtype=torch.int64, device=gpu))
    with pytest.raises(ValueError):
        sdm.gated_delta_bwd(*(good[n] for n in NAMES), good["v"][:, :4])

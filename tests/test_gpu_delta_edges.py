"""The gated delta rule on the GPU at the ends of what it takes."""

import pytest
import torch

from oracle import dense as oracle
from tests.test_gpu_delta import NAMES, f64_of, gpu_of, make

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("dtype,K,V", [("f32", 32, 24), ("bf16", 128, 40), ("f32", 200, 70)])
def test_no_tokens_in_training(gpu, dtype, K, V, state):
    """A forward of no tokens that keeps for its backward, and gated_delta_rule: the final state is the start state (zeros without
    one), and its gradient the start state's."""
    import chunked_sparse_delta_amd as sdm
    P, Hk, Hv = 2, 1, 2
    g = {n: None if t is None else t[:, :0].contiguous() if n != "state" else t
         for n, t in gpu_of(make(P, 3, Hk, Hv, K, V, DT[dtype], state=state), gpu).items()}
    start = g["state"] if state else torch.zeros(P, Hv, K, V, device=gpu)
    end = torch.full_like(start, float("nan"))
    ws = torch.empty(sdm.gated_delta_workspace_bytes(P, 0, Hk, Hv, K, V, DT[dtype], True), dtype=torch.uint8, device=gpu)
    out = sdm.gated_delta_fwd(*(g[n] for n in NAMES), state_out=end, workspace=ws, keep=True)
    assert out.shape == (P, 0, Hv, V) and torch.equal(end, start)
    gs = torch.randn_like(start)
    assert torch.equal(sdm.gated_delta_bwd(*(g[n] for n in NAMES), g["v"], grad_state=gs, kept=ws)["state"], gs)
    for recompute in (False, True):
        old = torch.full_like(start, float("nan"))      # what the final state's memory holds if nobody writes it
        del old
        x = {n: None if t is None else t.clone().requires_grad_() for n, t in g.items()}
        out, final = sdm.gated_delta_rule(*(x[n] for n in NAMES), recompute=recompute)
        assert out.shape == (P, 0, Hv, V) and torch.equal(final, start)
        names = [n for n in NAMES if x[n] is not None]
        grads = dict(zip(names, torch.autograd.grad((final * gs).sum(), [x[n] for n in names], allow_unused=True)))
        assert not state or torch.equal(grads["state"], gs)
        assert all(t.shape == x[n].shape for n, t in grads.items())


# Terms that cancel show how many bits an operand had on the way: 24 in float32, where a bfloat16 result is rounded once at its end.
# Two terms of 24 bits and opposite signs that differ by 2^-18 are set against each other, with everything else exact. An
# operand cut to 16 bits is off by up to 2^-17 of the terms, 2^-18 in the mean. In float32 a term carries a rounding of each of its
# factors and of itself, 2^-24 each, and exp's (the decays' argument stays below 1.5: 2^-23): 4 of them line up to 2^-22 at worst.
# The bar is twice that, beside the result's own rounding (2^-8 of it at most).
CANCEL = 2.0 ** -21
SMALL = 2.0 ** -18
WIDTHS = [(64, "bf16"), (128, "bf16"), (200, "bf16"), (64, "f32"), (200, "f32")]


def cancelling(kind, K, dtype):
    """Inputs in float64 (exact in their own types) and for `out`, `q` or `k` the terms' size and where they cancel."""
    gen = torch.Generator().manual_seed(K)
    T, V = 48, 8

    def rand(*s):
        return torch.rand(s, generator=gen)

    sign = torch.where(rand(T, V) < 0.5, -1.0, 1.0)
    v = (sign * (0.5 + rand(T, V))).bfloat16().float()
    beta, g = 0.5 + 0.5 * rand(T), torch.zeros(T)
    k, q = torch.zeros(T, K), torch.zeros(T, K)
    state = torch.zeros(K, V)
    at = torch.arange(T)
    pair = 2 * (rand(T) * ((at + 1) // 2)).long()       # the even one of a pair of tokens up to the token
    pair[0] = 0
    live = at > 0
    go = torch.zeros(T, V)
    if kind == "state":           # out = S_j + S_{j + 1}
        beta = torch.zeros(T)
        state[0::2] = torch.where(rand(K // 2, V) < 0.5, -1.0, 1.0) * (0.5 + rand(K // 2, V))
        state[1::2] = -state[0::2] * (1 + SMALL)
        j = 2 * (rand(T) * (K // 2)).long()
        q[at, j] = q[at, j + 1] = 1.0
        live, terms = at >= 0, 2 * state[j].abs()
    elif kind in ("u", "p"):      # out = P_tj u_j + P_t,j+1 u_{j + 1}
        k[at, at] = 1.0
        q[at, pair] = q[at, pair + 1] = 1.0
        v[1::2] = -v[0::2]
        if kind == "u":
            beta[1::2] = beta[0::2] * (1 + SMALL)
        else:
            beta, g = torch.ones(T), -0.02 * rand(T)
            g[1::2] = -SMALL
        terms = 2 * (beta[:, None] * v)[pair].abs()
    elif kind == "q":             # grad q_t = sum over pairs of (go_t u_j + go_t u_{j + 1}) k_j
        k[at, at // 2 * 2] = 1.0
        beta[1::2] = 1.0
        v[1::2] = SMALL * v[1::2]
        go[at, at % V] = 1.0
        terms = torch.zeros(T, K)
        u = (beta[:, None] * v)[0::2]
        terms[:, 0:T:2] = 2 * (go @ u.abs().T)
        live = torch.arange(K)[None] < at[:, None]      # both tokens of the pair are there
    else:                         # grad k_j = sum over pairs of (go_i D_ij - go_i D_i+1,j) u_j q_i, with q k = 0
        k[at, at // 2] = 1.0
        q[at, 32 + at // 2] = 1.0
        beta, g = torch.ones(T), -0.02 * rand(T)
        k[at, at // 2] = torch.where(at % 2 == 0, 1.0, 0.0)
        beta[0::2] = 0.5 + 0.5 * rand(T // 2)
        g[1::2] = -SMALL
        go[at, at // 2 % V] = torch.where(at % 2 == 0, 1.0, -1.0)
        u = torch.where(at % 2 == 0, beta, torch.ones(()))[:, None] * v
        D = (g.double().cumsum(0)[None, 0::2] - g.double().cumsum(0)[:, None]).exp()
        terms = torch.zeros(T, K)
        terms[:, 32:32 + T // 2] = 2 * (u.abs() @ go[0::2].T) * D
        live = (torch.arange(K)[None] >= 32) & (2 * (torch.arange(K)[None] - 32) >= at[:, None])
    x = dict(state=state[None, None], k=k[None, :, None].to(dtype), v=v[None, :, None].to(dtype), beta=beta[None, :, None],
             log_decay=g[None, :, None], q=q[None, :, None].to(dtype))
    return {n: t.float() if n in ("state", "beta", "log_decay") else t for n, t in x.items()}, go[None, :, None].to(dtype), live, terms


@pytest.mark.parametrize("kind", ["state", "u", "p", "q", "k"])
@pytest.mark.parametrize("K,dtype", WIDTHS)
def test_operands_have_float32s_bits(gpu, K, dtype, kind):
    import chunked_sparse_delta_amd as sdm
    x, go, live, terms = cancelling(kind, K, DT[dtype])
    y, g = f64_of(x, grad=True), gpu_of(x, gpu)
    out, _ = oracle.gated_delta(*(y[n] for n in NAMES), 1.0)
    if kind in ("q", "k"):
        (out * go.double()).sum().backward()
        want = y[kind].grad[0, :, 0]
        got = [sdm.gated_delta_bwd(*(g[n] for n in NAMES), go.to(gpu), scale=1.0)[kind]]
    else:
        want = out.detach()[0, :, 0]
        ws = torch.empty(sdm.gated_delta_workspace_bytes(1, 48, 1, 1, K, 8, DT[dtype], True), dtype=torch.uint8, device=gpu)
        end = torch.empty_like(g["state"])
        got = [sdm.gated_delta_fwd(*(g[n] for n in NAMES), scale=1.0, state_out=end, **kw) for kw in ({}, dict(workspace=ws, keep=True))]
    live = live if live.dim() == 2 else live[:, None].expand_as(want)
    want, terms = want[live], terms.double()[live]
    assert want.norm() < 2.0 ** -15 * terms.norm()       # they do cancel
    for one in got:
        err = (one[0, :, 0].double().cpu()[live] - want).norm()
        assert err <= CANCEL * terms.norm() + 2.0 ** -8 * want.norm(), (err / terms.norm()).item()


@pytest.mark.parametrize("T", [1, 70])
def test_tokens_far_apart(gpu, T):
    """Rows of tokens 2^24 elements and more apart (a time-major array of a large batch), and one token with any stride: the bits of
    dense rows."""
    import chunked_sparse_delta_amd as sdm
    P, H, K, V = 2, 2, 64, 64
    g = gpu_of(make(P, T, H, H, K, V, torch.bfloat16), gpu)
    far = 2 ** 24 + 64
    room = torch.empty(70 * far, dtype=torch.bfloat16, device=gpu)
    f = dict(g)
    for i, n in enumerate("qkv"):
        f[n] = room.as_strided((P, T, H, K), (2 ** 20, far if T > 1 else 2 ** 40, K, 1), i * 2 ** 22).copy_(g[n])
    go = torch.randn((P, T, H, V), device=gpu).bfloat16()
    res = []
    for x in (g, f):
        one = []
        for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
            end = torch.empty_like(g["state"])
            one += [call(*(x[n] for n in NAMES), state_out=end), end]
        res.append(one + list(sdm.gated_delta_bwd(*(x[n] for n in NAMES), go).values()))
    assert all(torch.equal(a, b) for a, b in zip(*res))

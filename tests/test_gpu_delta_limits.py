"""How far the gated delta rule's results are off, and how far an infinity or a NaN reaches."""

import pytest
import torch

from oracle import dense as oracle
from tests.test_gpu_delta import NAMES, f64_of, gpu_of, make

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# Float32 results of inputs whose sums do not cancel, whatever the inputs' type: the roundings of a sum of up to 320 products are
# independent, about sqrt(320) 0.3 2^-24 = 3.2e-7 of it, and a result is at most five such sums deep: 1.6e-6 if all of them lined up.
# The gradients of beta and log_decay are differences of sums about twice their size.
TIGHT = {"state": 2e-6, "out": 2e-6, "k": 2e-6, "v": 2e-6, "q": 2e-6, "beta": 4e-6, "log_decay": 4e-6}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,T,Hk,Hv,K,V", [(1, 300, 2, 4, 128, 64), (2, 97, 1, 2, 64, 48), (1, 200, 1, 1, 200, 33), (1, 1500, 1, 1, 64, 64)])
def test_float32_results(gpu, P, T, Hk, Hv, K, V, dtype):
    import chunked_sparse_delta_amd as sdm
    x = make(P, T, Hk, Hv, K, V, DT[dtype], seed=21)
    gen = torch.Generator().manual_seed(7)
    go = torch.randn((P, T, Hv, V), generator=gen).to(DT[dtype])
    gs = 0.3 * torch.randn((P, Hv, K, V), generator=gen)
    y, g = f64_of(x, grad=True), gpu_of(x, gpu)
    out, final = oracle.gated_delta(*(y[n] for n in NAMES), K ** -0.5)
    ((out * go.double()).sum() + (final * gs.double()).sum()).backward()

    def check(name, got, want):
        if got.dtype == torch.float32:
            want = want.detach()
            err = (got.double().cpu() - want).norm() / want.norm()
            assert err <= TIGHT[name], (name, err.item())

    for call in (sdm.gated_delta_fwd, sdm.gated_delta_step):
        end = torch.empty_like(g["state"])
        check("out", call(*(g[n] for n in NAMES), state_out=end), out)
        check("state", end, final)
    got = sdm.gated_delta_bwd(*(g[n] for n in NAMES), go.to(gpu), grad_state=gs.to(gpu))
    for n in NAMES:
        check(n, got[n], y[n].grad)


# Streams, tokens (the second is long enough for segments), key heads, value heads, widths
BAD = [(2, 200, 2, 4, 72, 40, "f32"), (2, 200, 2, 4, 128, 40, "bf16"), (1, 2200, 2, 2, 64, 24, "bf16")]


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["k", "v", "beta", "log_decay", "q", "state"])
@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype", BAD)
def test_reach_of_what_is_not_finite(gpu, P, T, Hk, Hv, K, V, dtype, name, value):
    """One infinity or NaN in a live token's inputs, or in a state: no other stream, no head that does not read it, no token before
    its chunk changes a bit; in a state or v, no other column."""
    import chunked_sparse_delta_amd as sdm
    C = 64 if dtype == "bf16" and K <= 128 else 32
    p, t, h, col = P - 1, T // 2 + 5, Hv - 1, 3
    g = gpu_of(make(P, T, Hk, Hv, K, V, DT[dtype], seed=22), gpu)
    bad = {n: x.clone() for n, x in g.items()}
    where = {"k": (p, t, Hk - 1, 1), "q": (p, t, Hk - 1, 1), "v": (p, t, h, col), "state": (p, h, 1, col)}.get(name, (p, t, h))
    bad[name][where] = value
    group = Hv // Hk
    heads = slice(Hv - group, Hv) if name in "kq" else slice(h, h + 1)      # those that read it
    columns = slice(col, col + 1) if name in ("v", "state") else slice(0, V)
    first = {"step": t, "fwd": t // C * C}
    for form, call in (("fwd", sdm.gated_delta_fwd), ("step", sdm.gated_delta_step)):
        ends = [torch.empty_like(g["state"]) for _ in range(2)]
        outs = [call(*(x[n] for n in NAMES), state_out=e) for x, e in zip((g, bad), ends)]
        reach = torch.zeros_like(outs[0], dtype=torch.bool)
        reach[p, 0 if name == "state" else first[form]:, heads, columns] = True
        assert torch.equal(outs[0][~reach], outs[1][~reach])
        reach = torch.zeros_like(ends[0], dtype=torch.bool)
        if name != "q":
            reach[p, heads, :, columns] = True
        assert torch.equal(ends[0][~reach], ends[1][~reach])
        assert not torch.isfinite(outs[1][p, t, h, col])
    go = torch.randn((P, T, Hv, V), device=gpu).to(DT[dtype])
    want, got = (sdm.gated_delta_bwd(*(x[n] for n in NAMES), go) for x in (g, bad))
    for n in NAMES:
        a, b = want[n].clone(), got[n].clone()
        for x in (a, b):
            x[p, heads if n == "state" else slice(None), slice(Hk - 1, Hk) if n in "kq" else slice(None) if n == "state" else heads] = 0
        assert torch.equal(a, b), n

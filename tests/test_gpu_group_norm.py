"""Group norm with an activation on the GPU against its definition in 64 bits (oracle/linear.py).

Bars. u = 2^-24. A thread adds up to about 64 values (its rows, the joins), each addition u of the terms: the mean and the
variance are right to 64 u of the terms' sizes, so xh = (x - mean) rstd is off by at most 64 u of s = (|x| + |mean|) rstd,
z = xh w + b by e = 64 u (s |w| + |b|), and act(z), whose slope is at most 1.2, by 1.2 e + 16 u |z|. The slope itself bends by at
most 1: dz = dy act'(z) is off by |dy| (e + 16 u); the sums over rows and channels add 64 u of their terms, more than 64
rows one after another in a join over samples 256 u. On top a result is rounded by half a step: 2^-8 of a bfloat16 value, u of a
float32 one.
"""

import math

import pytest
import torch

from oracle import linear as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(N, L, C, dtype, wdtype=None, seed=0, mean=1.0):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=gen)

    wdtype = wdtype or dtype
    return {"x": (2 * randn(N, L, C) + mean * randn(N, 1, C)).to(dtype), "weight": (1 + 0.3 * randn(C)).to(wdtype),
            "bias": (0.3 * randn(C)).to(wdtype), "go": randn(N, L, C).to(dtype)}



def bars(x, G, w, b, act, go, valid, eps=1e-5):
    """References and bars: dict name -> (value, bar without the last rounding)."""
    N, L, C = x.shape
    D = C // G
    x, go = x.double(), go.double()
    w1, b1 = (None if t is None else t.double() for t in (w, b))
    w_, b_ = (torch.ones(C, dtype=torch.float64) if w is None else w1), (torch.zeros(C, dtype=torch.float64) if b is None else b1)
    counts = [L if valid is None else max(0, min(int(v), L)) for v in (valid if valid is not None else [L] * N)]
    live = (torch.arange(L) < torch.tensor(counts)[:, None])[:, :, None]
    x, go = torch.where(live, x, 0.0), torch.where(live, go, 0.0)
    xr = x.clone().requires_grad_()
    wr, br = w_.clone().requires_grad_(), b_.clone().requires_grad_()
    y, mean, rstd = oracle.group_norm(xr, G, wr, br, act, eps, counts)
    dx, dw, db = torch.autograd.grad((y * go).sum(), [xr, wr, br], allow_unused=True)
    y, mean, rstd = y.detach(), mean.detach(), rstd.detach()

    def spread(t):
        return t.repeat_interleave(D, 1)[:, None]

    def per_group(t):     # the mean over a sample's group's valid elements
        c = torch.tensor(counts).clamp(min=1).double()[:, None] * D
        return spread(t.reshape(N, L, G, D).sum((1, 3)) / c)

    m, r = spread(mean), spread(rstd)
    xh = torch.where(live, (x - m) * r, 0.0)
    z = xh * w_ + b_
    s = (x.abs() + m.abs()) * r
    e = 64 * U * (s * w_.abs() + b_.abs())
    if act == "silu":
        sg = torch.sigmoid(z)
        slope = sg * (1 + z * (1 - sg))
    elif act == "gelu":
        slope = 0.5 * torch.erfc(-z * 0.5 ** 0.5) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        slope = torch.ones_like(z)
    dz, dz_e = (go * slope).abs(), go.abs() * (e + 16 * U)
    h, h_e = dz * w_.abs(), dz_e * w_.abs()
    xa, x_e = xh.abs(), 64 * U * s
    size = r * (h + per_group(h) + xa * per_group(h * xa))
    dx_bar = r * (h_e + per_group(h_e) + xa * per_group(h_e * xa + h * x_e) + x_e * per_group(h * xa)) + 256 * U * size
    out = {"y": (y, 1.2 * e + 16 * U * z.abs()),
           "mean": (mean, 64 * U * (x.abs().reshape(N, L, G, D).sum((1, 3)) / torch.tensor(counts).clamp(min=1).double()[:, None] / D)),
           "rstd": (rstd, 64 * U * rstd * (1 + mean ** 2 * rstd ** 2)),
           "grad_x": (torch.where(live, dx, 0.0), dx_bar),
           "grad_weight": (dw, (dz_e * xa + dz * x_e + 256 * U * dz * xa).sum((0, 1))),
           "grad_bias": (db, (dz_e + 256 * U * dz).sum((0, 1)))}
    return {n: (torch.zeros_like(bar) if v is None else v, bar) for n, (v, bar) in out.items()}


def close(got, ref, dtype, name):
    value, bar = ref
    got = got.double().cpu()
    assert got.shape == value.shape, name
    bar = bar + HALF[dtype] * (value.abs() + bar) + 1e-38
    bad = ~((got - value).abs() <= bar)
    assert not bad.any(), f"{name}: {int(bad.sum())} over the bar, worst {((got - value).abs() / bar).max():.3g} times"


def check(gpu, N, L, C, G, dtype, act, wdtype=None, valid=None, seed=0, params="wb", mean=1.0, poison=False):
    import chunked_sparse_delta_amd as sdm
    dt, wdt = DT[dtype], DT[wdtype or dtype]
    d = make(N, L, C, dt, wdt, seed, mean)
    w, b = d["weight"] if "w" in params else None, d["bias"] if "b" in params else None
    ref = bars(d["x"], G, w, b, act, d["go"], valid)
    x, go = d["x"].clone(), d["go"].clone()
    if poison:
        for n, v in enumerate(valid):
            x[n, max(0, v):], go[n, max(0, v):] = math.nan, math.inf
    x, go, w, b = (None if t is None else t.to(gpu) for t in (x, go, w, b))
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    kw = {"activation": act, "valid_rows": vt}
    y, m, r = sdm.group_norm_fwd(x, G, w, b, **kw)
    close(m, ref["mean"], torch.float32, "mean")
    close(r, ref["rstd"], torch.float32, "rstd")
    close(y, ref["y"], dt, "y")
    g = sdm.group_norm_bwd(go, x, G, m, r, w, b, **kw)
    pdt = dt if w is None and b is None else wdt
    assert g["weight"].dtype == g["bias"].dtype == pdt
    close(g["x"], ref["grad_x"], dt, "grad_x")
    close(g["weight"], ref["grad_weight"], pdt, "grad_weight")
    close(g["bias"], ref["grad_bias"], pdt, "grad_bias")
    if valid is not None:
        for n, v in enumerate(valid):
            assert not y[n, max(0, v):].any() and not g["x"][n, max(0, v):].any()
    return y, g


SHAPES = [
    # N, L, C, G: groups of one lane to several wavefronts, of widths no vector divides, one row to thousands
    (1, 1, 1, 1), (3, 1, 4096, 32), (5, 1, 64, 64), (2, 1, 10, 5), (70, 1, 128, 2), (4097, 1, 64, 4), (3, 1, 512, 1), (3, 1, 2048, 1),
    (4, 3, 48, 4), (2, 7, 320, 32), (3, 50, 24, 2), (9, 16, 512, 16), (2, 300, 64, 4), (3, 2, 96, 2), (2, 1, 4096, 1), (2, 3, 8192, 1),
    (33, 1, 2056, 1), (2, 2, 16384, 2),
    # in blocks of rows: many rows, groups wider than a workgroup, odd ones
    (1, 2500, 40, 8), (2, 4100, 16, 1), (2, 1200, 96, 32), (2, 1, 9000, 1), (2, 5, 2100, 1), (1, 3, 20001, 3), (3, 777, 1000, 8), (1, 9001, 7, 7),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,C,G", SHAPES)
def test_matches_definition(gpu, N, L, C, G, dtype):
    check(gpu, N, L, C, G, dtype, ("silu", "gelu", None)[(N + L + C) % 3], seed=N + L + C)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("N,L,C,G", [(3, 1, 256, 4), (2, 40, 72, 6), (2, 3000, 32, 4)])
def test_parameters(gpu, N, L, C, G, act):
    """bfloat16 rows with float32 parameters, with the weight alone, the bias alone, with none."""
    check(gpu, N, L, C, G, "bf16", act, wdtype="f32")
    for params in ("w", "b", ""):
        check(gpu, N, L, C, G, "f32", act, params=params)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,C,G", [(1, 64, 4), (5, 64, 2), (130, 48, 16), (3000, 32, 4), (700, 640, 32)])
def test_ragged_padding_may_hold_anything(gpu, L, C, G, dtype):
    counts = [0, 1, L, L // 2, (L + 1) // 2]
    check(gpu, 5, L, C, G, dtype, "silu", valid=counts, poison=True)
    check(gpu, 1, L, C, G, dtype, None, valid=[0], poison=True)


@pytest.mark.parametrize("N,L,C,G", [(2, 1, 512, 4), (2, 20, 64, 4), (2, 4000, 24, 3)])
def test_large_means(gpu, N, L, C, G):
    """Means a thousand times the spread: the bars grow with them, and hold."""
    check(gpu, N, L, C, G, "f32", "silu", mean=2000.0)


def test_constant_rows(gpu):
    """No spread at all: y is the bias, the gradient that of eps alone."""
    import chunked_sparse_delta_amd as sdm
    x = torch.full((2, 40, 64), 3.0, device=gpu)
    b = torch.randn(64, device=gpu)
    y, m, r = sdm.group_norm_fwd(x, 4, None, b)
    assert torch.equal(y, b.expand_as(y)) and torch.equal(m, torch.full_like(m, 3.0))
    assert torch.allclose(r, torch.full_like(r, 1e5 ** 0.5), rtol=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,C,G", [(1, 256, 2), (37, 33, 11), (5000, 24, 2)])
def test_views(gpu, L, C, G, dtype):
    """x as a slice of a wider array at odd offsets: the same bits as a dense copy; [N, H, W, C] and [N, C] shapes."""
    import chunked_sparse_delta_amd as sdm
    wide = torch.randn((3, L, C + 7), device=gpu).to(DT[dtype])
    x = wide[..., 3:3 + C]
    go = torch.randn((3, L, C), device=gpu).to(DT[dtype])
    a, b = sdm.group_norm_fwd(x, G, activation="silu"), sdm.group_norm_fwd(x.contiguous(), G, activation="silu")
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    ga, gb = (sdm.group_norm_bwd(go, t, G, a[1], a[2], activation="silu") for t in (x, x.contiguous()))
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    if L % 5 == 0:
        four = sdm.group_norm_fwd(x.contiguous().view(3, L // 5, 5, C), G, activation="silu")
        assert torch.equal(four[0].view(3, L, C), a[0])
    if L == 1:
        assert torch.equal(sdm.group_norm_fwd(x[:, 0], G, activation="silu")[0], a[0][:, 0])


def test_no_rows(gpu):
    import chunked_sparse_delta_amd as sdm
    w = torch.ones(8, device=gpu)
    y, m, r = sdm.group_norm_fwd(torch.empty((3, 0, 8), device=gpu), 2, w, w)
    assert y.shape == (3, 0, 8) and not m.any() and torch.allclose(r, torch.full_like(r, 1e5 ** 0.5), rtol=1e-6)
    g = sdm.group_norm_bwd(y, y, 2, m, r, w, w)
    assert not g["weight"].any() and not g["bias"].any()
    y, m, r = sdm.group_norm_fwd(torch.empty((0, 5, 8), device=gpu), 2, w, w)
    assert y.shape == (0, 5, 8) and m.shape == (0, 2)
    g = sdm.group_norm_bwd(y, y, 2, m, r, w, w)
    assert not g["weight"].any() and not g["bias"].any()
    y, m, r = sdm.group_norm_fwd(torch.empty((2, 0, 3, 8), device=gpu), 2, w, w)
    assert y.shape == (2, 0, 3, 8)


@pytest.mark.parametrize("N,L,C,G", [(4, 1, 96, 3), (2, 30, 40, 4), (2, 3000, 16, 2)])
def test_against_differences(gpu, N, L, C, G):
    """Central differences of the library's own forward along random directions, step 2^-7: the third-order term and the
    forward's float32 rounding over the step stay below 1e-3 of the gradient's norm along them."""
    import chunked_sparse_delta_amd as sdm
    d = {n: t.to(gpu) for n, t in make(N, L, C, torch.float32, seed=3).items()}
    for act in ("silu", "gelu"):
        leaves = {n: d[n].clone().requires_grad_() for n in ("x", "weight", "bias")}
        y = sdm.group_norm(leaves["x"], G, leaves["weight"], leaves["bias"], activation=act)
        grads = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), d["go"])))
        gen = torch.Generator().manual_seed(1)
        for n in leaves:
            u = torch.randn(d[n].shape, generator=gen).to(gpu)
            h = 2.0 ** -7
            value = [sdm.group_norm_fwd(*[(d[m] + s * h * u) if m == n else d[m] for m in ("x",)], G,
                                        *[(d[m] + s * h * u) if m == n else d[m] for m in ("weight", "bias")], activation=act)[0]
                     for s in (1, -1)]
            slope = ((value[0].double() - value[1].double()) * d["go"].double()).sum() / (2 * h)
            exact = (grads[n].double() * u).sum()
            assert (slope - exact).abs() <= 1e-3 * (grads[n].double() * u).norm() * 4 + 1e-3 * exact.abs(), (act, n)


def test_autograd_partial_needs(gpu):
    import chunked_sparse_delta_amd as sdm
    d = {n: t.to(gpu) for n, t in make(3, 4, 32, torch.float32).items()}
    full = None
    for need in (("x", "weight", "bias"), ("x",), ("weight",), ("bias", "x")):
        t = {n: d[n].clone().requires_grad_(n in need) for n in ("x", "weight", "bias")}
        y = sdm.group_norm(t["x"], 4, t["weight"], t["bias"], activation="gelu")
        g = dict(zip(need, torch.autograd.grad(y.sum() * 2, [t[n] for n in need])))     # an expanded gradient
        full = full or g
        assert all(torch.equal(g[n], full[n]) for n in need)
    x = d["x"].clone().requires_grad_()
    with pytest.raises(RuntimeError):     # no second derivative
        g, = torch.autograd.grad(sdm.group_norm(x, 4).square().sum(), [x], create_graph=True)
        g.sum().backward()


@pytest.mark.parametrize("N,L,C,G", [(40, 1, 256, 4), (2, 2500, 64, 8)])
def test_streams_and_graph(gpu, N, L, C, G):
    """The same bits on another stream; forward and backward captured, every replay against the eager result."""
    import chunked_sparse_delta_amd as sdm
    d = {n: t.to(gpu) for n, t in make(N, L, C, torch.bfloat16).items()}
    args = (G, d["weight"], d["bias"])

    def work(stream=None):
        y, m, r = sdm.group_norm_fwd(d["x"], *args, activation="silu", stream=stream)
        g = sdm.group_norm_bwd(d["go"], d["x"], G, m, r, *args[1:], activation="silu", stream=stream)
        return [y, m, r, *g.values()]

    first = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = work(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for i in range(3):
        d["x"].copy_(torch.randn_like(d["x"], dtype=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, work())), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,C,G", [(40, 1, 256, 4), (6, 5, 320, 2), (9, 3, 21, 3), (2, 2500, 64, 8)])
def test_in_place(gpu, N, L, C, G, dtype):
    """y in x's place: the same bits."""
    import chunked_sparse_delta_amd as sdm
    d = {n: t.to(gpu) for n, t in make(N, L, C, DT[dtype]).items()}
    kw = {"activation": "silu"}
    first = sdm.group_norm_fwd(d["x"], G, d["weight"], d["bias"], **kw)
    got = sdm.group_norm_fwd(d["x"], G, d["weight"], d["bias"], out=d["x"], **kw)
    assert got[0].data_ptr() == d["x"].data_ptr() and all(torch.equal(a, b) for a, b in zip(first, got))

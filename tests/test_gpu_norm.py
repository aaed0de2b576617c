"""Layer norm on the GPU, forward and backward, against its definition in 64 bits (oracle/dense.py).

Bars, as the 2-norm of the error over that of the result, per output: float32 results 4e-6 (sums of up to 2^16 terms in
float32 as a tree of at most 8 * 8 serial additions per lane and 10 levels, (64 + 10 + a few) 2^-24 = 4.7e-6 at worst,
gradient sums over rows likewise); bfloat16 results 2^-8 * 0.6 (one rounding, at most 2^-9, and the float32 bar).
The gradient of x is a difference that can be far smaller than its terms: with two columns it is eps rstd^2 of them,
2e-6 at a spread of 2, and mean and rstd, which are float32, alone are off by 2^-24 of the terms. Its float32 bar is
therefore one of its terms' norm."""

import pytest
import torch

from oracle import dense as oracle

pytestmark = pytest.mark.gpu

BAR = {torch.float32: 4e-6, torch.bfloat16: 0.6 * 2.0 ** -8}

SHAPES = [(1, 1), (3, 2), (5, 7), (1, 63), (4, 64), (6, 65), (9, 255), (130, 256), (7, 511), (5, 512), (6, 1000),
          (3, 1025), (700, 1024), (2, 2048), (3, 4095), (1030, 4096), (2, 8191), (3, 8192), (2, 16384), (3, 16387),
          (2, 32768), (2, 40001), (1, 65539)]


def make(rows, N, dtype, wdtype, seed=0, shift=3.0):
    gen = torch.Generator().manual_seed(seed + rows * 31 + N)

    def randn(*s):
        return torch.randn(s, generator=gen)

    return ((2 * randn(rows, N) + shift * randn(rows, 1)).to(dtype), (1 + 0.3 * randn(N)).to(wdtype),
            (0.5 * randn(N)).to(wdtype), randn(rows, N).to(dtype))


def check(got, want, what, terms=None):
    bar, dtype = BAR[got.dtype], got.dtype
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, what
    err, most = (got - want).norm().item(), bar * want.norm().item()
    if terms is not None:
        most = BAR[torch.float32] * terms.norm().item() + (most if dtype == torch.bfloat16 else 0.0)
    assert err <= most, f"{what}: {err:.2e}, at most {most:.2e}"


def x_terms(x, w, dy, eps=1e-5):
    """The size of the terms of the gradient of x: rstd (|h| + |mean h| + |xh mean(h xh)|)."""
    x, dy = x.double(), dy.double()
    _, mean, rstd = oracle.layer_norm(x, eps=eps)
    xh, h = (x - mean[:, None]) * rstd[:, None], dy if w is None else dy * w.double()
    return rstd[:, None] * (h.abs() + h.mean(1, keepdim=True).abs() + (xh * (h * xh).mean(1, keepdim=True)).abs())


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,N", SHAPES)
def test_matches_oracle(gpu, rows, N, dtype, wdtype):
    import chunked_sparse_delta_amd as sdm
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    x, w, b, dy = make(rows, N, dt[dtype], dt[wdtype])
    X, W, B = (t.double().requires_grad_() for t in (x, w, b))
    y, mean, rstd = oracle.layer_norm(X, W, B, 1e-5)
    # a row of one column is its own mean: y is the bias and the gradients of x and the weight are 0
    (y * dy.double()).sum().backward()
    g = [t.to(gpu) for t in (x, w, b, dy)]
    gy, gm, gr = sdm.layer_norm_fwd(g[0], g[1], g[2])
    check(gy, y, "y")
    check(gm, mean, "mean")
    check(gr, rstd, "rstd")
    got = sdm.layer_norm_bwd(g[3], g[0], gm, gr, g[1])
    if N == 1:
        assert (got["x"] == 0).all() and (got["weight"] == 0).all()
        check(got["bias"], B.grad, "grad bias")
    else:
        check(got["x"], X.grad, "grad x", x_terms(x, w, dy))
        check(got["weight"], W.grad, "grad weight")
        check(got["bias"], B.grad, "grad bias")
    again = sdm.layer_norm_bwd(g[3], g[0], gm, gr, g[1])
    assert all(torch.equal(got[n], again[n]) for n in got)


def test_without_parameters_and_parts(gpu):
    import chunked_sparse_delta_amd as sdm
    x, w, b, dy = make(50, 300, torch.float32, torch.float32)
    X = x.double().requires_grad_()
    y, _, _ = oracle.layer_norm(X)
    (y * dy.double()).sum().backward()
    xg, wg, bg, dg = (t.to(gpu) for t in (x, w, b, dy))
    got, mean, rstd = sdm.layer_norm_fwd(xg)
    check(got, y, "y")
    g = sdm.layer_norm_bwd(dg, xg, mean, rstd, need=("x",))
    assert set(g) == {"x"}
    check(g["x"], X.grad, "grad x", x_terms(x, None, dy))
    full = sdm.layer_norm_bwd(dg, xg, mean, rstd, wg)
    for part in (("weight",), ("bias",), ("x", "bias")):
        some = sdm.layer_norm_bwd(dg, xg, mean, rstd, wg, need=part)
        assert set(some) == set(part) and all(torch.equal(some[n], full[n]) for n in part)
    check(sdm.layer_norm_fwd(xg, None, bg)[0], y + b.double(), "y")
    check(sdm.layer_norm_fwd(xg, wg, None)[0], y * w.double(), "y")


def test_shapes_and_no_rows(gpu):
    import chunked_sparse_delta_amd as sdm
    x, w, b, dy = (t.to(gpu) for t in make(12, 40, torch.bfloat16, torch.float32))
    y, mean, rstd = sdm.layer_norm_fwd(x, w, b)
    z, _, _ = sdm.layer_norm_fwd(x.view(3, 2, 2, 40), w, b)
    assert z.shape == (3, 2, 2, 40) and torch.equal(z.view(12, 40), y)
    e, m, r = sdm.layer_norm_fwd(x[:0], w, b)
    assert e.shape == (0, 40) and m.shape == (0,)
    g = sdm.layer_norm_bwd(dy[:0], x[:0], m, r, w)
    assert g["x"].shape == (0, 40) and (g["weight"] == 0).all() and (g["bias"] == 0).all()


def test_large_mean_and_special_rows(gpu):
    """A mean 1e3 times the spread costs no more than x's own rounding; a constant row gives the bias; a row with an
    infinity or NaN is NaN and no other row is."""
    import chunked_sparse_delta_amd as sdm
    x, w, b, _ = make(8, 777, torch.float32, torch.float32)
    x = x + 1000.0
    x[3] = 2.5
    y, mean, rstd = oracle.layer_norm(x.double(), w.double(), b.double())
    got, gm, gr = sdm.layer_norm_fwd(x.to(gpu), w.to(gpu), b.to(gpu))
    assert torch.equal(got[3].cpu(), b)
    # the mean's own rounding (2^-24 of 1000, against a spread of 2): 3e-5 of every difference
    assert (got.double().cpu() - y).norm() <= 4e-5 * y.norm()
    x[1, 5], x[6, 700] = float("inf"), float("nan")
    bad = sdm.layer_norm_fwd(x.to(gpu), w.to(gpu), b.to(gpu))[0]
    assert torch.isnan(bad[1]).all() and torch.isnan(bad[6]).all()
    keep = [0, 2, 3, 4, 5, 7]
    assert torch.equal(bad[keep], got[keep])


def test_autograd_and_differences(gpu):
    """layer_norm's gradients are layer_norm_bwd's, and agree with central differences along the gradient (step 1e-2:
    curvature 1e-4 of the value)."""
    import chunked_sparse_delta_amd as sdm
    x, w, b, dy = (t.to(gpu) for t in make(20, 130, torch.float32, torch.float32))
    p = [t.clone().requires_grad_() for t in (x, w, b)]
    grads = torch.autograd.grad(sdm.layer_norm(*p), p, dy)
    _, mean, rstd = sdm.layer_norm_fwd(x, w, b)
    want = sdm.layer_norm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(g, want[n]) for g, n in zip(grads, ("x", "weight", "bias")))
    h = 1e-2
    for i, g in enumerate(grads):
        u = g / g.norm()
        args = [x, w, b]
        ends = []
        for s in (h, -h):
            args[i] = (x, w, b)[i] + s * u
            ends.append((sdm.layer_norm_fwd(*args)[0].double() * dy.double()).sum().item())
        d = (ends[0] - ends[1]) / (2 * h)
        assert abs(d - g.norm().item()) <= 1e-2 * g.norm().item()
    only = w.clone().requires_grad_()
    sdm.layer_norm(x, only, b).sum().backward()
    assert only.grad is not None


def test_stream(gpu):
    import chunked_sparse_delta_amd as sdm
    x, w, b, dy = (t.to(gpu) for t in make(300, 1024, torch.bfloat16, torch.bfloat16))
    y, mean, rstd = sdm.layer_norm_fwd(x, w, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z, m, r = sdm.layer_norm_fwd(x, w, b, stream=side)
    g = sdm.layer_norm_bwd(dy, x, m, r, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, z)
    f = sdm.layer_norm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(f[n], g[n]) for n in f)


def test_refusals(gpu):
    import chunked_sparse_delta_amd as sdm
    x, w, b, dy = (t.to(gpu) for t in make(4, 32, torch.float32, torch.float32))
    _, mean, rstd = sdm.layer_norm_fwd(x, w, b)
    for args, err in [((x.half(), None, None), TypeError), ((x.cpu(), None, None), ValueError), ((x.t(), None, None), ValueError),
                      ((x, w[:31], None), ValueError), ((x, w.double(), None), TypeError), ((x, w, b.bfloat16()), TypeError)]:
        with pytest.raises(err):
            sdm.layer_norm_fwd(*args)
    with pytest.raises(sdm.SdmError) as e:
        sdm.layer_norm_fwd(x, w.bfloat16(), b.bfloat16())       # float32 rows with bfloat16 parameters
    assert e.value.code == -1
    with pytest.raises(sdm.SdmError) as e:
        sdm.layer_norm_fwd(x, w, b, eps=-1.0)
    assert e.value.code == -3
    with pytest.raises(ValueError):
        sdm.layer_norm_bwd(dy, x, mean[:3], rstd, w)
    with pytest.raises(ValueError):
        sdm.layer_norm_bwd(dy[:3], x, mean, rstd, w)
    with pytest.raises(ValueError):
        sdm.layer_norm_bwd(dy, x, mean, rstd, w, need=("y",))
    with pytest.raises(sdm.SdmError) as e:
        sdm.layer_norm_bwd(dy, x, mean, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    assert e.value.code == -6

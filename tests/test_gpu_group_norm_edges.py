"""Group norm on the GPU where its sums cancel and where values end, against its definition in 64 bits: bars and helpers of
test_gpu_group_norm.py."""

import math

import pytest
import torch

from tests.test_gpu_group_norm import DT, U, bars, check, close, make

pytestmark = pytest.mark.gpu

# Every way in which a tile's threads meet (test_gpu_group_norm.py names them by their shapes), and blocks of rows: D divided by
# vectors of a power of two, by others, by none; groups wider than a workgroup.
FORMS = [(70, 1, 128, 2), (9, 16, 512, 16), (3, 1, 2048, 1), (2, 7, 320, 32), (2, 3000, 32, 4), (1, 3, 20001, 3), (3, 777, 1000, 8)]


@pytest.mark.parametrize("N,L,C,G", FORMS)
def test_means_far_from_zero(gpu, N, L, C, G):
    """Means a thousand times the spread, of each sample and group its own. With u = 2^-24 and r = |mean| rstd: a mean is right to
    64 u of itself, so a difference from it, or of two of them, to 64 u r spreads, and the sum of the squares to twice that of
    itself: rstd to 64 u r beside its own 64 u, 4e-3 here. (Sums of squares less the square of the sum: r^2 u = 6e-2 of the
    variance for each rounding of the sums.)"""
    import chunked_sparse_delta_amd as sdm
    d = make(N, L, C, torch.float32, seed=N + L)
    gen = torch.Generator().manual_seed(1)
    d["x"] = 2 * torch.randn((N, L, C), generator=gen) + (2000 + 2 * torch.randn((N, 1, G, 1), generator=gen)).expand(N, 1, G, C // G).reshape(N, 1, C)
    ref = bars(d["x"], G, d["weight"], d["bias"], "silu", d["go"], None)
    mean, rstd = ref["mean"][0], ref["rstd"][0]
    assert bool(((mean * rstd > 500) & (mean * rstd < 2500)).all())
    d = {n: t.to(gpu) for n, t in d.items()}
    y, m, r = sdm.group_norm_fwd(d["x"], G, d["weight"], d["bias"], activation="silu")
    close(m, ref["mean"], torch.float32, "mean")
    rel = (r.double().cpu() / rstd - 1).abs()
    assert bool((rel <= U * (65 + 64 * mean * rstd)).all()), f"rstd off by {rel.max():.3g}"
    close(y, ref["y"], torch.float32, "y")
    g = sdm.group_norm_bwd(d["go"], d["x"], G, m, r, d["weight"], d["bias"], activation="silu")
    close(g["x"], ref["grad_x"], torch.float32, "grad_x")


@pytest.mark.parametrize("N,L,C,G", FORMS)
def test_means_whose_squares_overflow(gpu, N, L, C, G):
    """Means of 2e19, whose squares are past float32, a thousand times the spread, whose squares are not: mean and rstd as in
    test_means_far_from_zero, and finite values."""
    import chunked_sparse_delta_amd as sdm
    gen = torch.Generator().manual_seed(2)
    x = 1e16 * (2 * torch.randn((N, L, C), generator=gen) + 2000)
    d = x.double().view(N, L, G, C // G)
    mean = d.mean((1, 3))
    rstd = 1 / (d - mean[:, None, :, None]).square().mean((1, 3)).sqrt()
    y, m, r = sdm.group_norm_fwd(x.to(gpu), G)
    assert torch.isfinite(y).all()
    assert bool(((m.double().cpu() - mean).abs() <= 64 * U * mean).all())
    rel = (r.double().cpu() / rstd - 1).abs()
    assert bool((rel <= U * (65 + 64 * mean * rstd)).all()), f"rstd off by {rel.max():.3g}"


@pytest.mark.parametrize("N,L,C,G", [(2048, 128, 1024, 1), (2048, 16384, 8, 1), (2, 3000, 32, 4), (1024, 600, 64, 64)])
def test_first_rows_far_from_the_others(gpu, N, L, C, G):
    """Rows alike but for the first ones, a thousand spreads away (as a first token's large activations): what a thread takes as its
    origin. With u = 2^-24, sums of at most m = 8 rows' differences and squares from an origin at a distance d are off by
    u m^2 d / 2 + u m d and u m^2 d^2 / 2 + 2 u m d^2, what is left of the squares by (1.5 m^2 + 6 m) u d^2 = 144 u d^2, of 7/8 d^2:
    165 u of the variance, 83 u of rstd; with the joins' 64 u below 256 u. All rows but those, and all channels, are the same, so that
    no roundings average out."""
    import chunked_sparse_delta_amd as sdm
    gen = torch.Generator(device=gpu).manual_seed(L)
    first = min(128, L // 4)
    x = torch.rand((N, 1, 1), generator=gen, device=gpu).repeat(1, L, 1)
    x[:, :first] += 1000.1
    x = x.expand(N, L, C).contiguous()
    _, m, r = sdm.group_norm_fwd(x, G)
    one = x[:, :, 0].double()
    mean = one.mean(1)
    rstd = 1 / torch.sqrt((one - mean[:, None]).square().mean(1) + 1e-5)
    assert bool(((m.double() - mean[:, None]).abs() <= 64 * U * 1000).all())
    rel = (r.double() / rstd[:, None] - 1).abs().max()
    assert rel <= 256 * U, f"rstd off by {rel / U:.1f} u"


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,C,G", FORMS)
def test_reach_of_a_live_value(gpu, N, L, C, G, dtype, value):
    """A NaN or infinity in a live row, or in its gradient, stays in its sample and group: everything else, to the bit, is as it was; the
    parameters' gradients of that group's channels show it."""
    import chunked_sparse_delta_amd as sdm
    d = {n: t.to(gpu) for n, t in make(N, L, C, DT[dtype], seed=3).items()}
    D, n, row, c = C // G, N - 1, L // 2, (G // 2) * (C // G) + C // G // 3
    here = slice(c // D * D, (c // D + 1) * D)
    valid = torch.full((N,), max(1, L - 1), dtype=torch.int32, device=gpu)
    row = min(row, max(1, L - 1) - 1)

    def work(x, go):
        y, m, r = sdm.group_norm_fwd(x, G, d["weight"], d["bias"], activation="silu", valid_rows=valid)
        return [y, m, r, *sdm.group_norm_bwd(go, x, G, m, r, d["weight"], d["bias"], activation="silu", valid_rows=valid).values()]

    clean = work(d["x"], d["go"])
    for into in ("x", "go"):
        t = {"x": d["x"].clone(), "go": d["go"].clone()}
        t[into][n, row, c] = value
        y, m, r, dx, dw, db = work(t["x"], t["go"])
        for got, was in ((y, clean[0]), (dx, clean[3])):
            hit = got != was
            hit[n, :, here] = False
            assert not hit.any()
        for got, was in ((m, clean[1]), (r, clean[2])):
            hit = got != was
            hit[n, c // D] = False
            assert not hit.any()
        for got, was in ((dw, clean[4]), (db, clean[5])):
            hit = got != was
            hit[here] = False
            assert not hit.any() and not torch.isfinite(got[c])
        live = int(valid[n])
        assert not torch.isfinite(dx[n, :live, here]).all() and not y[n, live:].any() and not dx[n, live:].any()
        if into == "x":
            assert torch.isnan(y[n, :live, here]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,C,G", [(3000, 1, 1024, 8), (5000, 40, 24, 2), (3000, 2, 640, 2)])
def test_workgroups_take_samples_in_turn(gpu, N, L, C, G, dtype):
    """More samples than workgroups, whose threads meet in each way: by shuffles, by vectors and by channels."""
    check(gpu, N, L, C, G, dtype, "silu", seed=N)


def test_no_eps(gpu):
    """eps 0: a sample without a valid row, whose rstd is infinite, reads 0 and has gradients of 0; the others are as ever."""
    import chunked_sparse_delta_amd as sdm
    for N, L, C, G in ((3, 4, 64, 4), (3, 5, 30, 3), (3, 3000, 32, 4)):
        d = {n: t.to(gpu) for n, t in make(N, L, C, torch.float32, seed=2).items()}
        valid = torch.tensor([L, 0, L - 1], dtype=torch.int32, device=gpu)
        kw = {"activation": "silu", "eps": 0.0, "valid_rows": valid}
        y, m, r = sdm.group_norm_fwd(d["x"], G, d["weight"], d["bias"], **kw)
        g = sdm.group_norm_bwd(d["go"], d["x"], G, m, r, d["weight"], d["bias"], **kw)
        assert torch.isinf(r[1]).all() and not y[1].any() and not g["x"][1].any()
        assert all(torch.isfinite(t).all() for t in (y, m, g["x"], g["weight"], g["bias"]))

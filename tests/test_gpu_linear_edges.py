"""Linear attention on the GPU where launches change form and where values end, against its definition in 64 bits: bars and
helpers of test_gpu_linear.py."""

import math

import pytest
import torch

from tests.test_gpu_linear import DT, check_grads, close, grads_of, make, on, run, want

pytestmark = pytest.mark.gpu


# At least 512 segments' heads: a workgroup takes all tiles of a segment in turn. P * Hk * segments is a multiple of eight or not
# (then the grid is padded). T: one segment and several, of two tiles and more (bfloat16 128 tokens to a tile, 64 where a width is above
# 128; float32 64).
WHOLE = [
    # P, T, Hk, Hv, K, V, dtype, decay, start state
    (33, 200, 8, 16, 16, 16, "bf16", "token", True), (33, 200, 8, 16, 16, 16, "f32", "token", True),
    (33, 200, 5, 20, 8, 24, "bf16", "head", False), (33, 128, 5, 20, 8, 24, "f32", "head", False),
    (11, 520, 5, 20, 17, 9, "bf16", "token", True), (11, 520, 5, 20, 17, 9, "f32", "token", True),
    (33, 180, 8, 16, 136, 16, "bf16", "token", True),
]


@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,decay,start", WHOLE)
def test_many_segments(gpu, P, T, Hk, Hv, K, V, dtype, decay, start):
    """Streams that end in every tile of a segment, at its borders, before it and behind it; NaN in the padding."""
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    counts = [(0, 1, 63, 64, 65, 100, 127, 128, 129, 140, T - 1, T, T + 5)[p % 13] for p in range(P)]
    x = make(P, T, Hk, Hv, K, V, dt, decay, ragged=counts, seed=P + T, state=start)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    d = on(x, gpu)
    for p, n in enumerate(counts):
        for name in ("q", "k", "v") + (("log_decay",) if decay == "token" else ()):
            d[name][p, min(n, T):] = math.nan
    final = torch.full((P, Hv, K, V), math.nan, device=gpu)
    out = sdm.linear_attention_fwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], valid_tokens=d["valid"], state_out=final)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)
    assert not any(out[p, min(n, T):].any() for p, n in enumerate(counts))
    if start:       # ... and the state in place
        close(sdm.linear_attention_fwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], valid_tokens=d["valid"]), o, ao, dt)
        close(d["state"], s, as_, torch.float32)


@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,decay,start", [WHOLE[i] for i in (0, 1, 2, 5)])
def test_many_segments_backward(gpu, P, T, Hk, Hv, K, V, dtype, decay, start):
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    counts = [(0, 1, 63, 64, 65, 100, 127, 128, 129, 140, T - 1, T, T + 5)[p % 13] for p in range(P)]
    x = make(P, T, Hk, Hv, K, V, dt, decay, ragged=counts, seed=P + T, state=start)
    gen = torch.Generator().manual_seed(T)
    go, gs = torch.randn((P, T, Hv, V), generator=gen).to(dt), torch.randn((P, Hv, K, V), generator=gen)
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu), valid_tokens=d["valid"])
    check_grads(got, x, go, gs, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hv", [16, 64])
def test_many_heads_share_keys(gpu, Hv, dtype):
    """One key head for 16 and 64 value heads, over several segments: readings, and dq and dk summed over all of them."""
    import chunked_sparse_delta_amd as sdm
    dt, T, K, V = DT[dtype], 300, 24, 16
    x = make(1, T, 1, Hv, K, V, dt, "head", seed=Hv)
    out, final = run(gpu, x)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)
    gen = torch.Generator().manual_seed(Hv)
    go, gs = torch.randn((1, T, Hv, V), generator=gen).to(dt), torch.randn((1, Hv, K, V), generator=gen)
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu))
    check_grads(got, x, go, gs, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_gates_at_their_ends(gpu, dtype):
    """Decays of 0 and -80, and ones that clear the state (-inf, -1e30, -200: e^-200 is 0 in float32) in the middle of a segment and
    as its first and last token: every gradient is finite and right, that of a log-decay whose exponential is 0 is 0."""
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    x = make(1, 400, 1, 3, 64, 64, dt, seed=5)
    g = x["log_decay"]
    g[:, 50:90] = 0.0
    cleared = [(0, 0, -math.inf), (0, 100, -math.inf), (0, 301, -1e30), (0, 399, -math.inf), (1, 255, -math.inf), (1, 256, -math.inf), (1, 127, -1e30),
               (1, 128, -200.0), (2, 30, -200.0), (2, 31, -math.inf), (2, 32, -torch.finfo(torch.float32).max)]
    for h, t, value in cleared:
        g[0, t, h] = value
    g[0, 17, 1] = -80.0
    gen = torch.Generator().manual_seed(7)
    go, gs = torch.randn((1, 400, 3, 64), generator=gen).to(dt), torch.randn((1, 3, 64, 64), generator=gen)
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu))
    assert all(torch.isfinite(t).all() for t in got.values())
    check_grads(got, x, go, gs, dt)
    for h, t, value in cleared:
        assert got["log_decay"][0, t, h] == 0, (h, t, value)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_head_that_forgets(gpu, dtype):
    """A decay of -inf for one head at every token: its gradient is 0, the other head's is the formula's."""
    import chunked_sparse_delta_amd as sdm
    dt = DT[dtype]
    x = make(2, 300, 1, 2, 32, 40, dt, "head", seed=6)
    x["log_decay"][0] = -math.inf
    gen = torch.Generator().manual_seed(8)
    go, gs = torch.randn((2, 300, 2, 40), generator=gen).to(dt), torch.randn((2, 2, 32, 40), generator=gen)
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu))
    check_grads(got, x, go, gs, dt)
    assert got["log_decay"][0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [24, 130])
@pytest.mark.parametrize("name,value", [("v", math.inf), ("v", -math.inf), ("v", math.nan), ("k", math.nan), ("k", math.inf), ("log_decay", math.nan)])
def test_readings_do_not_look_ahead(gpu, dtype, K, name, value):
    """An infinity or NaN in a live token's k, v or log-decay leaves the readings of every earlier token, of other heads and of other
    streams, to the bit, as they are; one in v stays in its column."""
    x = make(2, 300, 2, 2, K, 40, DT[dtype], seed=17)
    clean, clean_final = run(gpu, x)
    for t in (0, 1, 31, 32, 63, 64, 100, 128, 170, 255, 256, 298, 299):
        y = {n: None if a is None else a.clone() for n, a in x.items()}
        if name == "log_decay":
            y[name][1, t, 1] = value
        else:
            y[name][1, t, 1, 7] = value
        out, final = run(gpu, y)
        hit, hit_final = ~torch.eq(out, clean), ~torch.eq(final, clean_final)
        assert not hit[0].any() and not hit[1, :, 0].any() and not hit[1, :t].any(), t
        assert not hit_final[0].any() and not hit_final[1, 0].any(), t
        if name == "v":
            assert not torch.isfinite(out[1, t:, 1, 7]).any() and not torch.isfinite(final[1, 1, :, 7]).any()
            hit[1, :, 1, 7], hit_final[1, 1, :, 7] = False, False
            assert not hit.any() and not hit_final.any(), t
        else:
            assert not torch.isfinite(out[1, t, 1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_segments_do_not_look_ahead(gpu, dtype):
    """The same where a workgroup takes a segment's tiles in turn: NaN in v of one token of every stream and head."""
    x = make(33, 250, 8, 16, 16, 40, DT[dtype], "head", seed=18)
    clean, clean_final = run(gpu, x)
    for t in (0, 40, 63, 64, 127, 128, 200, 249):
        y = {n: None if a is None else a.clone() for n, a in x.items()}
        y["v"][:, t, :, 30] = math.nan
        out, final = run(gpu, y)
        assert torch.equal(out[:, :t], clean[:, :t]) and torch.isnan(out[:, t:, :, 30]).all() and torch.isnan(final[..., 30]).all()
        rest = [c for c in range(40) if c != 30]
        assert torch.equal(out[..., rest], clean[..., rest]) and torch.equal(final[..., rest], clean_final[..., rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_log_decay_errors_have_no_sign(gpu, dtype):
    """The errors of log-decays' gradients in the middle of a segment, where their sums cancel, are of either sign, for long
    memories and keys and queries that are mostly positive: over 64 streams' heads, relative to their gradients' size, the mean of errors without
    a common sign is within 4 / sqrt(64) of their root mean square; of ones with a common sign it is nearer to that."""
    import chunked_sparse_delta_amd as sdm
    P, T, H, W, dt = 4, 128, 16, 64, DT[dtype]
    x = make(P, T, H, H, W, W, dt, seed=23)
    for n in ("q", "k"):
        x[n] = torch.nn.functional.silu(x[n].float()).to(dt)
    x["log_decay"] = (-0.003 - 0.01 * torch.rand(H, generator=torch.Generator().manual_seed(3))).expand(P, T, H).contiguous()
    gen = torch.Generator().manual_seed(9)
    go, gs = torch.randn((P, T, H, W), generator=gen).to(dt), torch.randn((P, H, W, W), generator=gen)
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu))["log_decay"]
    ref = grads_of(x, go, gs)["log_decay"]
    off = (got.double().cpu() - ref)[:, 32:96].mean(1) / ref.square().mean(1).sqrt()
    assert off.mean().abs() <= 0.5 * off.square().mean().sqrt(), f"mean {off.mean():.3g} of {off.square().mean().sqrt():.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_states_that_grow(gpu, dtype, decay):
    """Log-decays above zero, sums of up to 75 over a segment, and ones that fall by 70 and rise again: decays are then of up to
    e^75, their exponents rounded to 75 / log 2 u = 108 * 2^-24, under the bar's 64 * 2^-23."""
    import chunked_sparse_delta_amd as sdm
    dt, T = DT[dtype], 256
    x = make(2, T, 1, 3, 40, 24, dt, decay, seed=31)
    rate = 75.0 / T
    if decay == "head":
        x["log_decay"] = torch.tensor([rate, -rate, 0.01])
    else:
        x["log_decay"] = torch.stack([torch.full((T,), rate), torch.linspace(-2.2, 2.2, T) * 0.5, -rate * torch.rand(T)], -1).expand(2, T, 3).contiguous()
    out, final = run(gpu, x)
    (o, s), (ao, as_) = want(x), want(x, absolute=True)
    close(out, o, ao, dt)
    close(final, s, as_, torch.float32)
    gen = torch.Generator().manual_seed(4)
    go, gs = torch.randn((2, T, 3, 24), generator=gen).to(dt), torch.randn((2, 3, 40, 24), generator=gen)
    d = on(x, gpu)
    got = sdm.linear_attention_bwd(d["state"], d["k"], d["v"], d["log_decay"], d["q"], go.to(gpu), grad_state=gs.to(gpu))
    check_grads(got, x, go, gs, dt)

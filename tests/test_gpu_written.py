"""Tensors of the caller's that linear attention and group norm write: their versions rise, so that a backward which saved one
of them is refused by autograd instead of reading what was not there in the forward."""

import pytest
import torch

pytestmark = pytest.mark.gpu
STALE = "modified by an inplace operation"


def inputs(gpu, P=2, T=40, Hk=1, Hv=2, K=16, V=24):
    gen = torch.Generator().manual_seed(T)

    def randn(*s):
        return torch.randn(s, generator=gen).to(gpu)

    return {"state": randn(P, Hv, K, V), "k": randn(P, T, Hk, K), "v": randn(P, T, Hv, V), "log_decay": -torch.rand(Hv, generator=gen).to(gpu),
            "q": randn(P, T, Hk, K)}


@pytest.mark.parametrize("form", ["fwd", "step"])
@pytest.mark.parametrize("into", ["state", "state_out"])
def test_state_advanced_before_the_backward(gpu, form, into):
    """recompute=True reads the start state in the backward: advanced meanwhile, the backward is refused. What a forward kept
    takes its place: then the state may be advanced, and the gradients are what they are without."""
    import chunked_sparse_delta_amd as sdm
    call = sdm.linear_attention_fwd if form == "fwd" else sdm.linear_attention_step
    for recompute in (True, False):
        x = inputs(gpu)
        x["v"].requires_grad_()
        rest = [x[n] for n in ("k", "v", "log_decay", "q")]
        want, = torch.autograd.grad(sdm.linear_attention(x["state"], *rest, recompute=recompute)[0].square().sum(), [x["v"]])
        out, _ = sdm.linear_attention(x["state"], *rest, recompute=recompute)
        version = x["state"]._version
        with torch.no_grad():
            if into == "state":
                call(x["state"], *rest)
            else:
                call(torch.zeros_like(x["state"]), *rest, state_out=x["state"])
        assert x["state"]._version > version
        if recompute:
            with pytest.raises(RuntimeError, match=STALE):
                out.square().sum().backward()
        else:
            out.square().sum().backward()
            assert torch.equal(x["v"].grad, want)


def test_given_outputs(gpu):
    """`out`, `kept` and views of a saved tensor count as much as the state."""
    import chunked_sparse_delta_amd as sdm
    x = inputs(gpu)
    rest = [x[n] for n in ("k", "v", "log_decay", "q")]
    saved = torch.randn_like(x["v"]).requires_grad_()
    for call in (lambda t: sdm.linear_attention_fwd(None, *rest, out=t), lambda t: sdm.linear_attention_step(x["state"].clone(), *rest, out=t),
                 lambda t: sdm.linear_attention_fwd(None, *rest, out=t.flatten().view_as(t))):
        held = saved.detach().clone()
        y = (saved * held).sum()
        call(held)
        with pytest.raises(RuntimeError, match=STALE):
            y.backward()
    kept = torch.empty(sdm.linear_attention_kept_bytes(2, 40, 1, 2, 16, 24, torch.float32), dtype=torch.uint8, device=gpu)
    version = kept._version
    sdm.linear_attention_fwd(x["state"], *rest, state_out=torch.empty_like(x["state"]), kept=kept)
    assert kept._version > version


@pytest.mark.parametrize("L", [1, 3000])
def test_group_norm_in_place(gpu, L):
    import chunked_sparse_delta_amd as sdm
    x = torch.randn((3, L, 32), device=gpu)
    w = torch.ones(32, device=gpu, requires_grad=True)
    y = sdm.group_norm(x, 4, w, activation="silu")
    sdm.group_norm_fwd(x, 4, w.detach(), activation="silu", out=x)
    with pytest.raises(RuntimeError, match=STALE):
        y.sum().backward()


def test_inference_tensors(gpu):
    """Tensors made under inference_mode, which have no version, are advanced as ever, in that mode and outside of it."""
    import chunked_sparse_delta_amd as sdm
    x = inputs(gpu)
    with torch.inference_mode():
        y = {n: t.clone() for n, t in x.items()}
        a = sdm.linear_attention_fwd(*y.values())
        b = sdm.linear_attention_step(*(y[n] if n in ("state", "log_decay") else y[n][:, :1] for n in y))
        z = torch.randn((2, 8), device=gpu)
        sdm.group_norm_fwd(z, 2, out=z)
    first = x["state"].clone()
    assert torch.equal(a, sdm.linear_attention_fwd(*x.values()))
    c = sdm.linear_attention_step(*(x[n] if n in ("state", "log_decay") else x[n][:, :1] for n in x))
    assert torch.equal(b, c) and torch.equal(x["state"], y["state"]) and not torch.equal(first, x["state"])
    sdm.linear_attention_fwd(*y.values())
    sdm.group_norm_fwd(z, 2, out=z)

"""Tensors of the caller's that the sparse memory, the gated delta rule and layer norm write: their versions rise, so that a
backward which saved one of them is refused by autograd instead of reading what was not there in the forward."""

import pytest
import torch

import workloads
from tests.gpu_util import generate, to_torch

pytestmark = pytest.mark.gpu
STALE = "modified by an inplace operation"
NAMES = ("k", "v", "beta", "log_decay", "q")


def inputs(gpu, P=2, T=40, Hk=1, Hv=2, K=16, V=24):
    gen = torch.Generator().manual_seed(T)

    def randn(*s):
        return torch.randn(s, generator=gen).to(gpu)

    return {"state": randn(P, Hv, K, V), "k": torch.nn.functional.normalize(randn(P, T, Hk, K), dim=-1), "v": randn(P, T, Hv, V),
            "beta": torch.rand((P, T, Hv), generator=gen).to(gpu), "log_decay": -torch.rand((P, T, Hv), generator=gen).to(gpu),
            "q": randn(P, T, Hk, K)}


@pytest.mark.parametrize("form", ["fwd", "step"])
@pytest.mark.parametrize("into", ["state", "state_out"])
def test_state_advanced_before_the_backward(gpu, form, into):
    import chunked_sparse_delta_amd as sdm
    call = sdm.gated_delta_fwd if form == "fwd" else sdm.gated_delta_step
    for recompute in (True, False):
        x = inputs(gpu)
        x["v"].requires_grad_()
        rest = [x[n] for n in NAMES]
        want, = torch.autograd.grad(sdm.gated_delta_rule(x["state"], *rest, recompute=recompute)[0].square().sum(), [x["v"]])
        out, _ = sdm.gated_delta_rule(x["state"], *rest, recompute=recompute)
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
    import chunked_sparse_delta_amd as sdm
    x = inputs(gpu)
    rest = [x[n] for n in NAMES]
    saved = torch.randn_like(x["v"]).requires_grad_()
    ws = torch.empty(sdm.gated_delta_workspace_bytes(2, 40, 1, 2, 16, 24, torch.float32, True), dtype=torch.uint8, device=gpu)
    for call in (lambda t: sdm.gated_delta_fwd(None, *rest, out=t), lambda t: sdm.gated_delta_step(x["state"].clone(), *rest, out=t),
                 lambda t: sdm.layer_norm_fwd(x["v"], out=t)):
        held = saved.detach().clone()
        y = (saved * held).sum()
        call(held)
        with pytest.raises(RuntimeError, match=STALE):
            y.backward()
    version = ws._version
    sdm.gated_delta_fwd(x["state"].clone(), *rest, workspace=ws, keep=True)
    assert ws._version > version


@pytest.mark.parametrize("form", ["sdm_fwd", "noalloc", "phases", "write_read"])
def test_bank(gpu, form):
    """The bank, the readings' buffer and the counter of repeated writes."""
    import chunked_sparse_delta_amd as sdm
    t = to_torch(generate(workloads.CONFIGS["0"].replace(P=2, T=40, hd=8, M=64)), gpu)
    args = [t[n] for n in ("k_idx", "k_val", "v", "beta", "log_decay", "q_idx", "q_val")]
    bank, out, count = t["bank"].clone(), torch.zeros_like(t["v"]), torch.zeros(1, dtype=torch.int64, device=gpu)
    before = [x._version for x in (bank, out, count)]
    if form == "sdm_fwd":
        sdm.sdm_fwd(bank, *args, chunk=16, out=out, repeated_writes=count)
    elif form == "noalloc":
        sdm.sdm_fwd_noalloc(bank, *args, chunk=16, out=out, repeated_writes=count)
    elif form == "phases":
        ws = torch.empty(sdm.workspace_bytes(2, 40, 16, 2, 2, 8), dtype=torch.uint8, device=gpu)
        sdm.sdm_fwd_phase1(bank, *args, chunk=16, workspace=ws, repeated_writes=count)
        assert bank._version == before[0]        # the first phase does not write it
        sdm.sdm_fwd_phase2(bank, *args, chunk=16, workspace=ws, out=out)
    else:
        k_idx, k_val, v, beta, g, q_idx, q_val = args
        v = v.clone().requires_grad_()
        y = sdm.sdm_write_read(bank, k_idx, k_val, v, beta, g, q_idx, q_val, chunk=16)
        assert bank._version > before[0]
        for _ in range(2):                       # the backward restores what it writes: it may run again
            y.sum().backward(retain_graph=True)
        return
    assert all(x._version > n for x, n in zip((bank, out, count), before))


def test_inference_tensors(gpu):
    """Tensors made under inference_mode, which have no version, are advanced as ever, in that mode and outside of it."""
    import chunked_sparse_delta_amd as sdm
    x = inputs(gpu)
    with torch.inference_mode():
        y = {n: t.clone() for n, t in x.items()}
        a = sdm.gated_delta_fwd(*y.values())
    assert torch.equal(a, sdm.gated_delta_fwd(*x.values())) and torch.equal(x["state"], y["state"])
    sdm.gated_delta_fwd(*y.values())

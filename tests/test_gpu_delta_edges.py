"""The gated delta rule on the GPU at the ends of what it takes."""

import pytest
import torch

from tests.test_gpu_delta import NAMES, gpu_of, make

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

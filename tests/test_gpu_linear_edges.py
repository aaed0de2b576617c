"""Linear attention on the GPU where launches change form and where values end, against its definition in 64 bits: bars and
helpers of test_gpu_linear.py."""

import math

import pytest
import torch

from tests.test_gpu_linear import DT, check_grads, make, on

pytestmark = pytest.mark.gpu


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

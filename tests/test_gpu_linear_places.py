"""Results of linear attention in the places that its header allows: the same bits as in places of their own."""

import pytest
import torch

from tests.test_gpu_linear import DT, NAMES, make, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5])
def test_steps_in_the_values_place(gpu, T, dtype):
    import chunked_sparse_delta_amd as sdm
    x = on(make(3, T, 2, 4, 40, 36, DT[dtype], ragged=[T, T - 1, T], seed=T), gpu)
    args = [x[n] for n in NAMES]
    want = sdm.linear_attention_step(*[t.clone() for t in args], valid_tokens=x["valid"])
    got = sdm.linear_attention_step(*args, valid_tokens=x["valid"], out=x["v"])
    assert got.data_ptr() == x["v"].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("form", ["fwd", "step"])
def test_readings_beside_strided_rows(gpu, form):
    """q, k and v as slices of streams far apart, the readings in the room between the streams."""
    import chunked_sparse_delta_amd as sdm
    P, T, Hk, Hv, K, V = 2, 7, 1, 2, 16, 8
    width = 2 * Hk * K + Hv * V
    room = torch.randn(2 * 4096, device=gpu)
    fused = room.as_strided((P, T, width), (4096, width, 1))
    q, k, v = (fused[..., a:a + h * w].unflatten(-1, (h, w)) for a, h, w in ((0, Hk, K), (Hk * K, Hk, K), (2 * Hk * K, Hv, V)))
    g, state = -torch.rand(Hv, device=gpu), torch.randn((P, Hv, K, V), device=gpu)
    call = sdm.linear_attention_fwd if form == "fwd" else sdm.linear_attention_step
    want = call(state.clone(), k, v, g, q)
    out = room[4096 - P * T * Hv * V:4096].view(P, T, Hv, V)
    assert torch.equal(call(state, k, v, g, q, out=out), want)
    with pytest.raises(sdm.SdmError, match="overlap"):
        call(state, k, v, g, q, out=room[4097 - P * T * Hv * V:4097].view(P, T, Hv, V))

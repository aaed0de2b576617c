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


def test_rows_far_apart(gpu):
    """Tokens 2^25 elements apart, the last past 2^32: the bits of dense copies, forward, backward and by single tokens."""
    import chunked_sparse_delta_amd as sdm
    T, H, W, far = 130, 2, 16, 1 << 25
    room = torch.empty((T - 1) * far + 3 * H * W, dtype=torch.bfloat16, device=gpu)
    fused = room.as_strided((1, T, 3 * H * W), (0, far, 1))
    fused.copy_(torch.randn((1, T, 3 * H * W), generator=torch.Generator().manual_seed(1)))
    q, k, v = (fused[..., i * H * W:(i + 1) * H * W].unflatten(-1, (H, W)) for i in range(3))
    g, go = -torch.rand(H, device=gpu), torch.randn((1, T, H, W), device=gpu).bfloat16()
    got = []
    for form in (lambda t: t, lambda t: t.contiguous()):
        a, b, c = (form(t) for t in (k, v, q))
        state, step = torch.empty((1, H, W, W), device=gpu), torch.zeros((1, H, W, W), device=gpu)
        got.append([sdm.linear_attention_fwd(None, a, b, g, c, state_out=state), state, sdm.linear_attention_step(step, a, b, g, c), step,
                    *sdm.linear_attention_bwd(None, a, b, g, c, go).values()])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_slots_far_apart(gpu):
    """Slots of a pool on both sides of 2^32 elements."""
    import chunked_sparse_delta_amd as sdm
    H, W = 4, 64
    slots = (1 << 32) // (H * W * W) + 4
    pool = torch.empty((slots, H, W, W), device=gpu)
    ids = torch.tensor([slots - 1, 3, slots - 5], dtype=torch.int32, device=gpu)
    start = torch.randn((3, H, W, W), device=gpu)
    pool[ids.long()] = start
    x = on(make(3, 2, 2, H, W, W, torch.bfloat16, "head", seed=4), gpu)
    rest = [x[n] for n in NAMES[1:]]
    want = sdm.linear_attention_step(start, *rest)
    assert torch.equal(sdm.linear_attention_step(pool, *rest, state_ids=ids), want) and torch.equal(pool[ids.long()], start)

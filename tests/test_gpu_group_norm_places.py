"""Results of group norm in the places that its header allows: the same bits as in places of their own."""

import pytest
import torch

from tests.test_gpu_group_norm import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,C,G", [(40, 1, 256, 4), (6, 5, 320, 2), (9, 3, 21, 3), (2, 2500, 64, 8)])
def test_norm_gradient_in_place(gpu, N, L, C, G, dtype):
    """grad_x in the place of grad_out and in that of x, through the C ABI (the binding makes a tensor of its own)."""
    import ctypes
    import chunked_sparse_delta_amd as sdm
    from chunked_sparse_delta_amd import _Exec, _load, group
    dt, lib = DT[dtype], _load()
    x, go = (torch.randn((N, L, C), device=gpu).to(dt) for _ in range(2))
    w, b = (torch.randn(C, device=gpu).to(dt) for _ in range(2))
    valid = torch.tensor([max(1, L - n % 2) for n in range(N)], dtype=torch.int32, device=gpu)
    _, m, r = sdm.group_norm_fwd(x, G, w, b, activation="silu", valid_rows=valid)
    want = sdm.group_norm_bwd(go, x, G, m, r, w, b, activation="silu", valid_rows=valid)
    shape = group._SHAPE(N, L, C, G, sdm._DTYPES[dt], sdm._DTYPES[dt], 1, 1e-5)
    ws = torch.empty(max(256, lib.sdm_group_norm_workspace_bytes(shape, 1)), dtype=torch.uint8, device=gpu)
    ex = _Exec(torch.cuda.current_stream().cuda_stream, ws.data_ptr(), ws.numel(), None, 0, None)
    for place in ("go", "x"):
        a = {"x": x.clone(), "go": go.clone()}
        dw, db = torch.empty_like(w), torch.empty_like(b)
        rc = lib.sdm_group_norm_bwd(shape, a["go"].data_ptr(), a["x"].data_ptr(), L * C, C, w.data_ptr(), b.data_ptr(), valid.data_ptr(), m.data_ptr(),
                                    r.data_ptr(), a[place].data_ptr(), dw.data_ptr(), db.data_ptr(), ctypes.byref(ex))
        assert rc == 0, lib.sdm_last_error()
        torch.cuda.synchronize()
        assert torch.equal(a[place], want["x"]) and torch.equal(dw, want["weight"]) and torch.equal(db, want["bias"])


@pytest.mark.parametrize("L", [1, 3000])
def test_norm_across_its_input(gpu, L):
    """A dense output across a strided or shifted x is refused."""
    import chunked_sparse_delta_amd as sdm
    room = torch.randn(3 * L * 40 + 64, device=gpu)
    x = room[:3 * L * 40].view(3, L, 40)[..., :32]
    for out in (room[:3 * L * 32], room[16:16 + 3 * L * 32]):
        with pytest.raises(sdm.SdmError, match="overlap"):
            sdm.group_norm_fwd(x, 4, out=out.view(3, L, 32))


@pytest.mark.parametrize("L,G", [(130, 2), (3000, 2)])
def test_rows_far_apart(gpu, L, G):
    """Rows so far apart that the last lies past 2^32 elements: the bits of a dense copy."""
    import chunked_sparse_delta_amd as sdm
    C = 24
    far = (1 << 32) // (L - 2)
    x = torch.empty((L - 1) * far + C, dtype=torch.bfloat16, device=gpu).as_strided((1, L, C), (0, far, 1))
    x.copy_(torch.randn((1, L, C), generator=torch.Generator().manual_seed(1)))
    go = torch.randn((1, L, C), device=gpu).bfloat16()
    got = []
    for t in (x, x.contiguous()):
        y, m, r = sdm.group_norm_fwd(t, G, activation="silu")
        got.append([y, m, r, *sdm.group_norm_bwd(go, t, G, m, r, activation="silu").values()])
    assert all(torch.equal(a, b) for a, b in zip(*got))

"""Layer norm of more rows than one launch takes (2^32 threads)."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,N", [(2 ** 29 + 40, 2), (2 ** 24 + 3, 1032)])
def test_many_rows(gpu, rows, N):
    """Short rows share wavefronts, longer ones have 256 threads each; a row's result is the one it has in a small call."""
    import chunked_sparse_delta_amd as sdm
    gen = torch.Generator(device=gpu).manual_seed(rows)
    part = torch.randn((2 ** 12 + 1, N), generator=gen, device=gpu).bfloat16()     # repeated: an odd period, so that none lines up
    x = torch.empty((rows, N), dtype=torch.bfloat16, device=gpu)
    whole = rows // len(part) * len(part)
    x[:whole].view(-1, len(part), N).copy_(part)
    x[whole:] = part[:rows - whole]
    y, mean, rstd = sdm.layer_norm_fwd(x)
    want = sdm.layer_norm_fwd(part)
    for got, one in zip((y, mean, rstd), want):
        assert (got[:whole].view(-1, *one.shape) == one).all() and torch.equal(got[whole:], one[:rows - whole])

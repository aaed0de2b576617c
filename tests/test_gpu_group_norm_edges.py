"""Group norm on the GPU where its sums cancel and where values end, against its definition in 64 bits: bars and helpers of
test_gpu_group_norm.py."""

import pytest
import torch

from tests.test_gpu_group_norm import U

pytestmark = pytest.mark.gpu

# Every way in which a tile's threads meet (test_gpu_group_norm.py names them by their shapes), and blocks of rows: D divided by
# vectors of a power of two, by others, by none; groups wider than a workgroup.
FORMS = [(70, 1, 128, 2), (9, 16, 512, 16), (3, 1, 2048, 1), (2, 7, 320, 32), (2, 3000, 32, 4), (1, 3, 20001, 3), (3, 777, 1000, 8)]


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

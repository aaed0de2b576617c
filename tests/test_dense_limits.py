"""Shapes that the dense operators' kernels could not address or launch are refused on the host (no GPU needed)."""

import pytest

from tests.test_dense_abi import NULL, RANGE, Delta, lib  # noqa: F401


def code_of(lib, form, **shape):
    """The call's code; q is NULL, so that nothing runs: a shape that is accepted gives NULL."""
    c = Delta(lib)
    c.shape |= shape
    c.ptr["q"] = None
    return c.run(form)[0]


def size(lib, backward, **shape):
    c = Delta(lib)
    return lib.sdm_gated_delta_workspace_bytes(c.dense._SHAPE(*(c.shape | shape).values()), backward)


# Rows that the kernels cannot load as they are come as copies with padded widths: the offsets in a chunk of those have
# to fit 32 bits.
KEYS = dict(streams=1, tokens=64, key_heads=540000, value_heads=540000, head_dim=31, value_dim=1, dtype=1)     # 63 x 540000 x 64
VALUES = dict(streams=1, tokens=64, key_heads=1, value_heads=5000000, head_dim=1, value_dim=1, dtype=1)        # 63 x 5000000 x 8


@pytest.mark.parametrize("shape", [KEYS, VALUES])
def test_offsets_of_padded_rows(lib, shape):
    for form in ("fwd", "bwd"):
        assert code_of(lib, form, **shape) == RANGE
        assert code_of(lib, form, **shape | dict(tokens=63)) == (RANGE if shape is VALUES else NULL)
        assert code_of(lib, form, **shape | dict(tokens=1)) == NULL
    assert code_of(lib, "step", **shape) == NULL
    for backward in (0, 1):
        assert size(lib, backward, **shape) == 0 and size(lib, backward, **shape | dict(tokens=1)) > 0
    # float32: chunks of 32 tokens
    assert code_of(lib, "fwd", **KEYS | dict(dtype=0)) == NULL


# A launch holds less than 2^32 threads: 512 for 64 columns of a state, 256 for a chunk of a head, 64 for 16 columns of a state
# in a call on single tokens.
def test_launches(lib):
    one = dict(streams=1 << 20, tokens=1, key_heads=1, value_heads=8, head_dim=1, value_dim=64, dtype=0)
    for form in ("fwd", "bwd"):
        assert code_of(lib, form, **one) == RANGE
        assert code_of(lib, form, **one | dict(streams=(1 << 20) - 1)) == NULL
        assert code_of(lib, form, **one | dict(streams=1 << 19, value_dim=65)) == RANGE
        assert code_of(lib, form, **one | dict(streams=1 << 19, tokens=129)) == RANGE      # chunks of 32 tokens
        assert code_of(lib, form, **one | dict(streams=1 << 19, tokens=96)) == NULL
    assert size(lib, 0, **one) == size(lib, 1, **one) == 0
    assert code_of(lib, "step", **one) == NULL
    assert code_of(lib, "step", **one | dict(value_dim=129)) == RANGE
    assert code_of(lib, "step", **one | dict(value_dim=112)) == NULL


def test_workspace_of_another_device():
    """A workspace on another GPU than the call's is refused: the kernels would reach for memory that is not theirs."""
    import torch
    from chunked_sparse_delta_amd import dense

    class On:      # as much of a tensor, and of a stream, as the check reads
        cuda_stream = 0

        def __init__(self, device):
            self.device = torch.device(device)

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 256

        def numel(self):
            return 512

        def element_size(self):
            return 1

    assert len(dense._exec(On("cuda:1"), 1, On("cuda:1"))) == len(dense._exec(On("cuda:1"), 1))
    for device in ("cuda:1", "cpu"):
        with pytest.raises(ValueError):
            dense._exec(On("cuda:0"), 0, On(device))

"""Arrays that overlap, and shapes past a launch, in group norm's entry points: refused on the host before any device work. (A call
that passes these checks is let down by its missing workspace here, which is looked at after them: no GPU needed.)"""

import os

import pytest

from tests.test_dense_abi import FAKE, RANGE, ROOT, SHAPE, WORKSPACE, lib  # noqa: F401
from tests.test_linear_abi import norm

N, L, C = 4, 5000, 32      # norm()'s sizes, dense rows by default: elements of four bytes
X, DY, WHOLE = FAKE, FAKE + (6 << 36), N * L * C * 4


def fwd(lib, y, **how):
    return norm(lib, False, y=y, ws_bytes=0, **how)


def bwd(lib, **how):
    return norm(lib, True, ws_bytes=0, **how)


@pytest.mark.parametrize("off", [4, -4, WHOLE - 4, 4 - WHOLE, C * 4, L * C * 4])
def test_output_across_its_input(lib, off):
    """y, or grad_x, shifted against x or grad_out by an element, a row, a sample, or all but one element."""
    assert fwd(lib, X + off) == SHAPE and b"overlap" in lib.sdm_last_error()
    assert bwd(lib, dx=X + off) == SHAPE and b"overlap" in lib.sdm_last_error()
    assert bwd(lib, dx=DY + off) == SHAPE
    for far in (WHOLE, -WHOLE):
        assert fwd(lib, X + far) == bwd(lib, dx=X + far) == bwd(lib, dx=DY + far) == WORKSPACE


@pytest.mark.parametrize("xs,xr", [(L * C, C), (L * (C + 8), C + 8), (L * C + 64, C), (0, C), (L * C, 0)])
def test_output_in_a_strided_input(lib, xs, xr):
    """In x's place only where x is dense; before it and behind it everywhere."""
    code = WORKSPACE if (xs, xr) == (L * C, C) else SHAPE
    assert fwd(lib, X, xs=xs, xr=xr) == bwd(lib, dx=X, xs=xs, xr=xr) == code
    end = X + ((N - 1) * xs + (L - 1) * xr + C) * 4
    for y in (end, X - WHOLE):
        assert fwd(lib, y, xs=xs, xr=xr) == bwd(lib, dx=y, xs=xs, xr=xr) == WORKSPACE
    assert fwd(lib, end - 4, xs=xs, xr=xr) == bwd(lib, dx=end - 4, xs=xs, xr=xr) == SHAPE


def test_output_between_samples_and_rows(lib):
    """Samples, or rows, far apart: in the room between them, but not an element more."""
    far = 2 * N * L * C
    for first, last in ((X + L * C * 4, -C * 4), (X + far * 4 - WHOLE, 4)):
        assert fwd(lib, first, xs=far) == bwd(lib, dx=first, xs=far) == WORKSPACE
        assert fwd(lib, first + last, xs=far) == bwd(lib, dx=first + last, xs=far) == SHAPE
    one = dict(samples=1, rows=2, xs=0)
    assert bwd(lib, dx=X + C * 4, xr=8 * C, **one) == bwd(lib, dx=X + C * 4, xr=3 * C, **one) == WORKSPACE
    assert bwd(lib, dx=X + C * 4, xr=3 * C - 1, **one) == SHAPE
    # one row is dense whatever its strides are, none overlaps nothing
    assert bwd(lib, dx=X, samples=1, rows=1, xs=12345, xr=1) == bwd(lib, dx=X + 4, rows=0) == WORKSPACE


@pytest.mark.parametrize("name,count", [("w", C), ("b", C), ("valid", N)])
def test_output_over_the_others(lib, name, count):
    p = {name: FAKE + (1 << 44)}
    at = p[name]
    assert fwd(lib, at + 4 - WHOLE, **p) == fwd(lib, at + count * 4 - 4, **p) == SHAPE
    assert fwd(lib, at - WHOLE, **p) == fwd(lib, at + count * 4, **p) == WORKSPACE
    assert bwd(lib, dx=at + 4 - WHOLE, **p) == bwd(lib, dw=at, **p) == bwd(lib, db=at, **p) == SHAPE


def test_gradients_in_place(lib):
    """grad_x may take grad_out's place, or a dense x's; the parameters' gradients nobody's."""
    assert bwd(lib, dx=DY) == bwd(lib, dx=X) == bwd(lib, dx=X, dy=X) == WORKSPACE
    assert bwd(lib, dx=X, xr=C + 8, xs=L * (C + 8)) == SHAPE
    for name in ("dw", "db"):
        for at in (X, X + 64, DY, DY + 64, FAKE + (4 << 36), FAKE + (5 << 36)):      # x, grad_out, mean, rstd
            assert bwd(lib, **{name: at}) == SHAPE


def test_launches(lib):
    """Samples that are cut into blocks: samples * blocks * tiles stays below 2^24, the header says so, and what is refused
    needs a workspace of 0 bytes."""
    from chunked_sparse_delta_amd import group
    text = " ".join(open(os.path.join(ROOT, "include", "sdm_linear.h")).read().replace("*", " ").split())
    assert "2^24" in text[text.index("Group norm with an activation over"):text.index("SDM_ACT_NONE")]
    for back in (False, True):
        for samples, code in ((1 << 24, RANGE), ((1 << 24) - 1, WORKSPACE)):
            assert norm(lib, back, ws_bytes=0, samples=samples, x=FAKE << 4, y=FAKE << 5, dx=FAKE << 5, dy=FAKE << 6) == code
            size = lib.sdm_group_norm_workspace_bytes(group._SHAPE(samples, 5000, 32, 4, 0, 0, 1, 1e-5), 1 if back else 0)
            assert (size == 0) == (code == RANGE)

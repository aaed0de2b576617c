"""Results of linear attention's entry points that overlap an input: refused on the host before any device work. (A sequence that
passes these checks is let down by its missing workspace here, which is looked at after them: no GPU needed.)"""

import pytest

from tests.test_dense_abi import FAKE, SHAPE, WORKSPACE, lib  # noqa: F401
from tests.test_linear_abi import Attention

# Attention()'s: 2 streams of 600 tokens, float32, q and k 2 heads of 64, v 4 of 32, strides 2^16, 2^9 and 2^6
OUT = 2 * 600 * 4 * 32 * 4


def code(lib, form, stride=None, shape=None, **ptr):
    c = Attention(lib)
    c.ptr |= ptr
    c.ws_bytes = 0
    c.stride = stride or c.stride
    c.shape |= shape or {}
    rc, msg = c.run(form)
    assert rc == (SHAPE if "overlap" in msg else WORKSPACE), msg
    return rc


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "state", "valid"])
def test_readings_over_an_input(lib, name):
    p = FAKE + (40 << 36)
    for form in ("fwd", "step"):
        assert code(lib, form, **{name: p, "out": p + 4 - OUT}) == SHAPE
        if (form, name) != ("step", "v"):
            assert code(lib, form, **{name: p, "out": p}) == SHAPE
    assert code(lib, "fwd", **{name: p, "out": p - OUT}) == WORKSPACE
    if name in "qkv":      # past the last row
        width, heads = (32, 4) if name == "v" else (64, 2)
        end = p + 4 * ((1 << 16) + 599 * (1 << 9) + (heads - 1) * (1 << 6) + width)
        assert code(lib, "fwd", **{name: p, "out": end}) == WORKSPACE
        assert code(lib, "fwd", **{name: p, "out": end - 4}) == code(lib, "step", **{name: p, "out": end - 4}) == SHAPE


def test_readings_between_rows(lib):
    """Streams far apart with the readings between them; tokens far apart likewise; heads before tokens."""
    v = FAKE + (40 << 36)
    far = dict(stride=[1 << 24, 1 << 9, 1 << 6], v=v)
    last = v + 4 * (1 << 24) - OUT
    assert code(lib, "fwd", out=last, **far) == WORKSPACE
    assert code(lib, "fwd", out=last + 4, **far) == code(lib, "step", out=last + 4, **far) == SHAPE
    two = dict(stride=[0, 1 << 9, 1 << 6], shape=dict(streams=1, tokens=2), v=v)
    first = v + 4 * (3 * 64 + 32)
    assert code(lib, "fwd", out=first, **two) == WORKSPACE
    assert code(lib, "fwd", out=first - 4, **two) == code(lib, "step", out=first - 4, **two) == SHAPE
    heads = dict(stride=[0, 1 << 6, 1 << 20], shape=dict(streams=1), v=v)
    first = v + 4 * (599 * 64 + 32)
    assert code(lib, "fwd", out=first, **heads) == WORKSPACE
    assert code(lib, "fwd", out=first - 4, **heads) == SHAPE


def test_readings_in_the_values_place(lib):
    """Sequences read v again after they wrote; single tokens' readings may take a dense v's place (test_gpu_linear_places.py), not
    lie across it."""
    v = FAKE + (40 << 36)
    dense = dict(stride=[600 * 4 * 32, 4 * 32, 32], shape=dict(key_heads=4, head_dim=32), v=v)
    assert code(lib, "fwd", out=v, **dense) == SHAPE
    assert code(lib, "step", out=v + 4 * 32, **dense) == SHAPE
    assert code(lib, "step", out=v, v=v) == SHAPE


def test_state_over_the_inputs(lib):
    for name in ("q", "k", "v", "g", "valid", "out"):
        for form in ("fwd", "step"):
            p = Attention(lib).ptr[name]
            assert code(lib, form, state=p, state_out=p) == SHAPE, name
            assert code(lib, form, state_out=p) == SHAPE, name


@pytest.mark.parametrize("grad", ["gq", "gk", "gv", "gg", "gstate"])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "state", "valid", "go", "gs"])
def test_gradients_over_an_input(lib, grad, name):
    p = Attention(lib).ptr[name]
    assert code(lib, "bwd", **{grad: p}) == (WORKSPACE if (grad, name) == ("gstate", "gs") else SHAPE)

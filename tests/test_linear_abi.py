"""The C ABI of linear attention and group norm on the host: include/sdm_linear.h's functions are exported and reject
malformed calls with the documented code before any device work (no GPU needed)."""

import ctypes
import os
import re

import pytest

from tests.test_dense_abi import ALIGN, DTYPE, FAKE, NULL, RANGE, ROOT, SHAPE, WORKSPACE, lib  # noqa: F401

HEADER = os.path.join(ROOT, "include", "sdm_linear.h")


def test_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sdm_\w+)\s*\(", text)))
    assert names == ["sdm_group_norm_bwd", "sdm_group_norm_fwd", "sdm_group_norm_workspace_bytes", "sdm_linear_attention_bwd",
                     "sdm_linear_attention_fwd", "sdm_linear_attention_kept_bytes", "sdm_linear_attention_step",
                     "sdm_linear_attention_workspace_bytes"]
    assert all(hasattr(lib, n) for n in names)


class Attention:
    def __init__(self, lib):
        from chunked_sparse_delta_amd import dense
        self.lib, self.dense = lib, dense
        self.shape = dict(streams=2, tokens=600, key_heads=2, value_heads=4, head_dim=64, value_dim=32, dtype=0, scale=1.0)
        self.ptr = {n: FAKE + (i << 36) for i, n in enumerate(
            ["q", "k", "v", "g", "state", "state_out", "valid", "out", "ws", "ids", "go", "gs", "gq", "gk", "gv", "gg", "gstate",
             "kept"])}
        self.ptr["kept"] = None
        self.stride, self.ws_bytes, self.slots, self.per_token = [1 << 16, 1 << 9, 1 << 6], None, 2, 1

    def run(self, form):
        from chunked_sparse_delta_amd import _Exec
        D, r, lib, p = self.dense, ctypes.byref, self.lib, self.ptr
        sh = D._SHAPE(*self.shape.values())
        q, k, v = (D._ROWS(p[n] or 0, *self.stride) for n in "qkv")
        what = 0 if form == "fwd" else 1 if p["kept"] is None else 2
        need = lib.sdm_linear_attention_workspace_bytes(sh, what)
        ex = _Exec(None, p["ws"], max(need, 256) if self.ws_bytes is None else self.ws_bytes, None, 0, None)
        head = (sh, q, k, v, p["g"], self.per_token, p["state"])
        if form == "fwd":
            rc = lib.sdm_linear_attention_fwd(*head, p["state_out"], p["valid"], p["out"], p["kept"], r(ex))
        elif form == "step":
            rc = lib.sdm_linear_attention_step(*head, p["state_out"], p["ids"], self.slots, p["valid"], p["out"], r(ex))
        else:
            gr = D._GRADS(*(p[n] or 0 for n in ("gq", "gk", "gv")), 0, *(p[n] or 0 for n in ("gg", "gstate")))
            rc = lib.sdm_linear_attention_bwd(*head, p["valid"], p["go"], p["gs"], p["kept"], gr, r(ex))
        return rc, lib.sdm_last_error().decode()


@pytest.mark.parametrize("form", ["fwd", "step", "bwd"])
@pytest.mark.parametrize("field,value,code", [
    ("streams", 0, SHAPE), ("tokens", -1, SHAPE), ("key_heads", 0, SHAPE), ("value_heads", 0, SHAPE), ("value_heads", 3, SHAPE),
    ("head_dim", 0, SHAPE), ("head_dim", 257, RANGE), ("value_dim", 0, SHAPE), ("value_dim", 65537, RANGE), ("dtype", 2, DTYPE),
    ("streams", 1 << 23, RANGE), ("tokens", (1 << 30) + 1, RANGE)])
def test_shapes(lib, form, field, value, code):
    c = Attention(lib)
    c.shape[field] = value
    rc, msg = c.run(form)
    assert rc == code and msg


def test_value_dim(lib):
    """Sequences take value_dim up to 256, single tokens up to 65536."""
    for form, code in (("fwd", RANGE), ("bwd", RANGE), ("step", NULL)):
        c = Attention(lib)
        c.shape["value_dim"] = 257
        c.ptr["q"] = None      # a shape that is accepted gives NULL
        assert c.run(form)[0] == code


@pytest.mark.parametrize("form,name", [(f, n) for f in ("fwd", "step", "bwd") for n in ("q", "k", "v", "g")]
                         + [("fwd", "out"), ("step", "out"), ("step", "state"), ("step", "state_out"), ("bwd", "go"),
                            ("bwd", "gq"), ("bwd", "gk"), ("bwd", "gv")])
def test_nulls(lib, form, name):
    c = Attention(lib)
    c.ptr[name] = None
    rc, msg = c.run(form)
    assert rc == NULL and msg


@pytest.mark.parametrize("form,name,off,dtype", [
    ("fwd", "q", 2, 0), ("fwd", "k", 1, 1), ("step", "v", 1, 1), ("bwd", "g", 2, 1), ("fwd", "state", 2, 1),
    ("fwd", "state_out", 1, 0), ("fwd", "valid", 2, 0), ("step", "ids", 2, 0), ("bwd", "gq", 1, 1), ("bwd", "gg", 2, 1),
    ("fwd", "ws", 16, 0), ("bwd", "ws", 128, 0), ("bwd", "gs", 2, 0), ("fwd", "out", 1, 1)])
def test_alignment(lib, form, name, off, dtype):
    c = Attention(lib)
    c.shape["dtype"] = dtype
    c.ptr[name] += off
    rc, msg = c.run(form)
    assert rc == ALIGN and msg
    for form in ("fwd", "bwd"):
        c = Attention(lib)
        c.ptr["kept"] = FAKE + 64
        assert c.run(form)[0] == ALIGN


def test_workspace_overlap_slots_and_decays(lib):
    for form in ("fwd", "bwd"):
        c = Attention(lib)
        c.ws_bytes = 255
        assert c.run(form)[0] == WORKSPACE
        c = Attention(lib)
        c.ptr["ws"] = None
        assert c.run(form)[0] == WORKSPACE
    c = Attention(lib)
    c.ptr["kept"], c.ptr["ws"] = FAKE, None
    assert c.run("bwd")[0] == WORKSPACE
    for form in ("fwd", "step"):
        c = Attention(lib)
        c.ptr["state_out"] = c.ptr["state"] + 64
        assert c.run(form)[0] == SHAPE
    c = Attention(lib)
    c.ptr["gstate"] = c.ptr["gs"] - 64
    assert c.run("bwd")[0] == SHAPE
    c = Attention(lib)
    c.ptr["ids"], c.slots = None, 1
    assert c.run("step")[0] == SHAPE
    for form in ("fwd", "step", "bwd"):
        c = Attention(lib)
        c.stride[1] = -1
        assert c.run(form)[0] == SHAPE
        c = Attention(lib)
        c.per_token = 2
        assert c.run(form)[0] == SHAPE


def test_launches(lib):
    """A launch holds less than 2^32 threads: shapes past that are refused, also by the size queries."""
    def code(**shape):
        c = Attention(lib)
        c.shape |= shape
        c.ptr["q"] = None
        return c.run("fwd")[0]

    one = dict(streams=1 << 19, tokens=1, key_heads=1, value_heads=4, head_dim=16, value_dim=16)
    assert code(**one) == RANGE and code(**one | dict(value_heads=2)) == NULL                           # tokens / 64 + 4
    assert code(**one | dict(value_heads=2, head_dim=65)) == RANGE                                      # two slices
    assert code(**one | dict(streams=1 << 15, head_dim=256, value_dim=256, tokens=0)) == RANGE          # the scan: 256 blocks to a state
    assert code(streams=1, tokens=1 << 28, key_heads=1, value_heads=1, head_dim=64, value_dim=64) == NULL
    assert code(streams=1, tokens=1 << 29, key_heads=1, value_heads=1, head_dim=64, value_dim=64) == RANGE
    c = Attention(lib)
    sh = c.dense._SHAPE(*(c.shape | one).values())
    assert lib.sdm_linear_attention_workspace_bytes(sh, 0) == 0 and lib.sdm_linear_attention_kept_bytes(sh) == 0


def test_sizes(lib):
    f, k = lib.sdm_linear_attention_workspace_bytes, lib.sdm_linear_attention_kept_bytes
    c = Attention(lib)
    sh = c.dense._SHAPE(*c.shape.values())
    assert f(None, 0) == 0 and k(None) == 0 and f(sh, 3) == 0 and f(sh, -1) == 0
    sizes = [f(sh, w) for w in (0, 1, 2)] + [k(sh)]
    assert all(s >= 256 and s % 256 == 0 for s in sizes) and sizes[1] > sizes[2]


def norm(lib, bwd, samples=4, rows=5000, channels=32, groups=4, dtype=0, wdtype=0, act=1, eps=1e-5, ws_bytes=None, xs=160000, xr=32, **ptr):
    from chunked_sparse_delta_amd import _Exec, group
    p = {n: FAKE + (i << 36) for i, n in enumerate(["x", "w", "b", "y", "mean", "rstd", "dy", "dx", "dw", "db", "ws", "valid"])} | ptr
    need = lib.sdm_group_norm_workspace_bytes(group._SHAPE(4, 5000, 32, 4, 0, 0, 1, 1e-5), 1 if bwd else 0)
    assert need > 0
    ex = _Exec(None, p["ws"], need if ws_bytes is None else ws_bytes, None, 0, None)
    sh = group._SHAPE(samples, rows, channels, groups, dtype, wdtype, act, eps)
    if bwd:
        return lib.sdm_group_norm_bwd(sh, p["dy"], p["x"], xs, xr, p["w"], p["b"], p["valid"], p["mean"], p["rstd"], p["dx"], p["dw"],
                                      p["db"], ctypes.byref(ex))
    return lib.sdm_group_norm_fwd(sh, p["x"], xs, xr, p["w"], p["b"], p["valid"], p["y"], p["mean"], p["rstd"], ctypes.byref(ex))


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(samples=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(channels=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=5), SHAPE),
    (dict(samples=1 << 31), RANGE), (dict(rows=1 << 31), RANGE), (dict(channels=(1 << 20) + 4), RANGE), (dict(act=3), RANGE),
    (dict(act=-1), RANGE), (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE), (dict(dtype=2), DTYPE), (dict(wdtype=-1), DTYPE),
    (dict(dtype=0, wdtype=1), DTYPE), (dict(xr=-1), SHAPE), (dict(xs=-1), SHAPE), (dict(x=None), NULL), (dict(mean=None), NULL),
    (dict(rstd=FAKE + 2), ALIGN), (dict(dtype=1, x=FAKE + 1), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(valid=FAKE + 2), ALIGN),
    (dict(ws_bytes=16), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), ALIGN)])
def test_norm_rejects(lib, bwd, change, code):
    assert norm(lib, bwd, **change) == code
    assert lib.sdm_last_error()


def test_norm_sizes(lib):
    from chunked_sparse_delta_amd import group
    assert norm(lib, False, y=None) == NULL and norm(lib, True, dy=None) == NULL
    assert norm(lib, True, dx=FAKE + 2) == ALIGN
    f = lib.sdm_group_norm_workspace_bytes
    assert f(None, 0) == 0 and f(group._SHAPE(4, 1, 32, 5, 0, 0, 0, 0.0), 1) == 0
    assert f(group._SHAPE(4, 1, 64, 4, 0, 0, 0, 0.0), 0) == 0         # rows in registers: none
    assert f(group._SHAPE(4, 1, 64, 4, 0, 0, 0, 0.0), 1) % 256 == 0


def test_python_refusals():
    """What the bindings refuse without a GPU: types, devices, names."""
    import torch
    import chunked_sparse_delta_amd as sdm
    x = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(2)
    s = torch.zeros(1, 2, 8, 8)
    with pytest.raises(ValueError, match="expected GPU tensors"):
        sdm.linear_attention_fwd(s, x, x, g, x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sdm.linear_attention_step(s, x.half(), x.half(), g, x.half())
    with pytest.raises(TypeError, match="must be torch tensors"):
        sdm.linear_attention_fwd(s, x, x, None, x)
    with pytest.raises(ValueError, match="P, T, heads, width"):
        sdm.linear_attention_bwd(s, x[0], x[0], g, x[0], x[0])
    with pytest.raises(ValueError, match="one of"):
        sdm.linear_attention_workspace_bytes(1, 1, 1, 1, 1, 1, torch.float32, "training")
    assert sdm.linear_attention_workspace_bytes(1, 1, 1, 1, 1, 1, torch.float16) == 0
    assert sdm.linear_attention_kept_bytes(1, 300, 1, 1, 16, 16, torch.bfloat16) > 0
    with pytest.raises(ValueError, match="expected GPU tensors"):
        sdm.group_norm(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sdm.group_norm_fwd(torch.zeros(2, 8).half(), 2)
    with pytest.raises(ValueError, match="activation"):
        sdm.group_norm_fwd(torch.zeros(2, 8), 2, activation="relu")
    with pytest.raises(ValueError, match="channels"):
        sdm.group_norm_fwd(torch.zeros(8), 2)
    assert sdm.group_norm_workspace_bytes(2, 5000, 64, 4, torch.bfloat16) > 0

"""The C ABI of the dense operators on the host: include/sdm_dense.h's functions are exported and reject malformed calls
with the documented code before any device work (no GPU needed)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sdm_dense.h")

DTYPE, SHAPE, RANGE, NULL, ALIGN, WORKSPACE = -1, -2, -3, -4, -5, -6
FAKE = 0x7f0000000000     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import chunked_sparse_delta_amd as sdm
    if not os.path.exists(sdm.library_path()):
        from chunked_sparse_delta_amd import build
        build.build()
    return sdm._load()


def test_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sdm_\w+)\s*\(", text)))
    assert names == ["sdm_gated_delta_bwd", "sdm_gated_delta_bwd_kept", "sdm_gated_delta_fwd", "sdm_gated_delta_fwd_keep",
                     "sdm_gated_delta_step", "sdm_gated_delta_workspace_bytes",
                     "sdm_layer_norm_bwd", "sdm_layer_norm_bwd_workspace_bytes", "sdm_layer_norm_fwd"]
    assert all(hasattr(lib, n) for n in names)


class Delta:
    def __init__(self, lib):
        from chunked_sparse_delta_amd import dense
        self.lib, self.dense = lib, dense
        self.shape = dict(streams=2, tokens=100, key_heads=2, value_heads=4, head_dim=64, value_dim=32, dtype=0, scale=1.0)
        self.ptr = {n: FAKE + (i << 36) for i, n in enumerate(
            ["q", "k", "v", "beta", "g", "state", "state_out", "valid", "out", "ws", "ids", "go", "gs", "gq", "gk", "gv",
             "gbeta", "gg", "gstate"])}
        self.stride, self.ws_bytes, self.slots = [1 << 16, 1 << 9, 1 << 6], None, 2

    def run(self, form):
        from chunked_sparse_delta_amd import _Exec
        D, r, lib = self.dense, ctypes.byref, self.lib
        sh = D._SHAPE(*self.shape.values())
        q, k, v = (D._ROWS(self.ptr[n] or 0, *self.stride) for n in "qkv")
        need = lib.sdm_gated_delta_workspace_bytes(sh, 1 if form == "bwd" else 0)
        ex = _Exec(None, self.ptr["ws"], max(need, 256) if self.ws_bytes is None else self.ws_bytes, None, 0, None)
        p = self.ptr
        head = (sh, q, k, v, p["beta"], p["g"], p["state"])
        if form == "fwd":
            rc = lib.sdm_gated_delta_fwd(*head, p["state_out"], p["valid"], p["out"], r(ex))
        elif form == "step":
            rc = lib.sdm_gated_delta_step(*head, p["state_out"], p["ids"], self.slots, p["valid"], p["out"], r(ex))
        else:
            gr = D._GRADS(*(p[n] or 0 for n in ("gq", "gk", "gv", "gbeta", "gg", "gstate")))
            rc = lib.sdm_gated_delta_bwd(*head, p["valid"], p["go"], p["gs"], gr, r(ex))
        return rc, lib.sdm_last_error().decode()


@pytest.mark.parametrize("form", ["fwd", "step", "bwd"])
@pytest.mark.parametrize("field,value,code", [
    ("streams", 0, SHAPE), ("tokens", -1, SHAPE), ("key_heads", 0, SHAPE), ("value_heads", 0, SHAPE), ("value_heads", 3, SHAPE),
    ("head_dim", 0, SHAPE), ("head_dim", 257, RANGE), ("value_dim", 0, SHAPE), ("value_dim", 65537, RANGE), ("dtype", 2, DTYPE),
    ("streams", 1 << 23, RANGE), ("tokens", (1 << 30) + 1, RANGE)])
def test_delta_shapes(lib, form, field, value, code):
    c = Delta(lib)
    c.shape[field] = value
    rc, msg = c.run(form)
    assert rc == code and msg


@pytest.mark.parametrize("form,name", [(f, n) for f in ("fwd", "step", "bwd") for n in ("q", "k", "v", "beta", "g")]
                         + [("fwd", "out"), ("step", "out"), ("step", "state"), ("step", "state_out"), ("bwd", "go"),
                            ("bwd", "gq"), ("bwd", "gk"), ("bwd", "gv"), ("bwd", "gbeta"), ("bwd", "gg")])
def test_delta_nulls(lib, form, name):
    c = Delta(lib)
    c.ptr[name] = None
    rc, msg = c.run(form)
    assert rc == NULL and msg


@pytest.mark.parametrize("form,name,off,dtype", [
    ("fwd", "q", 2, 0), ("fwd", "k", 1, 1), ("step", "v", 1, 1), ("bwd", "beta", 2, 1), ("fwd", "state", 2, 1),
    ("fwd", "state_out", 1, 0), ("fwd", "valid", 2, 0), ("step", "ids", 2, 0), ("bwd", "gq", 1, 1), ("bwd", "gg", 2, 1),
    ("fwd", "ws", 16, 0), ("bwd", "ws", 128, 0), ("bwd", "gs", 2, 0), ("fwd", "out", 1, 1)])
def test_delta_alignment(lib, form, name, off, dtype):
    c = Delta(lib)
    c.shape["dtype"] = dtype
    c.ptr[name] += off
    rc, msg = c.run(form)
    assert rc == ALIGN and msg


def test_delta_workspace_overlap_and_slots(lib):
    for form in ("fwd", "bwd"):
        c = Delta(lib)
        c.ws_bytes = 255
        assert c.run(form)[0] == WORKSPACE
        c = Delta(lib)
        c.ptr["ws"] = None
        assert c.run(form)[0] == WORKSPACE
    for form in ("fwd", "step"):
        c = Delta(lib)
        c.ptr["state_out"] = c.ptr["state"] + 64
        assert c.run(form)[0] == SHAPE
    c = Delta(lib)
    c.ptr["gstate"] = c.ptr["gs"] - 64
    assert c.run("bwd")[0] == SHAPE
    c = Delta(lib)
    c.ptr["ids"], c.slots = None, 1
    assert c.run("step")[0] == SHAPE
    c = Delta(lib)
    c.stride[1] = -1
    assert c.run("fwd")[0] == SHAPE


def norm(lib, bwd, rows=4, cols=32, dtype=0, wdtype=0, eps=1e-5, ws_bytes=None, **ptr):
    from chunked_sparse_delta_amd import _Exec
    p = {n: FAKE + (i << 36) for i, n in enumerate(["x", "w", "b", "y", "mean", "rstd", "dy", "dx", "dw", "db", "ws"])} | ptr
    need = lib.sdm_layer_norm_bwd_workspace_bytes(4, 32, 0)
    ex = _Exec(None, p["ws"], need if ws_bytes is None else ws_bytes, None, 0, None)
    if bwd:
        return lib.sdm_layer_norm_bwd(rows, cols, p["dy"], p["x"], dtype, p["w"], wdtype, p["mean"], p["rstd"], p["dx"], p["dw"],
                                      p["db"], ctypes.byref(ex))
    return lib.sdm_layer_norm_fwd(rows, cols, p["x"], dtype, p["w"], p["b"], wdtype, eps, p["y"], p["mean"], p["rstd"],
                                  ctypes.byref(ex))


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(rows=1 << 31), RANGE), (dict(cols=(1 << 24) + 1), RANGE),
    (dict(dtype=2), DTYPE), (dict(wdtype=-1), DTYPE), (dict(dtype=0, wdtype=1), DTYPE), (dict(x=None), NULL),
    (dict(mean=None), NULL), (dict(rstd=FAKE + 2), ALIGN), (dict(dtype=1, x=FAKE + 1), ALIGN), (dict(w=FAKE + 2), ALIGN)])
def test_norm_rejects(lib, bwd, change, code):
    assert norm(lib, bwd, **change) == code
    assert lib.sdm_last_error()


def test_norm_eps_workspace_and_sizes(lib):
    assert norm(lib, False, eps=-1.0) == RANGE and norm(lib, False, eps=float("nan")) == RANGE
    assert norm(lib, False, y=None) == NULL and norm(lib, True, dy=None) == NULL
    assert norm(lib, True, ws_bytes=16) == WORKSPACE and norm(lib, True, ws=None) == WORKSPACE
    assert norm(lib, True, ws=FAKE + 16) == ALIGN
    f = lib.sdm_layer_norm_bwd_workspace_bytes
    assert f(-1, 32, 0) == 0 and f(4, 0, 0) == 0 and f(4, 32, 7) == 0
    assert f(4, 32, 0) > 0 and f(4, 32, 0) % 256 == 0
    g = lib.sdm_gated_delta_workspace_bytes
    assert g(None, 0) == 0

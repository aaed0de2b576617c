"""The dense gated delta rule and layer norm: the binding of libsdm.so's entry points of these (include/sdm_dense.h).

    out = gated_delta_fwd(state, k, v, beta, log_decay, q)       # sequences; state advanced in place
    out = gated_delta_step(state, k, v, beta, log_decay, q)      # one or a few tokens, a pool of states
    grads = gated_delta_bwd(state0, k, v, beta, log_decay, q, grad_out)
    out, state = gated_delta_rule(state0, k, v, beta, log_decay, q)   # autograd

    y, mean, rstd = layer_norm_fwd(x, weight, bias)
    grads = layer_norm_bwd(grad_out, x, mean, rstd, weight)
    y = layer_norm(x, weight, bias)                               # autograd

The rule, per stream and value head with a float32 state S of [K, V]:
    S' = exp(g) S;  u = beta (v - k S');  S = S' + k u;  out = scale q S
Shapes: k, q [P, T, Hk, K]; v, out [P, T, Hv, V]; beta, log_decay float32 [P, T, Hv]; state float32 [P, Hv, K, V].
Value head h reads key head h // (Hv // Hk). k, q and v are float32 or bfloat16 and may be strided views whose last axis
is dense (slices of one projection); everything else is contiguous. ``valid_tokens`` (int32 [P] on the GPU): tokens at and
past it are padding, they leave the state alone and read 0. ``scale`` defaults to K ** -0.5.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _DTYPES, _Exec, _check_rc, _expect, _load, _ptr, _stream_ptr

__all__ = ["gated_delta_fwd", "gated_delta_step", "gated_delta_bwd", "gated_delta_rule", "gated_delta_workspace_bytes",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm"]


class _Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("streams", "tokens", "key_heads", "value_heads", "head_dim", "value_dim",
                                               "dtype")] + [("scale", ctypes.c_float)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stream", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class _DeltaGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "beta", "log_decay", "state")]


def bind(lib) -> None:
    """Declares the signatures (called once, when the library is loaded)."""
    i32, i64, f32, p, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    lib.sdm_gated_delta_workspace_bytes.argtypes = [p, i32]
    lib.sdm_gated_delta_workspace_bytes.restype = sz
    lib.sdm_gated_delta_fwd.argtypes = [p] * 11
    lib.sdm_gated_delta_step.argtypes = [p] * 9 + [i64, p, p, p]
    lib.sdm_gated_delta_bwd.argtypes = [p] * 12
    lib.sdm_layer_norm_fwd.argtypes = [i64, i32, p, i32, p, p, i32, f32, p, p, p, p]
    lib.sdm_layer_norm_bwd_workspace_bytes.argtypes = [i64, i32, i32]
    lib.sdm_layer_norm_bwd_workspace_bytes.restype = sz
    lib.sdm_layer_norm_bwd.argtypes = [i64, i32, p, p, i32, p, i32, p, p, p, p, p, p]
    for fn in (lib.sdm_gated_delta_fwd, lib.sdm_gated_delta_step, lib.sdm_gated_delta_bwd, lib.sdm_layer_norm_fwd,
               lib.sdm_layer_norm_bwd):
        fn.restype = ctypes.c_int


def _on(device: torch.device) -> None:
    """Calls run on the current device: the tensors have to be there."""
    if device.type != "cuda":
        raise ValueError(f"expected GPU tensors, got {device}")
    if device.index is not None and device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")


def _used_on(stream, *tensors) -> None:
    """Tensors made here (on the current stream's pool) but used on the caller's stream stay whole until that work ends."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _exec(stream, workspace=None) -> _Exec:
    if workspace is None:
        return _Exec(_stream_ptr(stream), None, 0, None, 0, None)
    if workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    return _Exec(_stream_ptr(stream), workspace.data_ptr(), workspace.numel() * workspace.element_size(), None, 0, None)


def _view(t: torch.Tensor, name: str, shape, dtype, device) -> _Rows:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, v on {device}")
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the last axis must be dense, its stride is {s[3]}")
    return _Rows(t.data_ptr(), s[0], s[1], s[2])


def _rule_inputs(state, k, v, beta, log_decay, q, scale, valid_tokens):
    if not isinstance(v, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError("k and v must be torch tensors")
    if v.dtype not in _DTYPES:
        raise TypeError(f"v must be float32 or bfloat16, got {v.dtype}")
    if v.dim() != 4 or k.dim() != 4:
        raise ValueError(f"k and v must be [P, T, heads, width], got {tuple(k.shape)} and {tuple(v.shape)}")
    dev = v.device
    _on(dev)
    P, T, Hv, V = v.shape
    Hk, K = k.shape[2:]
    if Hk < 1 or Hv % Hk:
        raise ValueError(f"the value heads ({Hv}) must be a multiple of the key heads ({Hk})")
    kr, qr = (_view(t, n, (P, T, Hk, K), v.dtype, dev) for t, n in ((k, "k"), (q, "q")))
    vr = _view(v, "v", v.shape, v.dtype, dev)
    for t, n in ((beta, "beta"), (log_decay, "log_decay")):
        _expect(t, n, (P, T, Hv), torch.float32, dev)
    if valid_tokens is not None:
        _expect(valid_tokens, "valid_tokens", (P,), torch.int32, dev)
    shape = _Shape(P, T, Hk, Hv, K, V, _DTYPES[v.dtype], K ** -0.5 if scale is None else float(scale))
    return shape, qr, kr, vr, dev


def _out(out, v):
    if out is None:
        return torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _expect(out, "out", tuple(v.shape), v.dtype, v.device)
    return out


def gated_delta_workspace_bytes(P: int, T: int, Hk: int, Hv: int, K: int, V: int, dtype: torch.dtype,
                                backward: bool = False) -> int:
    """Bytes of scratch gated_delta_fwd (or gated_delta_bwd) needs; 0 for shapes they reject."""
    return int(_load().sdm_gated_delta_workspace_bytes(ctypes.byref(_Shape(P, T, Hk, Hv, K, V, _DTYPES.get(dtype, -1), 1.0)),
                                                       1 if backward else 0))


def _scratch(lib, shape, backward, device):
    n = lib.sdm_gated_delta_workspace_bytes(ctypes.byref(shape), backward)
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=device)


def gated_delta_fwd(state, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, log_decay: torch.Tensor,
                    q: torch.Tensor, *, scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                    state_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The rule over whole sequences; returns the readings [P, T, Hv, V]. ``state`` is advanced in place, or left as it
    is where ``state_out`` is given, which then gets the final state. ``state=None`` starts from zeros (the final state
    goes to ``state_out`` if given). ``workspace`` (uint8, GPU, gated_delta_workspace_bytes) is allocated if omitted."""
    lib = _load()
    shape, qr, kr, vr, dev = _rule_inputs(state, k, v, beta, log_decay, q, scale, valid_tokens)
    full = (shape.streams, shape.value_heads, shape.head_dim, shape.value_dim)
    for t, n in ((state, "state"), (state_out, "state_out")):
        if t is not None:
            _expect(t, n, full, torch.float32, dev)
    made = [] if out is not None else [0]
    out = _out(out, v)
    if made:
        _used_on(stream, out)
    if workspace is None:
        workspace = _scratch(lib, shape, 0, dev)
        _used_on(stream, workspace)
    ex = _exec(stream, workspace)
    rc = lib.sdm_gated_delta_fwd(ctypes.byref(shape), ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr), _ptr(beta),
                                 _ptr(log_decay), _ptr(state), _ptr(state if state_out is None else state_out),
                                 _ptr(valid_tokens), _ptr(out), ctypes.byref(ex))
    _check_rc(lib, rc)
    return out


def gated_delta_step(state: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                     log_decay: torch.Tensor, q: torch.Tensor, *, state_ids: torch.Tensor | None = None,
                     scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                     state_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """The rule for one token of each stream, or a few (T small): every state is read and written once. ``state``
    [slots, Hv, K, V] is a pool; ``state_ids`` (int32 [P], distinct) names each stream's slot, an id outside the pool
    an idle stream, which reads 0; without it stream p has slot p. The states are advanced in place, or written to
    ``state_out`` (the same shape; slots that no stream names are left alone there)."""
    lib = _load()
    shape, qr, kr, vr, dev = _rule_inputs(state, k, v, beta, log_decay, q, scale, valid_tokens)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a [slots, Hv, K, V] tensor")
    full = (state.shape[0], shape.value_heads, shape.head_dim, shape.value_dim)
    _expect(state, "state", full, torch.float32, dev)
    if state_out is None:
        state_out = state
    else:
        _expect(state_out, "state_out", full, torch.float32, dev)
    if state_ids is not None:
        _expect(state_ids, "state_ids", (shape.streams,), torch.int32, dev)
    made = out is None
    out = _out(out, v)
    if made:
        _used_on(stream, out)
    ex = _exec(stream)
    rc = lib.sdm_gated_delta_step(ctypes.byref(shape), ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr), _ptr(beta),
                                  _ptr(log_decay), _ptr(state), _ptr(state_out), _ptr(state_ids), full[0],
                                  _ptr(valid_tokens), _ptr(out), ctypes.byref(ex))
    _check_rc(lib, rc)
    return out


def gated_delta_bwd(state, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, log_decay: torch.Tensor,
                    q: torch.Tensor, grad_out: torch.Tensor, *, grad_state: torch.Tensor | None = None,
                    scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Backward of gated_delta_fwd from the ``state`` it STARTED from (None: zeros). ``grad_out`` [P, T, Hv, V] is the
    gradient of the readings, ``grad_state`` (float32, optional) that of the final state. Returns dict(state, k, v, beta,
    log_decay, q): k, v and q in the inputs' dtype (sums over sharing heads in float32), the others float32."""
    lib = _load()
    shape, qr, kr, vr, dev = _rule_inputs(state, k, v, beta, log_decay, q, scale, valid_tokens)
    P, T, Hk, Hv, K, V = shape.streams, shape.tokens, shape.key_heads, shape.value_heads, shape.head_dim, shape.value_dim
    _expect(grad_out, "grad_out", (P, T, Hv, V), v.dtype, dev)
    for t, n in ((state, "state"), (grad_state, "grad_state")):
        if t is not None:
            _expect(t, n, (P, Hv, K, V), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(state=torch.empty((P, Hv, K, V), **f32), k=torch.empty((P, T, Hk, K), dtype=v.dtype, device=dev),
             v=torch.empty((P, T, Hv, V), dtype=v.dtype, device=dev), beta=torch.empty((P, T, Hv), **f32),
             log_decay=torch.empty((P, T, Hv), **f32), q=torch.empty((P, T, Hk, K), dtype=v.dtype, device=dev))
    _used_on(stream, *g.values())
    if workspace is None:
        workspace = _scratch(lib, shape, 1, dev)
        _used_on(stream, workspace)
    gr = _DeltaGrads(*(g[n].data_ptr() for n in ("q", "k", "v", "beta", "log_decay", "state")))
    ex = _exec(stream, workspace)
    rc = lib.sdm_gated_delta_bwd(ctypes.byref(shape), ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr), _ptr(beta),
                                 _ptr(log_decay), _ptr(state), _ptr(valid_tokens), _ptr(grad_out), _ptr(grad_state),
                                 ctypes.byref(gr), ctypes.byref(ex))
    _check_rc(lib, rc)
    return g


class _GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, state, k, v, beta, log_decay, q, scale, valid_tokens):
        final = torch.empty((v.shape[0], v.shape[2], k.shape[3], v.shape[3]), dtype=torch.float32, device=v.device)
        out = gated_delta_fwd(state, k, v, beta, log_decay, q, scale=scale, valid_tokens=valid_tokens, state_out=final)
        ctx.save_for_backward(state, k, v, beta, log_decay, q, valid_tokens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    def backward(ctx, grad_out, grad_state):
        state, k, v, beta, log_decay, q, valid = ctx.saved_tensors
        if grad_out is None and grad_state is None:
            return (None,) * 8
        go = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if grad_out is None else grad_out.contiguous()
        gs = None if grad_state is None else grad_state.contiguous()
        g = gated_delta_bwd(state, k, v, beta, log_decay, q, go, grad_state=gs, scale=ctx.scale, valid_tokens=valid)
        names = ("state", "k", "v", "beta", "log_decay", "q")
        return (*(g[n] if need else None for n, need in zip(names, ctx.needs_input_grad)), None, None)


def gated_delta_rule(state, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, log_decay: torch.Tensor,
                     q: torch.Tensor, *, scale: float | None = None, valid_tokens: torch.Tensor | None = None):
    """The rule for autograd: returns (readings, final state); ``state`` (None: zeros) is not changed. Gradients reach
    the state, k, v, beta, log_decay and q through gated_delta_bwd, which computes the forward again from its inputs."""
    return _GatedDeltaRule.apply(state, k, v, beta, log_decay, q, scale, valid_tokens)


# ---- layer norm ------------------------------------------------------------------------------------------------------

def _norm_inputs(x, params):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must be [..., cols], got {tuple(x.shape)}")
    _on(x.device)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    N = x.shape[-1]
    wdtype = None
    for t, n in params:
        if t is not None:
            if t.dtype not in _DTYPES or (wdtype is not None and t.dtype != wdtype):
                raise TypeError(f"{n}: expected {wdtype or 'float32 or bfloat16'}, got {t.dtype}")
            wdtype = t.dtype
            _expect(t, n, (N,), wdtype, x.device)
    return x.numel() // N, N, wdtype


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                   eps: float = 1e-5, out: torch.Tensor | None = None, stream=None):
    """Layer norm over the last axis of a contiguous x (float32 or bfloat16); weight and bias [cols] in x's dtype or
    float32, or None. Returns (y, mean, rstd); mean and rstd float32 [rows] are what layer_norm_bwd needs."""
    lib = _load()
    rows, N, wdtype = _norm_inputs(x, ((weight, "weight"), (bias, "bias")))
    made = out is None
    if made:
        out = torch.empty_like(x)
    else:
        _expect(out, "out", tuple(x.shape), x.dtype, x.device)
    mean, rstd = torch.empty((2, rows), dtype=torch.float32, device=x.device)
    _used_on(stream, out if made else None, mean, rstd)
    ex = _exec(stream)
    rc = lib.sdm_layer_norm_fwd(rows, N, _ptr(x), _DTYPES[x.dtype], _ptr(weight), _ptr(bias),
                                _DTYPES[wdtype or x.dtype], eps, _ptr(out), _ptr(mean), _ptr(rstd), ctypes.byref(ex))
    _check_rc(lib, rc)
    return out, mean, rstd


def layer_norm_bwd(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, *, weight_dtype: torch.dtype | None = None,
                   need: tuple = ("x", "weight", "bias"), workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Backward of layer_norm_fwd: dict(x, weight, bias) of the gradients named in ``need``. The weight's and bias's are
    in ``weight_dtype`` (default: the weight's dtype, or x's)."""
    lib = _load()
    rows, N, wdtype = _norm_inputs(x, ((weight, "weight"),))
    wdtype = weight_dtype or wdtype or x.dtype
    if wdtype not in _DTYPES or (weight is not None and weight.dtype != wdtype):
        raise TypeError(f"weight_dtype {wdtype} does not go with the weight")
    dev = x.device
    _expect(grad_out, "grad_out", tuple(x.shape), x.dtype, dev)
    for t, n in ((mean, "mean"), (rstd, "rstd")):
        _expect(t, n, (rows,), torch.float32, dev)
    if set(need) - {"x", "weight", "bias"}:
        raise ValueError(f"need names x, weight and bias, got {need}")
    g = {"x": torch.empty_like(x) if "x" in need else None}
    for n in ("weight", "bias"):
        g[n] = torch.empty((N,), dtype=wdtype, device=dev) if n in need else None
    _used_on(stream, *g.values())
    if workspace is None and (g["weight"] is not None or g["bias"] is not None):
        workspace = torch.empty(lib.sdm_layer_norm_bwd_workspace_bytes(rows, N, _DTYPES[x.dtype]), dtype=torch.uint8,
                                device=dev)
        _used_on(stream, workspace)
    ex = _exec(stream, workspace)
    rc = lib.sdm_layer_norm_bwd(rows, N, _ptr(grad_out), _ptr(x), _DTYPES[x.dtype], _ptr(weight), _DTYPES[wdtype],
                                _ptr(mean), _ptr(rstd), _ptr(g["x"]), _ptr(g["weight"]), _ptr(g["bias"]),
                                ctypes.byref(ex))
    _check_rc(lib, rc)
    return {n: t for n, t in g.items() if t is not None}


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    def backward(ctx, grad_out):
        x, weight, mean, rstd = ctx.saved_tensors
        need = tuple(n for n, on in zip(("x", "weight", "bias"), ctx.needs_input_grad) if on)
        g = layer_norm_bwd(grad_out.contiguous(), x, mean, rstd, weight,
                           weight_dtype=ctx.bias_dtype if weight is None else None, need=need)
        return g.get("x"), g.get("weight"), g.get("bias"), None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm for autograd (layer_norm_fwd, its backward layer_norm_bwd)."""
    return _LayerNorm.apply(x, weight, bias, eps)

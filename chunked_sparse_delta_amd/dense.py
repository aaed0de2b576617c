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
import struct

import torch
from torch.autograd.function import once_differentiable

from . import _DTYPES, _check_rc, _expect, _load, _stream_ptr

__all__ = ["gated_delta_fwd", "gated_delta_step", "gated_delta_bwd", "gated_delta_rule", "gated_delta_workspace_bytes",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm"]

# The ABI's structures, packed: a call of a few microseconds' work notices what building ctypes objects costs.
_SHAPE = struct.Struct("@7if").pack            # sdm_delta_shape
_ROWS = struct.Struct("@P3q").pack             # sdm_rows
_EXEC = struct.Struct("@PPNPiPi").pack         # sdm_exec
_GRADS = struct.Struct("@6P").pack             # sdm_delta_grads


def bind(lib) -> None:
    """Declares the signatures (called once, when the library is loaded)."""
    i32, i64, f32, p, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    lib.sdm_gated_delta_workspace_bytes.argtypes = [p, i32]
    lib.sdm_gated_delta_workspace_bytes.restype = sz
    lib.sdm_gated_delta_fwd.argtypes = [p] * 11
    lib.sdm_gated_delta_step.argtypes = [p] * 9 + [i64, p, p, p]
    lib.sdm_gated_delta_bwd.argtypes = [p] * 12
    lib.sdm_gated_delta_fwd_keep.argtypes = [p] * 11
    lib.sdm_gated_delta_bwd_kept.argtypes = [p] * 12
    lib.sdm_layer_norm_fwd.argtypes = [i64, i32, p, i32, p, p, i32, f32, p, p, p, p]
    lib.sdm_layer_norm_bwd_workspace_bytes.argtypes = [i64, i32, i32]
    lib.sdm_layer_norm_bwd_workspace_bytes.restype = sz
    lib.sdm_layer_norm_bwd.argtypes = [i64, i32, p, p, i32, p, i32, p, p, p, p, p, p]
    for fn in (lib.sdm_gated_delta_fwd, lib.sdm_gated_delta_step, lib.sdm_gated_delta_bwd, lib.sdm_gated_delta_fwd_keep,
               lib.sdm_gated_delta_bwd_kept, lib.sdm_layer_norm_fwd, lib.sdm_layer_norm_bwd):
        fn.restype = ctypes.c_int


_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(device: torch.device) -> int:
    """Calls run on the current device: the tensors have to be there. Returns its index."""
    if device.type != "cuda":
        raise ValueError(f"expected GPU tensors, got {device}")
    index = _current_device()
    if device.index != index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{index}")
    return index


def _new(shape, dtype, dev, stream):
    """A new tensor for work on ``stream``, in that stream's memory: whatever used the memory before did so in that stream's
    order. The caller may use it on the current stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(here)
    return t


def _exec(stream, index, workspace=None) -> bytes:
    if stream is None:
        s = _raw_stream(index) if _raw_stream is not None else _stream_ptr(None).value or 0
    else:
        s = stream.cuda_stream
    if workspace is None:
        return _EXEC(s, 0, 0, 0, 0, 0, 0)
    if workspace.device.type != "cuda" or workspace.device.index != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
    return _EXEC(s, workspace.data_ptr(), workspace.numel() * workspace.element_size(), 0, 0, 0, 0)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, shape, dtype, dev) -> None:
    """_expect's checks, without the words while they pass."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous()):
        _expect(t, name, shape, dtype, dev)


def _view(t, name, shape, dtype, dev) -> bytes:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, v on {dev}")
    p, tok, head, one = t.stride()
    if one != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the last axis must be dense, its stride is {one}")
    return _ROWS(t.data_ptr(), p, tok, head)


def _rule_inputs(k, v, beta, log_decay, q, scale, valid_tokens):
    if not isinstance(v, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError("k and v must be torch tensors")
    dtype, dev, vs, ks = v.dtype, v.device, v.shape, k.shape
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"v must be float32 or bfloat16, got {dtype}")
    if len(vs) != 4 or len(ks) != 4:
        raise ValueError(f"k and v must be [P, T, heads, width], got {tuple(ks)} and {tuple(vs)}")
    index = _on(dev)
    P, T, Hv, V = vs
    Hk, K = ks[2], ks[3]
    if Hk < 1 or Hv % Hk:
        raise ValueError(f"the value heads ({Hv}) must be a multiple of the key heads ({Hk})")
    keys, gates = (P, T, Hk, K), (P, T, Hv)
    kr, qr, vr = _view(k, "k", keys, dtype, dev), _view(q, "q", keys, dtype, dev), _view(v, "v", vs, dtype, dev)
    _need(beta, "beta", gates, torch.float32, dev)
    _need(log_decay, "log_decay", gates, torch.float32, dev)
    if valid_tokens is not None:
        _need(valid_tokens, "valid_tokens", (P,), torch.int32, dev)
    shape = _SHAPE(P, T, Hk, Hv, K, V, code, K ** -0.5 if scale is None else scale)
    return (P, Hv, K, V), shape, qr, kr, vr, dev, index


def _out(out, v, stream):
    if out is None:
        out = _new(v.shape, v.dtype, v.device, stream)   # dense whatever v's strides are
    else:
        _need(out, "out", v.shape, v.dtype, v.device)
    return out


def gated_delta_workspace_bytes(P: int, T: int, Hk: int, Hv: int, K: int, V: int, dtype: torch.dtype,
                                backward: bool = False) -> int:
    """Bytes of scratch gated_delta_fwd (or gated_delta_bwd) needs; 0 for shapes they reject."""
    return _load().sdm_gated_delta_workspace_bytes(_SHAPE(P, T, Hk, Hv, K, V, _DTYPES.get(dtype, -1), 1.0), 1 if backward else 0)


def _scratch(lib, shape, backward, dev, stream):
    return _new((max(lib.sdm_gated_delta_workspace_bytes(shape, backward), 256),), torch.uint8, dev, stream)


def gated_delta_fwd(state, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, log_decay: torch.Tensor,
                    q: torch.Tensor, *, scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                    state_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, keep: bool = False, stream=None) -> torch.Tensor:
    """The rule over whole sequences; returns the readings [P, T, Hv, V]. ``state`` is advanced in place, or left as it
    is where ``state_out`` is given, which then gets the final state. ``state=None`` starts from zeros (the final state
    goes to ``state_out`` if given). ``workspace`` (uint8, GPU, gated_delta_workspace_bytes) is allocated if omitted.
    ``keep``: the given workspace, of the backward's size, keeps what gated_delta_bwd(kept=workspace) then does not compute
    again."""
    lib = _load()
    full, shape, qr, kr, vr, dev, index = _rule_inputs(k, v, beta, log_decay, q, scale, valid_tokens)
    if keep and workspace is None:
        raise ValueError("keep needs a workspace (gated_delta_workspace_bytes(..., backward=True))")
    if state is not None:
        _need(state, "state", full, torch.float32, dev)
    if state_out is None:
        state_out = state
    else:
        _need(state_out, "state_out", full, torch.float32, dev)
    out = _out(out, v, stream)
    if workspace is None:
        workspace = _scratch(lib, shape, 0, dev, stream)
    call = lib.sdm_gated_delta_fwd_keep if keep else lib.sdm_gated_delta_fwd
    rc = call(shape, qr, kr, vr, beta.data_ptr(), log_decay.data_ptr(), _ptr(state), _ptr(state_out), _ptr(valid_tokens),
              out.data_ptr(), _exec(stream, index, workspace))
    if rc:
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
    full, shape, qr, kr, vr, dev, index = _rule_inputs(k, v, beta, log_decay, q, scale, valid_tokens)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a [slots, Hv, K, V] tensor")
    slots = state.shape[0]
    pool = (slots, *full[1:])
    _need(state, "state", pool, torch.float32, dev)
    if state_out is None:
        state_out = state
    else:
        _need(state_out, "state_out", pool, torch.float32, dev)
    if state_ids is not None:
        _need(state_ids, "state_ids", full[:1], torch.int32, dev)
    out = _out(out, v, stream)
    rc = lib.sdm_gated_delta_step(shape, qr, kr, vr, beta.data_ptr(), log_decay.data_ptr(), state.data_ptr(),
                                  state_out.data_ptr(), _ptr(state_ids), slots, _ptr(valid_tokens), out.data_ptr(),
                                  _exec(stream, index))
    if rc:
        _check_rc(lib, rc)
    return out


def gated_delta_bwd(state, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, log_decay: torch.Tensor,
                    q: torch.Tensor, grad_out: torch.Tensor, *, grad_state: torch.Tensor | None = None,
                    scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, kept: torch.Tensor | None = None, stream=None) -> dict:
    """Backward of gated_delta_fwd from the ``state`` it STARTED from (None: zeros). ``grad_out`` [P, T, Hv, V] is the
    gradient of the readings, ``grad_state`` (float32, optional) that of the final state. Returns dict(state, k, v, beta,
    log_decay, q): k, v and q in the inputs' dtype (sums over sharing heads in float32), the others float32. ``kept``: the
    workspace of a gated_delta_fwd(keep=True) with the same inputs, in place of ``workspace``; without it the forward is
    computed again."""
    lib = _load()
    full, shape, qr, kr, vr, dev, index = _rule_inputs(k, v, beta, log_decay, q, scale, valid_tokens)
    _need(grad_out, "grad_out", v.shape, v.dtype, dev)
    for t, n in ((state, "state"), (grad_state, "grad_state")):
        if t is not None:
            _need(t, n, full, torch.float32, dev)
    f32 = torch.float32
    g = {n: _new(size, dtype, dev, stream) for n, size, dtype in (
        ("state", full, f32), ("k", k.shape, k.dtype), ("v", v.shape, v.dtype), ("beta", beta.shape, f32),
        ("log_decay", beta.shape, f32), ("q", q.shape, q.dtype))}
    if kept is not None:
        workspace = kept
    elif workspace is None:
        workspace = _scratch(lib, shape, 1, dev, stream)
    call = lib.sdm_gated_delta_bwd if kept is None else lib.sdm_gated_delta_bwd_kept
    rc = call(shape, qr, kr, vr, beta.data_ptr(), log_decay.data_ptr(), _ptr(state), _ptr(valid_tokens), grad_out.data_ptr(),
              _ptr(grad_state), _GRADS(*(g[n].data_ptr() for n in ("q", "k", "v", "beta", "log_decay", "state"))),
              _exec(stream, index, workspace))
    if rc:
        _check_rc(lib, rc)
    return g


class _GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, state, k, v, beta, log_decay, q, scale, valid_tokens, recompute):
        P, T, Hv, V = v.shape
        Hk, K = k.shape[2:]
        final = torch.empty((P, Hv, K, V), dtype=torch.float32, device=v.device)
        kept = None
        if not recompute and any(ctx.needs_input_grad):
            n = gated_delta_workspace_bytes(P, T, Hk, Hv, K, V, v.dtype, True)
            kept = torch.empty(max(n, 256), dtype=torch.uint8, device=v.device)     # 0: the call itself reports why
        out = gated_delta_fwd(state, k, v, beta, log_decay, q, scale=scale, valid_tokens=valid_tokens, state_out=final,
                              workspace=kept, keep=kept is not None)
        ctx.save_for_backward(state, k, v, beta, log_decay, q, valid_tokens, kept)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_state):
        state, k, v, beta, log_decay, q, valid, kept = ctx.saved_tensors
        if grad_out is None and grad_state is None:
            return (None,) * 9
        go = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if grad_out is None else grad_out.contiguous()
        gs = None if grad_state is None else grad_state.contiguous()
        g = gated_delta_bwd(state, k, v, beta, log_decay, q, go, grad_state=gs, scale=ctx.scale, valid_tokens=valid, kept=kept)
        names = ("state", "k", "v", "beta", "log_decay", "q")
        return (*(g[n] if need else None for n, need in zip(names, ctx.needs_input_grad)), None, None, None)


def gated_delta_rule(state, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, log_decay: torch.Tensor,
                     q: torch.Tensor, *, scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                     recompute: bool = False):
    """The rule for autograd: returns (readings, final state); ``state`` (None: zeros) is not changed. Gradients reach
    the state, k, v, beta, log_decay and q through gated_delta_bwd. Until the backward the forward keeps what it computed
    per chunk (gated_delta_workspace_bytes(..., backward=True)); ``recompute=True`` keeps the inputs alone and computes the
    forward again, for less memory and about a sixth more time."""
    return _GatedDeltaRule.apply(state, k, v, beta, log_decay, q, scale, valid_tokens, recompute)


# ---- layer norm ------------------------------------------------------------------------------------------------------

def _norm_inputs(x, weight, bias):
    """rows, cols, x's and the parameters' dtype codes, the device index."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code, dev = _DTYPES.get(x.dtype), x.device
    if code is None:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must be [..., cols], got {tuple(x.shape)}")
    index = _on(dev)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    N = x.shape[-1]
    wdtype = None
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            if wdtype is None:
                wdtype = t.dtype
                if wdtype not in _DTYPES:
                    raise TypeError(f"{n}: expected float32 or bfloat16, got {wdtype}")
            _need(t, n, (N,), wdtype, dev)
    return x.numel() // N, N, code, wdtype, index


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                   eps: float = 1e-5, out: torch.Tensor | None = None, stream=None):
    """Layer norm over the last axis of a contiguous x (float32 or bfloat16); weight and bias [cols] in x's dtype or
    float32, or None. Returns (y, mean, rstd); mean and rstd float32 [rows] are what layer_norm_bwd needs."""
    lib = _load()
    rows, N, code, wdtype, index = _norm_inputs(x, weight, bias)
    if out is None:
        out = torch.empty_like(x) if stream is None else _new(x.shape, x.dtype, x.device, stream)
    else:
        _need(out, "out", x.shape, x.dtype, x.device)
    if stream is None:
        mean = x.new_empty((rows,), dtype=torch.float32)
        rstd = torch.empty_like(mean)
    else:
        mean, rstd = _new((rows,), torch.float32, x.device, stream), _new((rows,), torch.float32, x.device, stream)
    rc = lib.sdm_layer_norm_fwd(rows, N, x.data_ptr(), code, _ptr(weight), _ptr(bias), code if wdtype is None else _DTYPES[wdtype],
                                eps, out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _exec(stream, index))
    if rc:
        _check_rc(lib, rc)
    return out, mean, rstd


def layer_norm_bwd(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, *, weight_dtype: torch.dtype | None = None,
                   need: tuple = ("x", "weight", "bias"), workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Backward of layer_norm_fwd: dict(x, weight, bias) of the gradients named in ``need``. The weight's and bias's are
    in ``weight_dtype`` (default: the weight's dtype, or x's)."""
    lib = _load()
    rows, N, code, wdtype, index = _norm_inputs(x, weight, None)
    wdtype = weight_dtype or wdtype or x.dtype
    if wdtype not in _DTYPES or (weight is not None and weight.dtype != wdtype):
        raise TypeError(f"weight_dtype {wdtype} does not go with the weight")
    dev = x.device
    _need(grad_out, "grad_out", x.shape, x.dtype, dev)
    _need(mean, "mean", (rows,), torch.float32, dev)
    _need(rstd, "rstd", (rows,), torch.float32, dev)
    g = {}
    for n in need:
        if n == "x":
            g[n] = torch.empty_like(x) if stream is None else _new(x.shape, x.dtype, dev, stream)
        elif n in ("weight", "bias"):
            g[n] = _new((N,), wdtype, dev, stream)
        else:
            raise ValueError(f"need names x, weight and bias, got {need}")
    if workspace is None and ("weight" in g or "bias" in g):
        workspace = _new((lib.sdm_layer_norm_bwd_workspace_bytes(rows, N, code),), torch.uint8, dev, stream)
    rc = lib.sdm_layer_norm_bwd(rows, N, grad_out.data_ptr(), x.data_ptr(), code, _ptr(weight), _DTYPES[wdtype],
                                mean.data_ptr(), rstd.data_ptr(), _ptr(g.get("x")), _ptr(g.get("weight")), _ptr(g.get("bias")),
                                _exec(stream, index, workspace))
    if rc:
        _check_rc(lib, rc)
    return g


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
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

"""Linear attention with a decay for each head: the binding of libsdm.so's entry points of it (include/sdm_linear.h).

    out = linear_attention_fwd(state, k, v, log_decay, q)        # sequences; state advanced in place
    out = linear_attention_step(state, k, v, log_decay, q)       # one or a few tokens, a pool of states
    grads = linear_attention_bwd(state0, k, v, log_decay, q, grad_out)
    out, state = linear_attention(state0, k, v, log_decay, q)    # autograd

Per stream and value head, with a float32 state S of [K, V] (the gated delta rule without its correction):
    S = exp(g) S + k v;  out = scale q S
Shapes: k, q [P, T, Hk, K]; v, out [P, T, Hv, V]; state float32 [P, Hv, K, V]; log_decay float32 [Hv], a decay for each
head, or [P, T, Hv], one for each token. Value head h reads key head h // (Hv // Hk). k, q and v are float32 or bfloat16
and may be strided views whose last axis is dense; everything else is contiguous. ``valid_tokens`` (int32 [P] on the GPU):
tokens at and past it are padding, they leave the state alone and read 0. ``scale`` defaults to K ** -0.5.
"""

from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _DTYPES, _check_rc, _load
from .dense import _GRADS, _SHAPE, _exec, _need, _new, _on, _out, _ptr, _view

__all__ = ["linear_attention_fwd", "linear_attention_step", "linear_attention_bwd", "linear_attention",
           "linear_attention_workspace_bytes", "linear_attention_kept_bytes"]

_WORK = {"forward": 0, "backward": 1, "backward_kept": 2}      # SDM_LINEAR_*


def bind(lib) -> None:
    """Declares the signatures (called once, when the library is loaded)."""
    i32, i64, p, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    lib.sdm_linear_attention_workspace_bytes.argtypes = [p, i32]
    lib.sdm_linear_attention_kept_bytes.argtypes = [p]
    lib.sdm_linear_attention_workspace_bytes.restype = lib.sdm_linear_attention_kept_bytes.restype = sz
    lib.sdm_linear_attention_fwd.argtypes = [p] * 5 + [i32] + [p] * 6
    lib.sdm_linear_attention_step.argtypes = [p] * 5 + [i32, p, p, p, i64, p, p, p]
    lib.sdm_linear_attention_bwd.argtypes = [p] * 5 + [i32] + [p] * 7
    for fn in (lib.sdm_linear_attention_fwd, lib.sdm_linear_attention_step, lib.sdm_linear_attention_bwd):
        fn.restype = ctypes.c_int


def _inputs(k, v, log_decay, q, scale, valid_tokens):
    if not isinstance(v, torch.Tensor) or not isinstance(k, torch.Tensor) or not isinstance(log_decay, torch.Tensor):
        raise TypeError("k, v and log_decay must be torch tensors")
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
    keys = (P, T, Hk, K)
    kr, qr, vr = _view(k, "k", keys, dtype, dev), _view(q, "q", keys, dtype, dev), _view(v, "v", vs, dtype, dev)
    per_token = log_decay.dim() != 1
    _need(log_decay, "log_decay", (P, T, Hv) if per_token else (Hv,), torch.float32, dev)
    if valid_tokens is not None:
        _need(valid_tokens, "valid_tokens", (P,), torch.int32, dev)
    shape = _SHAPE(P, T, Hk, Hv, K, V, code, K ** -0.5 if scale is None else scale)
    return (P, Hv, K, V), (shape, qr, kr, vr, log_decay.data_ptr(), 1 if per_token else 0), dev, index


def linear_attention_workspace_bytes(P: int, T: int, Hk: int, Hv: int, K: int, V: int, dtype: torch.dtype,
                                     what: str = "forward") -> int:
    """Bytes of scratch that linear_attention_fwd ("forward") or linear_attention_bwd ("backward", or "backward_kept" with
    ``kept``) needs; 0 for shapes they reject."""
    if what not in _WORK:
        raise ValueError(f"what must be one of {tuple(_WORK)}, got {what!r}")
    return _load().sdm_linear_attention_workspace_bytes(_SHAPE(P, T, Hk, Hv, K, V, _DTYPES.get(dtype, -1), 1.0), _WORK[what])


def linear_attention_kept_bytes(P: int, T: int, Hk: int, Hv: int, K: int, V: int, dtype: torch.dtype) -> int:
    """Bytes that a forward with ``kept`` leaves for the backward; 0 for shapes they reject."""
    return _load().sdm_linear_attention_kept_bytes(_SHAPE(P, T, Hk, Hv, K, V, _DTYPES.get(dtype, -1), 1.0))


def _buffer(t, name, least, dev):
    """Checks a caller's buffer for what a forward keeps."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or not t.is_contiguous() or t.numel() * t.element_size() < least:
        raise ValueError(f"{name} must be a contiguous tensor of {least} bytes on {dev}")


def linear_attention_fwd(state, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, q: torch.Tensor, *,
                         scale: float | None = None, valid_tokens: torch.Tensor | None = None,
                         state_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, kept: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Linear attention over whole sequences; returns the readings [P, T, Hv, V]. ``state`` is advanced in place, or left
    as it is where ``state_out`` is given, which then gets the final state. ``state=None`` starts from zeros (the final
    state goes to ``state_out`` if given). ``workspace`` (uint8, GPU, linear_attention_workspace_bytes) is allocated if
    omitted. ``kept`` (uint8, GPU, linear_attention_kept_bytes) gets what linear_attention_bwd(kept=kept) then does not
    compute again."""
    lib = _load()
    plan = _inputs(k, v, log_decay, q, scale, valid_tokens)
    full, head, dev, _ = plan
    if state is not None:
        _need(state, "state", full, torch.float32, dev)
    if state_out is None:
        state_out = state
    else:
        _need(state_out, "state_out", full, torch.float32, dev)
    out = _out(out, v, stream)
    if kept is not None:
        _buffer(kept, "kept", lib.sdm_linear_attention_kept_bytes(head[0]), dev)
    _values(plan, state, state_out, valid_tokens, out, kept, workspace, stream)
    return out


def _values(plan, state, state_out, valid_tokens, out, kept, workspace=None, stream=None):
    """linear_attention_fwd of checked arguments."""
    lib = _load()
    _, head, dev, index = plan
    if workspace is None and kept is None:
        workspace = _new((max(lib.sdm_linear_attention_workspace_bytes(head[0], 0), 256),), torch.uint8, dev, stream)
    rc = lib.sdm_linear_attention_fwd(*head, _ptr(state), _ptr(state_out), _ptr(valid_tokens), out.data_ptr(), _ptr(kept),
                                      _exec(stream, index, workspace))
    if rc:
        _check_rc(lib, rc)


def linear_attention_step(state: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                          q: torch.Tensor, *, state_ids: torch.Tensor | None = None, scale: float | None = None,
                          valid_tokens: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                          out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Linear attention for one token of each stream, or a few (T small): every state is read and written once. ``state``
    [slots, Hv, K, V] is a pool; ``state_ids`` (int32 [P], distinct) names each stream's slot, an id outside the pool an
    idle stream, which reads 0; without it stream p has slot p. The states are advanced in place, or written to
    ``state_out`` (the same shape; slots that no stream names are left alone there)."""
    lib = _load()
    full, head, dev, index = _inputs(k, v, log_decay, q, scale, valid_tokens)
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
    rc = lib.sdm_linear_attention_step(*head, state.data_ptr(), state_out.data_ptr(), _ptr(state_ids), slots,
                                       _ptr(valid_tokens), out.data_ptr(), _exec(stream, index))
    if rc:
        _check_rc(lib, rc)
    return out


def linear_attention_bwd(state, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, q: torch.Tensor,
                         grad_out: torch.Tensor, *, grad_state: torch.Tensor | None = None, scale: float | None = None,
                         valid_tokens: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         kept: torch.Tensor | None = None, need: tuple = ("state", "k", "v", "log_decay", "q"),
                         stream=None) -> dict:
    """Backward of linear_attention_fwd from the ``state`` it STARTED from (None: zeros). ``grad_out`` [P, T, Hv, V] is the
    gradient of the readings, ``grad_state`` (float32, optional) that of the final state. Returns dict(state, k, v,
    log_decay, q): k, v and q (always there) in the inputs' dtype (sums over sharing heads in float32), state and log_decay
    float32, where ``need`` names them. ``kept``: what a linear_attention_fwd(kept=...) with the same inputs left; without
    it the states are computed again."""
    plan = _inputs(k, v, log_decay, q, scale, valid_tokens)
    full, head, dev, _ = plan
    _need(grad_out, "grad_out", v.shape, v.dtype, dev)
    for t, n in ((state, "state"), (grad_state, "grad_state")):
        if t is not None:
            _need(t, n, full, torch.float32, dev)
    for n in need:
        if n not in ("state", "k", "v", "log_decay", "q"):
            raise ValueError(f"need names state, k, v, log_decay and q, got {need}")
    if kept is not None:
        _buffer(kept, "kept", _load().sdm_linear_attention_kept_bytes(head[0]), dev)
    return _grads(plan, state, k, v, log_decay, q, grad_out, grad_state, valid_tokens, kept, need, workspace, stream)


def _grads(plan, state, k, v, log_decay, q, grad_out, grad_state, valid_tokens, kept, need, workspace=None, stream=None):
    """linear_attention_bwd of checked arguments."""
    lib = _load()
    full, head, dev, index = plan
    f32 = torch.float32
    g = {"k": _new(k.shape, k.dtype, dev, stream), "v": _new(v.shape, v.dtype, dev, stream), "q": _new(q.shape, q.dtype, dev, stream)}
    if "state" in need:
        g["state"] = _new(full, f32, dev, stream)
    if "log_decay" in need:
        g["log_decay"] = _new(log_decay.shape, f32, dev, stream)
    if workspace is None:
        n = lib.sdm_linear_attention_workspace_bytes(head[0], 1 if kept is None else 2)
        workspace = _new((max(n, 256),), torch.uint8, dev, stream)
    rc = lib.sdm_linear_attention_bwd(*head, _ptr(state), _ptr(valid_tokens), grad_out.data_ptr(), _ptr(grad_state), _ptr(kept),
                                      _GRADS(g["q"].data_ptr(), g["k"].data_ptr(), g["v"].data_ptr(), 0,
                                             _ptr(g.get("log_decay")) or 0, _ptr(g.get("state")) or 0),
                                      _exec(stream, index, workspace))
    if rc:
        _check_rc(lib, rc)
    return g


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, state, k, v, log_decay, q, scale, valid_tokens, recompute):
        ctx.plan = plan = _inputs(k, v, log_decay, q, scale, valid_tokens)
        full, head, dev, _ = plan
        if state is not None:
            _need(state, "state", full, torch.float32, dev)
        final = torch.empty(full, dtype=torch.float32, device=dev)
        kept = None
        if not recompute and any(ctx.needs_input_grad):
            n = _load().sdm_linear_attention_kept_bytes(head[0])
            kept = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)     # 0: the call itself reports why
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
        _values(plan, state, final, valid_tokens, out, kept)
        ctx.save_for_backward(state, k, v, log_decay, q, valid_tokens, kept)
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_state):
        state, k, v, log_decay, q, valid, kept = ctx.saved_tensors
        if grad_out is None and grad_state is None:
            return (None,) * 8
        go = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if grad_out is None else grad_out.contiguous()
        gs = None if grad_state is None else grad_state.contiguous()
        wants = ctx.needs_input_grad
        need = [n for n, on in (("state", wants[0]), ("log_decay", wants[3])) if on]
        g = _grads(ctx.plan, state, k, v, log_decay, q, go, gs, valid, kept, need)
        return (g.get("state"), g["k"] if wants[1] else None, g["v"] if wants[2] else None, g.get("log_decay"),
                g["q"] if wants[4] else None, None, None, None)


def linear_attention(state, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, q: torch.Tensor, *,
                     scale: float | None = None, valid_tokens: torch.Tensor | None = None, recompute: bool = False):
    """Linear attention for autograd: returns (readings, final state); ``state`` (None: zeros) is not changed. Gradients
    reach the state, k, v, log_decay and q through linear_attention_bwd. Until the backward the forward keeps the states
    between segments of tokens (linear_attention_kept_bytes); ``recompute=True`` keeps the inputs alone."""
    return _LinearAttention.apply(state, k, v, log_decay, q, scale, valid_tokens, recompute)

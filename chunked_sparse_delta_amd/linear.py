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
Given tensors that a call writes (``state``, ``state_out``, ``out``, ``kept``) count as written to autograd: a backward that saved one
of them is refused. They must not overlap an input but where it is said.
"""

from __future__ import annotations

import ctypes
import threading

import torch

from . import _DTYPES, SdmError, _load
from .dense import _SHAPE

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


_lock = threading.Lock()
_module = None


def _binding():
    """The binding's C++ part (csrc/binding.cpp), with the loaded library's functions."""
    global _module
    if _module is None:
        lib = _load()
        with _lock:
            if _module is None:
                try:
                    from . import _binding as module
                except ImportError as e:
                    raise RuntimeError(f"_binding.so cannot be loaded ({e}): build it first "
                                       "(python -m chunked_sparse_delta_amd.build)") from e
                names = ["sdm_linear_attention_fwd", "sdm_linear_attention_step", "sdm_linear_attention_bwd",
                         "sdm_linear_attention_workspace_bytes", "sdm_linear_attention_kept_bytes", "sdm_group_norm_fwd",
                         "sdm_group_norm_bwd", "sdm_group_norm_workspace_bytes", "sdm_last_error"]
                module.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names}, SdmError)
                _module = module
    return _module


def _on(stream, call, *args):
    """``call`` on ``stream``: what it allocates comes from that stream's memory (whatever used it before did so in that
    stream's order); the caller may use the results on the current stream."""
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        got = call(*args)
    for t in (got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)):
        t.record_stream(here)
    return got


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
    call = _binding().linear_attention_fwd
    if stream is not None:
        return _on(stream, call, state, k, v, log_decay, q, scale, valid_tokens, state_out, out, workspace, kept)
    return call(state, k, v, log_decay, q, scale, valid_tokens, state_out, out, workspace, kept)


def linear_attention_step(state: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                          q: torch.Tensor, *, state_ids: torch.Tensor | None = None, scale: float | None = None,
                          valid_tokens: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                          out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Linear attention for one token of each stream, or a few (T small): every state is read and written once. ``state``
    [slots, Hv, K, V] is a pool; ``state_ids`` (int32 [P], distinct) names each stream's slot, an id outside the pool an
    idle stream, which reads 0; without it stream p has slot p. The states are advanced in place, or written to
    ``state_out`` (the same shape; slots that no stream names are left alone there). ``out`` may be v where that is dense."""
    call = _binding().linear_attention_step
    if stream is not None:
        return _on(stream, call, state, k, v, log_decay, q, state_ids, scale, valid_tokens, state_out, out)
    return call(state, k, v, log_decay, q, state_ids, scale, valid_tokens, state_out, out)


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
    call = _binding().linear_attention_bwd
    args = (state, k, v, log_decay, q, grad_out, grad_state, scale, valid_tokens, workspace, kept, list(need))
    return call(*args) if stream is None else _on(stream, call, *args)


def linear_attention(state, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, q: torch.Tensor, *,
                     scale: float | None = None, valid_tokens: torch.Tensor | None = None, recompute: bool = False):
    """Linear attention for autograd: returns (readings, final state); ``state`` (None: zeros) is not changed. Gradients
    reach the state, k, v, log_decay and q through linear_attention_bwd. Until the backward the forward keeps the states
    between segments of tokens (linear_attention_kept_bytes; the start state may then be advanced before the backward);
    ``recompute=True`` keeps the inputs alone. Under no_grad nothing is kept. A backward captured into a graph needs leaves that
    no eager autograd graph holds any longer (autograd would join that one's stream into the capture)."""
    return _binding().linear_attention(state, k, v, log_decay, q, scale, valid_tokens, recompute)

"""Group norm with an activation, channels last: the binding of libsdm.so's entry points of it (include/sdm_linear.h).

    y, mean, rstd = group_norm_fwd(x, groups, weight, bias, activation="silu")
    grads = group_norm_bwd(grad_out, x, groups, mean, rstd, weight, bias, activation="silu")
    y = group_norm(x, groups, weight, bias, activation="silu")                     # autograd

x [N, ..., C] (float32 or bfloat16): per sample and group of C / groups neighbouring channels, over all axes between,
    y = act((x - mean) / sqrt(var + eps) * weight + bias)
with act None, "silu" or "gelu" (z Phi(z)). [N, C] has one row to a sample: each head's norm of a token's readings. x may be
a view whose last axis is dense and whose middle axes count as one (a slice of a projection); weight and bias are [C], in
x's dtype or float32, or None. ``valid_rows`` (int32 [N] on the GPU): rows (of the middle axes) at and past it are
padding, they do not count and give 0.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import _DTYPES, _load
from .linear import _binding, _on

__all__ = ["group_norm_fwd", "group_norm_bwd", "group_norm", "group_norm_workspace_bytes"]

_SHAPE = struct.Struct("@2q5if").pack       # sdm_group_shape
_ACTS = {None: 0, "silu": 1, "gelu": 2}     # SDM_ACT_*


def bind(lib) -> None:
    """Declares the signatures (called once, when the library is loaded)."""
    i32, i64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    lib.sdm_group_norm_workspace_bytes.argtypes = [p, i32]
    lib.sdm_group_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.sdm_group_norm_fwd.argtypes = [p, p, i64, i64] + [p] * 7
    lib.sdm_group_norm_bwd.argtypes = [p, p, p, i64, i64] + [p] * 9
    lib.sdm_group_norm_fwd.restype = lib.sdm_group_norm_bwd.restype = ctypes.c_int


def _act(activation) -> int:
    code = _ACTS.get(activation)
    if code is None:
        raise ValueError(f"activation must be None, 'silu' or 'gelu', got {activation!r}")
    return code


def group_norm_workspace_bytes(N: int, rows: int, channels: int, groups: int, dtype: torch.dtype, backward: bool = False) -> int:
    """Bytes of scratch that group_norm_fwd (or group_norm_bwd) needs; 0 where none, and for shapes they reject (samples cut
    into 2^24 blocks or more among them)."""
    shape = _SHAPE(N, rows, channels, groups, _DTYPES.get(dtype, -1), 0, 0, 0.0)
    return _load().sdm_group_norm_workspace_bytes(shape, 1 if backward else 0)


def group_norm_fwd(x: torch.Tensor, groups: int, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                   activation: str | None = None, eps: float = 1e-5, valid_rows: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Group norm and activation. Returns (y, mean, rstd); mean and rstd float32 [N, groups] are what group_norm_bwd needs.
    ``out`` may be x where that is contiguous (autograd counts it as written), and must not overlap an input otherwise. ``workspace`` (uint8, GPU, group_norm_workspace_bytes) is allocated if
    omitted and needed."""
    call = _binding().group_norm_fwd
    if stream is not None:
        return _on(stream, call, x, groups, weight, bias, _act(activation), eps, valid_rows, out, workspace)
    return call(x, groups, weight, bias, _act(activation), eps, valid_rows, out, workspace)


def group_norm_bwd(grad_out: torch.Tensor, x: torch.Tensor, groups: int, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *, activation: str | None = None,
                   eps: float = 1e-5, valid_rows: torch.Tensor | None = None, need: tuple = ("x", "weight", "bias"),
                   workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Backward of group_norm_fwd: dict(x, weight, bias) of the gradients named in ``need``; the weight's and bias's in
    their dtype (x's where both are None)."""
    call = _binding().group_norm_bwd
    args = (grad_out, x, groups, mean, rstd, weight, bias, _act(activation), eps, valid_rows, list(need), workspace)
    return call(*args) if stream is None else _on(stream, call, *args)


def group_norm(x: torch.Tensor, groups: int, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               activation: str | None = None, eps: float = 1e-5, valid_rows: torch.Tensor | None = None) -> torch.Tensor:
    """Group norm and activation for autograd (group_norm_fwd, its backward group_norm_bwd). Captured into a graph: see
    linear_attention."""
    return _binding().group_norm(x, groups, weight, bias, _act(activation), eps, valid_rows)

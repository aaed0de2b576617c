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
from torch.autograd.function import once_differentiable

from . import _DTYPES, _check_rc, _load
from .dense import _exec, _need, _new, _on, _ptr

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


def _inputs(x, groups, weight, bias, activation, eps, valid_rows, wdtype=None):
    """The shape's bytes, x's pointer and strides, the parameters' dtype, the device, its index."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code, dev = _DTYPES.get(x.dtype), x.device
    if code is None:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() < 2 or x.shape[-1] < 1:
        raise ValueError(f"x must be [N, ..., channels], got {tuple(x.shape)}")
    if activation not in _ACTS:
        raise ValueError(f"activation must be None, 'silu' or 'gelu', got {activation!r}")
    index = _on(dev)
    N, C = x.shape[0], x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"the channels ({C}) must be a multiple of the groups ({groups})")
    if x.dim() == 3:
        rows = x
    elif x.dim() == 2:
        rows = x[:, None]
    elif x.numel() == 0:
        rows = x.new_empty((N, x[0, ..., 0].numel() if N else 0, C))
    else:
        try:
            rows = x.view(N, -1, C)
        except RuntimeError:
            raise ValueError(f"x: its axes between the first and the last must count as one, strides {x.stride()}") from None
    L = rows.shape[1]
    sample, row, one = rows.stride()
    if one != 1 and C > 1:
        raise ValueError(f"x: the last axis must be dense, its stride is {one}")
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            if wdtype is None:
                wdtype = t.dtype
                if wdtype not in _DTYPES:
                    raise TypeError(f"{n}: expected float32 or bfloat16, got {wdtype}")
            _need(t, n, (C,), wdtype, dev)
    if wdtype is None:
        wdtype = x.dtype
    if valid_rows is not None:
        _need(valid_rows, "valid_rows", (N,), torch.int32, dev)
    shape = _SHAPE(N, L, C, groups, code, _DTYPES[wdtype], _ACTS[activation], eps)
    return shape, (x.data_ptr(), sample, row), wdtype, dev, index


def group_norm_workspace_bytes(N: int, rows: int, channels: int, groups: int, dtype: torch.dtype, backward: bool = False) -> int:
    """Bytes of scratch that group_norm_fwd (or group_norm_bwd) needs; 0 where none, and for shapes they reject."""
    shape = _SHAPE(N, rows, channels, groups, _DTYPES.get(dtype, -1), 0, 0, 0.0)
    return _load().sdm_group_norm_workspace_bytes(shape, 1 if backward else 0)


def _scratch(lib, shape, backward, workspace, dev, stream):
    if workspace is None:
        n = lib.sdm_group_norm_workspace_bytes(shape, backward)
        if n:
            workspace = _new((n,), torch.uint8, dev, stream)
    return workspace


def group_norm_fwd(x: torch.Tensor, groups: int, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                   activation: str | None = None, eps: float = 1e-5, valid_rows: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Group norm and activation. Returns (y, mean, rstd); mean and rstd float32 [N, groups] are what group_norm_bwd needs.
    ``workspace`` (uint8, GPU, group_norm_workspace_bytes) is allocated if omitted and needed."""
    plan = _inputs(x, groups, weight, bias, activation, eps, valid_rows)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, plan[3])
    return _values(plan, x, groups, weight, bias, valid_rows, out, workspace, stream)


def _values(plan, x, groups, weight, bias, valid_rows, out=None, workspace=None, stream=None):
    """group_norm_fwd of checked arguments."""
    lib = _load()
    shape, rows, _, dev, index = plan
    if out is None:
        out = _new(x.shape, x.dtype, dev, stream)     # dense whatever x's strides are
    size = (x.shape[0], groups)
    mean, rstd = _new(size, torch.float32, dev, stream), _new(size, torch.float32, dev, stream)
    workspace = _scratch(lib, shape, 0, workspace, dev, stream)
    rc = lib.sdm_group_norm_fwd(shape, *rows, _ptr(weight), _ptr(bias), _ptr(valid_rows), out.data_ptr(), mean.data_ptr(),
                                rstd.data_ptr(), _exec(stream, index, workspace))
    if rc:
        _check_rc(lib, rc)
    return out, mean, rstd


def group_norm_bwd(grad_out: torch.Tensor, x: torch.Tensor, groups: int, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *, activation: str | None = None,
                   eps: float = 1e-5, valid_rows: torch.Tensor | None = None, need: tuple = ("x", "weight", "bias"),
                   workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Backward of group_norm_fwd: dict(x, weight, bias) of the gradients named in ``need``; the weight's and bias's in
    their dtype (x's where both are None)."""
    plan = _inputs(x, groups, weight, bias, activation, eps, valid_rows)
    dev = plan[3]
    _need(grad_out, "grad_out", x.shape, x.dtype, dev)
    for t, n in ((mean, "mean"), (rstd, "rstd")):
        _need(t, n, (x.shape[0], groups), torch.float32, dev)
    for n in need:
        if n not in ("x", "weight", "bias"):
            raise ValueError(f"need names x, weight and bias, got {need}")
    return _grads(plan, grad_out, x, mean, rstd, weight, bias, valid_rows, need, workspace, stream)


def _grads(plan, grad_out, x, mean, rstd, weight, bias, valid_rows, need, workspace=None, stream=None):
    """group_norm_bwd of checked arguments."""
    lib = _load()
    shape, rows, wdtype, dev, index = plan
    g = {n: _new(x.shape, x.dtype, dev, stream) if n == "x" else _new(x.shape[-1:], wdtype, dev, stream) for n in need}
    workspace = _scratch(lib, shape, 1, workspace, dev, stream)
    rc = lib.sdm_group_norm_bwd(shape, grad_out.data_ptr(), *rows, _ptr(weight), _ptr(bias), _ptr(valid_rows), mean.data_ptr(),
                                rstd.data_ptr(), _ptr(g.get("x")), _ptr(g.get("weight")), _ptr(g.get("bias")),
                                _exec(stream, index, workspace))
    if rc:
        _check_rc(lib, rc)
    return g


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups, weight, bias, activation, eps, valid_rows):
        ctx.plan = plan = _inputs(x, groups, weight, bias, activation, eps, valid_rows)
        y, mean, rstd = _values(plan, x, groups, weight, bias, valid_rows)
        ctx.save_for_backward(x, weight, bias, valid_rows, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, weight, bias, valid, mean, rstd = ctx.saved_tensors
        wants = ctx.needs_input_grad
        need = [n for n, on in (("x", wants[0]), ("weight", wants[2]), ("bias", wants[3])) if on]
        g = _grads(ctx.plan, grad_out.contiguous(), x, mean, rstd, weight, bias, valid, need)
        return g.get("x"), None, g.get("weight"), g.get("bias"), None, None, None


def group_norm(x: torch.Tensor, groups: int, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               activation: str | None = None, eps: float = 1e-5, valid_rows: torch.Tensor | None = None) -> torch.Tensor:
    """Group norm and activation for autograd (group_norm_fwd, its backward group_norm_bwd)."""
    return _GroupNorm.apply(x, groups, weight, bias, activation, eps, valid_rows)

"""Thin Python binding of the block operators of libgrkan.so (C ABI in include/grkan_block.h):
the group norm with an activation, channels last, and their autograd wrappers.

Argument marshalling only, as in binding.py: shapes, strides and pointers are
checked and handed over; every step of the computation is a HIP kernel.
Outputs and workspaces that are not given are allocated on the stream the
call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding
from .binding import GRKAN_OK, GRKANError, _check_coefs, _check_out, _io, _on_gpu, _ptr, _stream, _workspace

GRKAN_ACT_NONE, GRKAN_ACT_SILU, GRKAN_ACT_GELU, GRKAN_ACT_RATIONAL = 0, 1, 2, 3
_ACTS = {"none": GRKAN_ACT_NONE, "silu": GRKAN_ACT_SILU, "gelu": GRKAN_ACT_GELU, "rational": GRKAN_ACT_RATIONAL}

_lib = None


def _library() -> ctypes.CDLL:
    """libgrkan.so with the block operators' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load_library()
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    lib.grkan_group_norm_forward.argtypes = [vp] * 8 + [i64] * 5 + [i32, i32, f32, i32, i32, vp, sz, vp]
    lib.grkan_group_norm_forward.restype = ctypes.c_int
    lib.grkan_group_norm_backward.argtypes = [vp] * 13 + [i64] * 7 + [i32] * 4 + [vp, sz, vp]
    lib.grkan_group_norm_backward.restype = ctypes.c_int
    for name in ("forward", "backward"):
        size = getattr(lib, f"grkan_group_norm_{name}_workspace_size")
        size.argtypes = [i64, i64, i64, i32, i32, i32, i32]
        size.restype = sz
    _lib = lib
    return lib


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    return _ACTS[act]


def _scope(stream, dev):
    """Allocations and the launch belong to `stream` (the current one if None) of device dev."""
    if stream is None and dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    if stream is None:
        return torch.cuda.device(dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _act_coefs(act: int, A, B, n_groups: int, channels: int, dev):
    """(A, B, n_groups) to hand over: checked for the rational, absent for the others."""
    if act != GRKAN_ACT_RATIONAL:
        return None, None, 1
    if A is None or B is None:
        raise ValueError("the rational activation needs A and B")
    if n_groups < 1 or channels % n_groups:
        raise ValueError(f"{channels} channels are not a multiple of n_groups = {n_groups}")
    _check_coefs(A, B, n_groups, dev)
    return A, B, n_groups


def _channel_vector(t, name: str, channels: int, dev):
    if t is not None and (t.dtype != torch.float32 or t.device != dev or not t.is_contiguous()
                          or t.numel() != channels):
        raise ValueError(f"{name} must be a contiguous float32 tensor of {channels} elements on {dev}")


def _samples(t: torch.Tensor, name: str):
    """(samples, positions, channels, sample stride, position stride) of a channels-last tensor
    [samples, ..., channels] whose inner dimensions are equally spaced."""
    if t.dim() < 2:
        raise ValueError(f"{name} must be [samples, ..., channels]")
    size, stride = t.shape, t.stride()
    n, c = size[0], size[-1]
    s = 1
    for k in size[1:-1]:
        s *= k
    if t.is_contiguous():
        return n, s, c, s * c, c
    if c > 1 and stride[-1] != 1:
        raise ValueError(f"{name} must have its channels last and contiguous")
    row, run = None, 0
    for k in range(t.dim() - 2, 0, -1):
        if size[k] == 1:
            continue
        if row is None:
            row = stride[k]
        elif stride[k] != run:
            raise ValueError(f"the positions of {name} must be equally spaced")
        run = stride[k] * size[k]
    if row is None:
        row = c
    if row < c:
        raise ValueError(f"the positions of {name} must not overlap")
    return n, s, c, stride[0], row


def grkan_group_norm_forward(x: torch.Tensor, norm_groups: int, weight=None, bias=None, eps: float = 1e-5,
                             act: str = "none", A=None, B=None, n_groups: int = 8, out=None, mean=None, rstd=None,
                             workspace=None, stream=None):
    """(y, mean, rstd): y = act(group norm of x) (``grkan_group_norm_forward``).

    ``x`` is [samples, ..., channels] in float32 or bfloat16, its positions (the dimensions between)
    equally spaced: a slice of channels or of positions will do.  ``norm_groups`` = 1 on [rows, channels]
    is the norm per token.  ``weight`` and ``bias`` are float32 [channels] or None.  ``act`` is "none",
    "silu", "gelu" or "rational"; the last takes A [n_groups, 6], B [n_groups, 4].  y is dense, mean and
    rstd are float32 [samples, norm_groups], for the backward."""
    io, code = _io(x), _act(act)
    _on_gpu(x)
    n, s, c, xs, xr = _samples(x, "x")
    dev = x.device
    if norm_groups < 1 or c < 1 or c % norm_groups:
        raise ValueError(f"{c} channels are not a multiple of norm_groups = {norm_groups}")
    _channel_vector(weight, "weight", c, dev)
    _channel_vector(bias, "bias", c, dev)
    A, B, ng = _act_coefs(code, A, B, n_groups, c, dev)
    lib = _library()
    with _scope(stream, dev):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        elif out.shape != x.shape:
            raise ValueError("out must match x")
        _check_out(out, "out", x.dtype, x.numel(), dev)
        if mean is None:
            mean = torch.empty((n, norm_groups), dtype=torch.float32, device=dev)
        _check_out(mean, "mean", torch.float32, n * norm_groups, dev)
        if rstd is None:
            rstd = torch.empty((n, norm_groups), dtype=torch.float32, device=dev)
        _check_out(rstd, "rstd", torch.float32, n * norm_groups, dev)
        need = lib.grkan_group_norm_forward_workspace_size(n, s, c, norm_groups, ng, code, io)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        wsp, wsn = _workspace(workspace, dev)
        st = lib.grkan_group_norm_forward(_ptr(x), _ptr(out), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(bias),
                                          _ptr(A), _ptr(B), n, s, c, xs, xr, norm_groups, ng, eps, code, io, wsp,
                                          wsn, _stream(stream))
    if st != GRKAN_OK:
        raise GRKANError(st, "grkan_group_norm_forward")
    return out, mean, rstd


def grkan_group_norm_backward(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                              norm_groups: int, weight=None, bias=None, act: str = "none", A=None, B=None,
                              n_groups: int = 8, dx=None, dweight=None, dbias=None, dA=None, dB=None,
                              workspace=None, stream=None):
    """(dx, dweight, dbias, dA, dB) of ``grkan_group_norm_forward`` from its x, mean and rstd
    (``grkan_group_norm_backward``); dweight and dbias also without weight and bias (of ones and zeros),
    dA and dB None but for the rational."""
    io, code = _io(x), _act(act)
    _on_gpu(x)
    n, s, c, xs, xr = _samples(x, "x")
    dev = x.device
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != dev:
        raise ValueError("dy must match x")
    _, _, _, ds, dr = _samples(dy, "dy")
    if norm_groups < 1 or c < 1 or c % norm_groups:
        raise ValueError(f"{c} channels are not a multiple of norm_groups = {norm_groups}")
    _channel_vector(weight, "weight", c, dev)
    _channel_vector(bias, "bias", c, dev)
    _check_out(mean, "mean", torch.float32, n * norm_groups, dev)
    _check_out(rstd, "rstd", torch.float32, n * norm_groups, dev)
    A, B, ng = _act_coefs(code, A, B, n_groups, c, dev)
    lib = _library()
    with _scope(stream, dev):
        if dx is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        elif dx.shape != x.shape:
            raise ValueError("dx must match x")
        _check_out(dx, "dx", x.dtype, x.numel(), dev)
        if dweight is None:
            dweight = torch.empty(c, dtype=torch.float32, device=dev)
        _check_out(dweight, "dweight", torch.float32, c, dev)
        if dbias is None:
            dbias = torch.empty(c, dtype=torch.float32, device=dev)
        _check_out(dbias, "dbias", torch.float32, c, dev)
        dA, dB = _coef_grads(code, dA, dB, ng, dev)
        need = lib.grkan_group_norm_backward_workspace_size(n, s, c, norm_groups, ng, code, io)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        wsp, wsn = _workspace(workspace, dev)
        st = lib.grkan_group_norm_backward(_ptr(x), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(bias),
                                           _ptr(A), _ptr(B), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(dA),
                                           _ptr(dB), n, s, c, xs, xr, ds, dr, norm_groups, ng, code, io, wsp, wsn,
                                           _stream(stream))
    if st != GRKAN_OK:
        raise GRKANError(st, "grkan_group_norm_backward")
    return dx, dweight, dbias, dA, dB


def _coef_grads(code: int, dA, dB, n_groups: int, dev):
    if code != GRKAN_ACT_RATIONAL:
        return None, None
    if dA is None:
        dA = torch.empty((n_groups, 6), dtype=torch.float32, device=dev)
    _check_out(dA, "dA", torch.float32, n_groups * 6, dev)
    if dB is None:
        dB = torch.empty((n_groups, 4), dtype=torch.float32, device=dev)
    _check_out(dB, "dB", torch.float32, n_groups * 4, dev)
    return dA, dB


class GRKANGroupNorm(torch.autograd.Function):
    """Autograd wrapper: y = act(group norm of x), ``apply(x, norm_groups, weight, bias, eps, act, A, B,
    n_groups)``."""

    @staticmethod
    def forward(ctx, x, norm_groups, weight=None, bias=None, eps=1e-5, act="none", A=None, B=None, n_groups=8):
        y, mean, rstd = grkan_group_norm_forward(x, norm_groups, weight, bias, eps, act, A, B, n_groups)
        ctx.save_for_backward(x, weight, bias, A, B, mean, rstd)
        ctx.args = norm_groups, act, n_groups
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, A, B, mean, rstd = ctx.saved_tensors
        norm_groups, act, n_groups = ctx.args
        dx, dw, db, dA, dB = grkan_group_norm_backward(x, dy.contiguous(), mean, rstd, norm_groups, weight, bias,
                                                       act, A, B, n_groups)
        return (dx, None, None if weight is None else dw.view_as(weight), None if bias is None else db.view_as(bias),
                None, None, None if dA is None else dA.view_as(A), None if dB is None else dB.view_as(B), None)

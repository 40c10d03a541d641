"""Thin Python binding of the block operators of libgrkan.so (C ABI in include/grkan_block.h):
the group norm with an activation, channels last, the linear map with bias, activation and residual in
its epilogue, and their autograd wrappers.

Argument marshalling only, as in binding.py: shapes, strides and pointers are
checked and handed over; every step of the computation is a HIP kernel.
Outputs and workspaces that are not given are allocated on the stream the
call runs on.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .binding import GRKAN_BF16, GRKAN_F32, GRKAN_OK, GRKANError, _check_coefs, _check_out, _on_gpu, _written

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
    lib.grkan_linear_act_forward.argtypes = [vp] * 8 + [i64] * 5 + [i32, i32, vp, sz, vp]
    lib.grkan_linear_act_forward.restype = ctypes.c_int
    lib.grkan_linear_act_backward.argtypes = [vp] * 11 + [i64] * 5 + [i32, i32, vp, sz, vp]
    lib.grkan_linear_act_backward.restype = ctypes.c_int
    for name in ("forward", "backward"):
        size = getattr(lib, f"grkan_linear_act_{name}_workspace_size")
        size.argtypes = [i64, i64, i64, i32, i32]
        size.restype = sz
    _lib = lib
    return lib


@functools.lru_cache(maxsize=256)
def _need(name: str, *shape) -> int:
    """Workspace bytes of an operator, a function of its shape alone."""
    return getattr(_library(), f"grkan_{name}_workspace_size")(*shape)


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    return _ACTS[act]


# The handle of a device's current stream without a Stream object around it, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_stream(stream, dev, launch):
    """launch(handle) with allocations and kernels on `stream` (the current one if None) of device dev."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return launch(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return launch(_raw_stream(dev.index))
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return launch(stream.cuda_stream)


_IO = {torch.float32: GRKAN_F32, torch.bfloat16: GRKAN_BF16}


def _io(t: torch.Tensor) -> int:
    io = _IO.get(t.dtype)
    if io is None:
        raise TypeError(f"GR-KAN I/O dtype must be float32 or bfloat16, got {t.dtype}")
    return io


def _ptr(t):
    return None if t is None else t.data_ptr()


def _given(t, name: str, shape, dtype, dev):
    """A caller's output checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    numel = 1
    for k in shape:
        numel *= k
    _check_out(t, name, dtype, numel, dev)
    return t


def _wanted(skip, name: str, t, shape, dtype, dev):
    """A gradient's tensor as _given, or None if it is to be skipped."""
    if name not in skip:
        return _given(t, name, shape, dtype, dev)
    if t is not None:
        raise ValueError(f"{name} is given and skipped")
    return None


def _skipped(skip, names):
    if not set(skip) <= set(names):
        raise ValueError(f"skip takes names among {names}")


def _space(ws, need: int, dev):
    """(tensor, pointer, size in bytes) of the workspace: the caller's, or a new one of `need` bytes."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not ws.is_contiguous() or ws.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


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
    if out is not None and out.shape != x.shape:
        raise ValueError("out must match x")
    lib = _library()
    need = _need("group_norm_forward", n, s, c, norm_groups, ng, code, io)

    def launch(handle):
        y = _given(out, "out", x.shape, x.dtype, dev)
        mu = _given(mean, "mean", (n, norm_groups), torch.float32, dev)
        rs = _given(rstd, "rstd", (n, norm_groups), torch.float32, dev)
        ws, wsp, wsn = _space(workspace, need, dev)
        st = lib.grkan_group_norm_forward(x.data_ptr(), y.data_ptr(), mu.data_ptr(), rs.data_ptr(), _ptr(weight),
                                          _ptr(bias), _ptr(A), _ptr(B), n, s, c, xs, xr, norm_groups, ng, eps, code,
                                          io, wsp, wsn, handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_group_norm_forward")
        _written(out, mean, rstd)
        return y, mu, rs

    return _on_stream(stream, dev, launch)


def grkan_group_norm_backward(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                              norm_groups: int, weight=None, bias=None, act: str = "none", A=None, B=None,
                              n_groups: int = 8, dx=None, dweight=None, dbias=None, dA=None, dB=None,
                              workspace=None, stream=None, skip=()):
    """(dx, dweight, dbias, dA, dB) of ``grkan_group_norm_forward`` from its x, mean and rstd
    (``grkan_group_norm_backward``); dweight and dbias also without weight and bias (of ones and zeros),
    dA and dB None but for the rational.  ``skip``: names among "dweight" and "dbias" that are not computed
    (None in their place)."""
    io, code = _io(x), _act(act)
    _skipped(skip, ("dweight", "dbias"))
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
    if dx is not None and dx.shape != x.shape:
        raise ValueError("dx must match x")
    lib = _library()
    need = _need("group_norm_backward", n, s, c, norm_groups, ng, code, io)

    def launch(handle):
        gx = _given(dx, "dx", x.shape, x.dtype, dev)
        gw = _wanted(skip, "dweight", dweight, (c,), torch.float32, dev)
        gb = _wanted(skip, "dbias", dbias, (c,), torch.float32, dev)
        gA, gB = _coef_grads(code, dA, dB, ng, dev)
        ws, wsp, wsn = _space(workspace, need, dev)
        st = lib.grkan_group_norm_backward(x.data_ptr(), dy.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                           _ptr(weight), _ptr(bias), _ptr(A), _ptr(B), gx.data_ptr(), _ptr(gw),
                                           _ptr(gb), _ptr(gA), _ptr(gB), n, s, c, xs, xr, ds, dr, norm_groups,
                                           ng, code, io, wsp, wsn, handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_group_norm_backward")
        _written(dx, dweight, dbias, dA, dB)
        return gx, gw, gb, gA, gB

    return _on_stream(stream, dev, launch)


def _coef_grads(code: int, dA, dB, n_groups: int, dev):
    if code != GRKAN_ACT_RATIONAL:
        return None, None
    return (_given(dA, "dA", (n_groups, 6), torch.float32, dev), _given(dB, "dB", (n_groups, 4), torch.float32, dev))


def _rows(t: torch.Tensor, name: str, dev):
    """(rows, width, row stride) of a bf16 tensor [..., width] whose rows are equally spaced."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if t.dim() < 1:
        raise ValueError(f"{name} must be [..., width]")
    w = t.shape[-1]
    rows = 1
    for k in t.shape[:-1]:
        rows *= k
    if t.is_contiguous():
        return rows, w, w
    if w > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    row, run = None, 0
    for k in range(t.dim() - 2, -1, -1):
        if t.shape[k] == 1:
            continue
        if row is None:
            row = t.stride(k)
        elif t.stride(k) != run:
            raise ValueError(f"the rows of {name} must be equally spaced")
        run = t.stride(k) * t.shape[k]
    if row is None:
        row = w
    if row < w:
        raise ValueError(f"the rows of {name} must not overlap")
    return rows, w, row


def _linear_dims(x: torch.Tensor, W: torch.Tensor):
    _on_gpu(x)
    dev = x.device
    rows, d_in, ldx = _rows(x, "x", dev)
    if W.dtype != torch.bfloat16:
        raise TypeError(f"W must be bfloat16, got {W.dtype}")
    if W.dim() != 2 or not W.is_contiguous() or W.device != dev or W.shape[1] != d_in:
        raise ValueError(f"W must be a contiguous [d_out, {d_in}] tensor on {dev}")
    return rows, d_in, W.shape[0], ldx, dev


def grkan_linear_act_forward(x: torch.Tensor, W: torch.Tensor, bias=None, act: str = "none", A=None, B=None,
                             n_groups: int = 8, residual=None, keep: bool = False, out=None, pre=None,
                             workspace=None, stream=None):
    """(z, pre): z = act(x W^T + bias) + residual (``grkan_linear_act_forward``).

    bf16 x [..., d_in] and residual [..., d_out] with equally spaced rows, W [d_out, d_in]; float32 bias
    [d_out].  ``pre`` is the bf16 product before the activation, for the backward, if ``keep`` (or a tensor
    for it) is given, else None."""
    code = _act(act)
    rows, d_in, d_out, ldx, dev = _linear_dims(x, W)
    _channel_vector(bias, "bias", d_out, dev)
    A, B, ng = _act_coefs(code, A, B, n_groups, d_out, dev)
    shape = (*x.shape[:-1], d_out)
    ldr = 0
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual must be {list(shape)}")
        ldr = _rows(residual, "residual", dev)[2]
    lib = _library()
    need = _need("linear_act_forward", rows, d_in, d_out, ng, code)

    def launch(handle):
        z = _given(out, "out", shape, torch.bfloat16, dev)
        h = _given(pre, "pre", shape, torch.bfloat16, dev) if keep or pre is not None else None
        ws, wsp, wsn = _space(workspace, need, dev)
        st = lib.grkan_linear_act_forward(x.data_ptr(), W.data_ptr(), _ptr(bias), _ptr(residual), _ptr(A), _ptr(B),
                                          z.data_ptr(), _ptr(h), rows, d_in, d_out, ldx, ldr, ng, code, wsp, wsn,
                                          handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_linear_act_forward")
        _written(out, pre)
        return z, h

    return _on_stream(stream, dev, launch)


def grkan_linear_act_backward(x: torch.Tensor, W: torch.Tensor, dz: torch.Tensor, pre=None, act: str = "none",
                              A=None, B=None, n_groups: int = 8, dx=None, dW=None, dbias=None, dA=None, dB=None,
                              workspace=None, stream=None, skip=()):
    """(dx, dW, dbias, dA, dB) of ``grkan_linear_act_forward`` from its pre (not needed for act "none")
    (``grkan_linear_act_backward``): bf16 dx and dW, float32 dbias; dA and dB None but for the rational.
    The residual's gradient is dz.  ``skip``: names among "dx", "dW" and "dbias" that are not computed (None
    in their place)."""
    code = _act(act)
    _skipped(skip, ("dx", "dW", "dbias"))
    rows, d_in, d_out, ldx, dev = _linear_dims(x, W)
    if dz.shape != (*x.shape[:-1], d_out):
        raise ValueError(f"dz must be {[*x.shape[:-1], d_out]}")
    lddz = _rows(dz, "dz", dev)[2]
    if code == GRKAN_ACT_NONE:
        pre = None
    elif pre is None:
        raise ValueError("the backward of an activation needs the forward's pre")
    else:
        _check_out(pre, "pre", torch.bfloat16, rows * d_out, dev)
    A, B, ng = _act_coefs(code, A, B, n_groups, d_out, dev)
    lib = _library()
    need = _need("linear_act_backward", rows, d_in, d_out, ng, code)

    def launch(handle):
        gx = _wanted(skip, "dx", dx, x.shape, torch.bfloat16, dev)
        gW = _wanted(skip, "dW", dW, (d_out, d_in), torch.bfloat16, dev)
        gb = _wanted(skip, "dbias", dbias, (d_out,), torch.float32, dev)
        gA, gB = _coef_grads(code, dA, dB, ng, dev)
        ws, wsp, wsn = _space(workspace, need, dev)
        st = lib.grkan_linear_act_backward(x.data_ptr(), W.data_ptr(), dz.data_ptr(), _ptr(pre), _ptr(A), _ptr(B),
                                           _ptr(gx), _ptr(gW), _ptr(gb), _ptr(gA), _ptr(gB), rows, d_in,
                                           d_out, ldx, lddz, ng, code, wsp, wsn, handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_linear_act_backward")
        _written(dx, dW, dbias, dA, dB)
        return gx, gW, gb, gA, gB

    return _on_stream(stream, dev, launch)


def _like(grad, t):
    return None if grad is None else grad.view_as(t)


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
    @once_differentiable  # the kernels' results carry no graph: a second derivative would silently lack them
    def backward(ctx, dy):
        x, weight, bias, A, B, mean, rstd = ctx.saved_tensors
        norm_groups, act, n_groups = ctx.args
        needs = *ctx.needs_input_grad, False, False  # as many as apply was given, two at least
        skip = [name for name, i in (("dweight", 2), ("dbias", 3)) if not needs[i]]
        dx, dw, db, dA, dB = grkan_group_norm_backward(x, dy.contiguous(), mean, rstd, norm_groups, weight, bias,
                                                       act, A, B, n_groups, skip=skip)
        return dx, None, _like(dw, weight), _like(db, bias), None, None, _like(dA, A), _like(dB, B), None


class GRKANLinearAct(torch.autograd.Function):
    """Autograd wrapper: z = act(x W^T + bias) + residual, ``apply(x, W, bias, act, A, B, n_groups, residual)``.

    The product before the activation is written and kept only for a backward that reads it: not without
    gradients (``torch.no_grad``, or no input that asks for one), for act "none" or for the residual's alone."""

    @classmethod
    def apply(cls, x, W, bias=None, act="none", A=None, B=None, n_groups=8, residual=None):
        # (inside forward the grad mode is off and needs_input_grad does not know of it)
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, W, bias, A, B, residual)):
            return super().apply(x, W, bias, act, A, B, n_groups, residual)
        return grkan_linear_act_forward(x, W, bias, act, A, B, n_groups, residual)[0]

    @staticmethod
    def forward(ctx, x, W, bias=None, act="none", A=None, B=None, n_groups=8, residual=None):
        keep = act != "none" and any(ctx.needs_input_grad[:-1])
        z, pre = grkan_linear_act_forward(x, W, bias, act, A, B, n_groups, residual, keep=keep)
        ctx.save_for_backward(x, W, bias, A, B, pre)
        ctx.args = act, n_groups, residual is not None
        return z

    @staticmethod
    @once_differentiable
    def backward(ctx, dz):
        x, W, bias, A, B, pre = ctx.saved_tensors
        act, n_groups, residual = ctx.args
        if not any(ctx.needs_input_grad[:-1]):
            return (None,) * 7 + (dz,)
        dz = dz.contiguous()
        skip = [name for i, name in enumerate(("dx", "dW", "dbias")) if not ctx.needs_input_grad[i]]
        dx, dW, db, dA, dB = grkan_linear_act_backward(x, W, dz, pre, act, A, B, n_groups, skip=skip)
        return dx, dW, _like(db, bias), None, _like(dA, A), _like(dB, B), None, dz if residual else None

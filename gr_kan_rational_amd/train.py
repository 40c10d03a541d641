"""Thin Python binding of the operators that a deep stack of GR-KAN blocks is trained and served with (C ABI
in include/grkan_train.h): the 8-bit quantiser and matrix product, the residual path with its norms, the
AdamW step over many tensors; their autograd wrappers and the optimizer.

Argument marshalling only, as in block.py: every step of the computation is a HIP kernel.
"""
from __future__ import annotations

import array
import ctypes
import operator
from itertools import chain

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import binding
from .binding import GRKAN_BF16, GRKAN_F32, GRKAN_OK, GRKANError, _check_out, _on_gpu, _written
from .block import (_IO, GRKAN_ACT_NONE, GRKAN_ACT_RATIONAL, _act_coefs, _channel_vector, _given, _io, _like,
                    _need, _on_stream, _ptr, _skipped, _space, _wanted, grkan_linear_act_backward)

BLOCK = 128  # values that share a scale
F8 = torch.float8_e4m3fn
GRKAN_NORM_NONE, GRKAN_NORM_LAYER, GRKAN_NORM_RMS = 0, 1, 2
_NORMS = {"layer": GRKAN_NORM_LAYER, "rms": GRKAN_NORM_RMS}
_POSTS = {"none": GRKAN_NORM_NONE, **_NORMS}
GRKAN_FP8_SUMS_CUT = 16

_lib = None


class grkan_adamw_tensor_t(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("avg", ctypes.c_void_p), ("sq", ctypes.c_void_p), ("avg_scale", ctypes.c_void_p),
                ("sq_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("io", ctypes.c_int)]


class grkan_adamw_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("lr_ptr", ctypes.c_void_p), ("step_ptr", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p),
                ("seed", ctypes.c_uint32)]


def _library() -> ctypes.CDLL:
    """libgrkan.so with these operators' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load_library()
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    lib.grkan_fp8_quantize.argtypes = [vp] * 7 + [i64] * 7 + [i32] * 4 + [vp]
    lib.grkan_fp8_matmul.argtypes = [vp] * 7 + [i64] * 9 + [i32, i64, i32, vp, sz, vp]
    lib.grkan_fp8_matmul_workspace_size.argtypes = [i64] * 3
    lib.grkan_residual_norm_forward.argtypes = [vp] * 11 + [i64] * 6 + [f32] + [i32] * 4 + [vp]
    lib.grkan_residual_norm_backward.argtypes = [vp] * 18 + [i64] * 7 + [i32] * 4 + [vp, sz, vp]
    lib.grkan_residual_norm_backward_workspace_size.argtypes = [i64] * 4 + [i32] * 2
    lib.grkan_adamw_step.argtypes = [vp, i64, ctypes.POINTER(grkan_adamw_t), i32, vp]
    for name in ("fp8_quantize", "fp8_matmul", "residual_norm_forward", "residual_norm_backward", "adamw_step"):
        getattr(lib, f"grkan_{name}").restype = ctypes.c_int
    lib.grkan_fp8_matmul_workspace_size.restype = sz
    lib.grkan_residual_norm_backward_workspace_size.restype = sz
    _lib = lib
    return lib


# ---------------------------------------------------------------- 8 bits

def _up(n: int, d: int) -> int:
    return -(-n // d) * d


def _matrix(t: torch.Tensor, name: str, dev=None):
    """(rows, width, row stride) of [..., width] whose rows are equally spaced, any dtype."""
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    size = t.shape
    if not size:
        raise ValueError(f"{name} must be [..., width]")
    w, rows = size[-1], 1
    for k in size[:-1]:
        rows *= k
    if t.is_contiguous():
        return rows, w, w
    stride = t.stride()
    if w > 1 and stride[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    row, run = None, 0
    for k in range(len(size) - 2, -1, -1):
        if size[k] == 1:
            continue
        if row is None:
            row = stride[k]
        elif stride[k] != run:
            raise ValueError(f"the rows of {name} must be equally spaced")
        run = stride[k] * size[k]
    if row is None:
        row = w
    if row < w:
        raise ValueError(f"the rows of {name} must not overlap")
    return rows, w, row


def _codes(rows: int, cols: int, dev):
    """An e4m3 [rows, cols] tensor whose rows start 16 bytes apart or a multiple."""
    if cols % 16 == 0:
        return torch.empty((rows, cols), dtype=F8, device=dev)
    return torch.empty((rows, _up(cols, 16)), dtype=F8, device=dev)[:, :cols]


def _scales(rows: int, blocks: int, dev):
    """A float32 [rows, blocks] tensor, the rows of a block side by side."""
    return torch.empty_strided((rows, blocks), (1, max(rows, 1)), dtype=torch.float32, device=dev)


def grkan_fp8_quantize(x: torch.Tensor, outputs: str = "rows", tile: bool = False, act: str = "none", A=None, B=None,
                       n_groups: int = 8, stream=None):
    """e4m3 codes and power-of-two scales of x, or F(x), in blocks of 128 (``grkan_fp8_quantize``).

    ``x`` is float32 or bfloat16 [..., cols] with equally spaced rows.  ``outputs``: "rows" gives (q, scale)
    with q [rows, cols] and a scale [rows, cols / 128] for each 128 of a row; "columns" gives (qt, scale_t) of
    the transpose, qt [cols, rows], a scale for each 128 of a column; "both" gives all four from one read of
    x.  ``tile``: a scale for each 128 x 128, the same values in both layouts.  ``act`` "rational" takes A
    [n_groups, 6], B [n_groups, 4]."""
    if outputs not in ("rows", "columns", "both"):
        raise ValueError('outputs must be "rows", "columns" or "both"')
    if act not in ("none", "rational"):
        raise ValueError('act must be "none" or "rational"')
    io, code = _io(x), GRKAN_ACT_RATIONAL if act == "rational" else GRKAN_ACT_NONE
    _on_gpu(x)
    rows, cols, ldx = _matrix(x, "x")
    if cols < 1:
        raise ValueError("x must have a column")
    dev = x.device
    A, B, ng = _act_coefs(code, A, B, n_groups, cols, dev)
    rb, cb = _up(rows, BLOCK) // BLOCK, _up(cols, BLOCK) // BLOCK
    lib = _library()

    def launch(handle):
        q = s = qt = st = None
        if outputs != "columns":
            q, s = _codes(rows, cols, dev), _scales(rb if tile else rows, cb, dev)
        if outputs != "rows":
            qt, st = _codes(cols, rows, dev), _scales(cb if tile else cols, rb, dev)
        got = lib.grkan_fp8_quantize(x.data_ptr(), _ptr(A), _ptr(B), _ptr(q), _ptr(s), _ptr(qt), _ptr(st), rows, cols,
                                     ldx, _up(cols, 16), rb if tile else rows, _up(rows, 16), cb if tile else cols,
                                     int(tile), ng, code, io, handle)
        if got != GRKAN_OK:
            raise GRKANError(got, "grkan_fp8_quantize")
        return {"rows": (q, s), "columns": (qt, st), "both": (q, s, qt, st)}[outputs]

    return _on_stream(stream, dev, launch)


def _operand8(t: torch.Tensor, name: str, dev):
    if t.dtype is not F8:
        raise TypeError(f"{name} must be float8_e4m3fn, got {t.dtype}")
    size, stride = t.shape, t.stride()
    if len(size) != 2:
        raise ValueError(f"{name} must be [rows, k]")
    rows, k = size
    if rows <= 1 or (stride[1] != 1 and k > 1) or stride[0] < k or t.device != dev:
        _matrix(t, name, dev)  # (raises unless there is but one row)
    ld = _up(k, 16) if rows <= 1 else stride[0]  # (the stride of a single row is not used)
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"the rows of {name} must start at multiples of 16 bytes, as grkan_fp8_quantize's do")
    return rows, k, ld


def _scale8(t: torch.Tensor, name: str, rows, k: int, dev):
    """(row stride, block stride) of the scales of an operand with `rows` rows (or, one of two, row blocks)."""
    size, blocks = t.shape, _up(k, BLOCK) // BLOCK
    if t.dtype is not torch.float32 or len(size) != 2 or size[1] != blocks or size[0] not in rows or t.device != dev:
        raise ValueError(f"{name} must be a float32 tensor [{' or '.join(map(str, rows))}, "
                         f"{blocks}] on {dev}")
    return t.stride()


_SUMS = {"fp32": 0, "fast": GRKAN_FP8_SUMS_CUT}


def grkan_fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, bias=None,
                     residual=None, dtype=torch.bfloat16, out=None, workspace=None, stream=None, sums: str = "fp32"):
    """a b^T + bias + residual [m, n] in ``dtype`` (bfloat16 or float32) for e4m3 a [m, k], b [n, k]
    (``grkan_fp8_matmul``).

    ``a_scale`` is float32 [m, k / 128] (rounded up), ``b_scale`` [n, k / 128], or [n / 128, k / 128] for 128 x
    128 tiles (if n / 128 rounded up is n itself, n = 1, the two are the same); any strides, expanded ones
    too.  The codes' rows start at multiples of 16 bytes, as the quantiser's do.  float32 ``bias`` [n];
    ``residual`` [m, n] in ``dtype``; ``out`` may be the residual itself.  ``sums``: how the products of a block
    are summed, "fp32", or for a bfloat16 result "fast": twice the rate, products cut off at 2^-13 of the largest of
    each 8, which values whose large products cancel can show (a float32 result's sums stay fp32's)."""
    if sums not in _SUMS:
        raise ValueError(f"sums must be one of {sorted(_SUMS)}")
    _on_gpu(a)
    dev = a.device
    if dtype not in _IO:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    m, k, lda = _operand8(a, "a", dev)
    n, kb, ldb = _operand8(b, "b", dev)
    if kb != k or k < 1 or n < 1:
        raise ValueError(f"a and b must be [m, k] and [n, k], got {list(a.shape)} and {list(b.shape)}")
    nt = _up(n, BLOCK) // BLOCK
    ar, ab = _scale8(a_scale, "a_scale", (m,), k, dev)
    br, bb = _scale8(b_scale, "b_scale", (n, nt), k, dev)
    tile = b_scale.shape[0] != n
    _channel_vector(bias, "bias", n, dev)
    ldr = 0
    if residual is not None:
        if residual.shape != (m, n) or residual.dtype != dtype:
            raise ValueError(f"residual must be [{m}, {n}] in {dtype}")
        ldr = _matrix(residual, "residual", dev)[2]
    lib = _library()
    need = _need("fp8_matmul", m, n, k)

    def launch(handle):
        c = _given(out, "out", (m, n), dtype, dev)
        ws, wsp, wsn = _space(workspace, need, dev)
        st = lib.grkan_fp8_matmul(a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), _ptr(bias),
                                  _ptr(residual), c.data_ptr(), m, n, k, lda, ar, ab, ldb, br, bb,
                                  int(tile) | _SUMS[sums], ldr, _IO[dtype], wsp, wsn, handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_fp8_matmul")
        _written(out)
        return c

    return _on_stream(stream, dev, launch)


class GRKANFp8Linear(torch.autograd.Function):
    """Autograd wrapper: y = F(x) W^T + bias with 8-bit operands, ``apply(x, W, bias, act, A, B, n_groups, sums)``,
    act "none" (F the identity) or "rational"; ``sums`` of all three products as ``grkan_fp8_matmul``'s.

    bf16 x [..., d_in] and W [d_out, d_in], float32 bias.  F(x) and the incoming gradient are quantised in blocks
    of 128 along the axis that each product sums over, W in tiles of 128 x 128 (one set of values for both of its
    products).  x is kept for the backward, which quantises F(x) along the rows: W's gradient sums over at most
    2^22 of them."""

    @classmethod
    def apply(cls, x, W, *args):
        # (inside forward the grad mode is off and needs_input_grad does not know of it)
        if torch.is_grad_enabled() and W.requires_grad and x.shape[:-1].numel() > 1 << 22:
            raise ValueError(f"W's gradient sums over at most {1 << 22} rows, got {x.shape[:-1].numel()}")
        return super().apply(x, W, *args)

    @staticmethod
    def forward(ctx, x, W, bias=None, act="none", A=None, B=None, n_groups=8, sums="fp32"):
        if W.dim() != 2 or W.shape[1] != x.shape[-1]:
            raise ValueError(f"W must be [d_out, {x.shape[-1]}], got {list(W.shape)}")
        if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
            raise TypeError(f"x and W must be bfloat16, got {x.dtype} and {W.dtype}")
        q, s = grkan_fp8_quantize(x, act=act, A=A, B=B, n_groups=n_groups)
        needs = (*ctx.needs_input_grad, False, False, False, False)
        if needs[0] or needs[4] or needs[5]:
            wq, ws, wt, wts = grkan_fp8_quantize(W, "both", tile=True)
        else:
            (wq, ws), wt, wts = grkan_fp8_quantize(W, "rows", tile=True), None, None
        y = grkan_fp8_matmul(q, s, wq, ws, bias=bias, sums=sums)
        ctx.save_for_backward(x, W, bias, A, B, wt, wts)
        ctx.args = act, n_groups, sums
        return y.view(*x.shape[:-1], W.shape[0])

    @staticmethod
    @once_differentiable  # the kernels' results carry no graph: a second derivative would silently lack them
    def backward(ctx, dy):
        x, W, bias, A, B, wt, wts = ctx.saved_tensors
        act, n_groups, sums = ctx.args
        needs = (*ctx.needs_input_grad, False, False, False, False)  # as many as apply was given, three at least
        rows, cols = needs[0] or needs[4] or needs[5], needs[1]
        dy = dy.contiguous().view(-1, W.shape[0])
        dx = dW = db = dA = dB = None
        if cols and not dy.shape[0]:
            cols, dW = False, torch.zeros(W.shape, dtype=W.dtype, device=W.device)
        if rows or cols:
            got = grkan_fp8_quantize(dy, "both" if rows and cols else ("rows" if rows else "columns"))
        if rows:
            dx = grkan_fp8_matmul(got[0], got[1], wt, wts, sums=sums).view(x.shape)
            if act == "rational":
                dx, dA, dB = binding.grkan_backward(x.contiguous(), dx, A, B, n_groups)
        if cols:
            xt, xts = grkan_fp8_quantize(x, "columns", act=act, A=A, B=B, n_groups=n_groups)
            dW = grkan_fp8_matmul(got[-2], got[-1], xt, xts, sums=sums)
        if bias is not None and needs[2]:
            db = grkan_linear_act_backward(x, W.contiguous(), dy.view(*x.shape[:-1], W.shape[0]), skip=("dx", "dW"))[2]
        return (dx, dW, _like(db, bias), None, _like(dA, A), _like(dB, B), None, None)[:len(ctx.needs_input_grad)]


# ---------------------------------------------------------------- residual path

def _gate(gate, lead, rows: int, channels: int, io_dtype, dev):
    """(gate rows, gate channels, dtype code) of a gate that spans x's leading dimensions `lead`."""
    if gate is None:
        return 0, 1, GRKAN_F32
    if gate.dtype not in (torch.float32, io_dtype) or gate.device != dev or not gate.is_contiguous():
        raise ValueError(f"gate must be a contiguous float32 or {io_dtype} tensor on {dev}")
    shape = tuple(gate.shape)
    if len(shape) != len(lead) + 1 or shape[-1] not in (1, channels):
        raise ValueError(f"gate must be [{', '.join(map(str, lead))}, 1 or {channels}] or 1 in its place from some "
                         "dimension on")
    gates, ended = 1, False
    for have, want in zip(shape, lead):
        if have == want and not (ended and have > 1):
            gates *= have
        elif have == 1:
            ended = True
        else:
            raise ValueError(f"gate {list(shape)} does not repeat over whole runs of rows of {[*lead, channels]}")
    return gates, shape[-1], _IO[gate.dtype]


def grkan_residual_norm_forward(x: torch.Tensor, f: torch.Tensor, norm: str = "layer", weight=None, bias=None,
                                scale=None, gate=None, post: str = "none", post_weight=None, post_bias=None,
                                eps: float = 1e-5, out=None, normed=None, stats=None, stream=None):
    """(h, z, stats): h = x + scale gate post(f), z = norm(h) (``grkan_residual_norm_forward``).

    ``x`` and ``f`` are [..., channels] in float32 or bfloat16 with equally spaced rows.  ``norm`` is "layer" or
    "rms", ``post`` those or "none".  ``weight``, ``bias``, ``scale``, ``post_weight`` and ``post_bias`` are float32
    [channels] or None.  ``gate`` (float32 or x's dtype) has x's dimensions, with 1 for the channels and for any
    trailing run of the leading dimensions: [samples, 1, 1] is one value for a sample.  stats is float32 [2,
    rows], [4, rows] with a post norm, for the backward.  ``out`` (for h) may be x itself."""
    if norm not in _NORMS or post not in _POSTS:
        raise ValueError('norm must be "layer" or "rms", post those or "none"')
    io = _io(x)
    _on_gpu(x)
    dev = x.device
    if f.shape != x.shape or f.dtype != x.dtype or f.device != dev:
        raise ValueError("f must match x")
    rows, c, ldx = _matrix(x, "x")
    ldf = _matrix(f, "f")[2]
    if c < 1:
        raise ValueError("x must have a channel")
    for t, name in ((weight, "weight"), (bias, "bias"), (scale, "scale"), (post_weight, "post_weight"),
                    (post_bias, "post_bias")):
        if t is not None:
            _channel_vector(t, name, c, dev)
    if post == "none" and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias need a post norm")
    gates, gc, gio = _gate(gate, x.shape[:-1], rows, c, x.dtype, dev)
    for t, name in ((out, "out"), (normed, "normed")):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name} must match x")
    lib, dense = _library(), x.is_contiguous()

    def launch(handle):
        h = _given(out, "out", x.shape, x.dtype, dev) if out is not None or not dense else torch.empty_like(x)
        z = _given(normed, "normed", x.shape, x.dtype, dev) if normed is not None or not dense else torch.empty_like(x)
        st = _given(stats, "stats", (2 if post == "none" else 4, rows), torch.float32, dev)
        got = lib.grkan_residual_norm_forward(x.data_ptr(), f.data_ptr(), _ptr(weight), _ptr(bias), _ptr(scale),
                                              _ptr(gate), _ptr(post_weight), _ptr(post_bias), h.data_ptr(),
                                              z.data_ptr(), st.data_ptr(), rows, c, ldx, ldf, gates, gc, eps,
                                              _NORMS[norm], _POSTS[post], io, gio, handle)
        if got != GRKAN_OK:
            raise GRKANError(got, "grkan_residual_norm_forward")
        _written(out, normed, stats)
        return h, z, st

    return _on_stream(stream, dev, launch)


_RESIDUAL_GRADS = ("dx", "df", "dscale", "dgate", "dweight", "dbias", "dpost_weight", "dpost_bias")


def grkan_residual_norm_backward(f: torch.Tensor, h: torch.Tensor, dh, dz, stats: torch.Tensor, norm: str = "layer",
                                 weight=None, bias=None, scale=None, gate=None, post: str = "none", post_weight=None,
                                 post_bias=None, dx=None, df=None, workspace=None, stream=None, skip=()):
    """(dx, df, dscale, dgate, dweight, dbias, dpost_weight, dpost_bias) of ``grkan_residual_norm_forward`` from its
    f, h and stats (``grkan_residual_norm_backward``).

    ``dh`` is the gradient that reaches h besides through z, ``dz`` that of z; one of them may be None.  dbias is
    None without bias, dgate without gate, dpost_weight and dpost_bias without theirs; dscale and dweight are
    given also without scale and weight (of ones).  ``skip``: names among the results that are not computed (None
    in their place).  ``dx`` (a tensor for it) may be dh itself, ``df`` dz itself."""
    if norm not in _NORMS or post not in _POSTS:
        raise ValueError('norm must be "layer" or "rms", post those or "none"')
    _skipped(skip, _RESIDUAL_GRADS)
    io = _io(h)
    _on_gpu(h)
    dev = h.device
    rows, c, _ = _matrix(h, "h")
    if not h.is_contiguous():
        raise ValueError("h must be contiguous")
    if dh is None and dz is None:
        raise ValueError("dh or dz must be given")
    lds = []
    for t, name in ((f, "f"), (dh, "dh"), (dz, "dz")):
        if t is not None and (t.shape != h.shape or t.dtype != h.dtype or t.device != dev):
            raise ValueError(f"{name} must match h")
        lds.append(0 if t is None else _matrix(t, name)[2])
    for t, name in ((weight, "weight"), (bias, "bias"), (scale, "scale"), (post_weight, "post_weight"),
                    (post_bias, "post_bias")):
        if t is not None:
            _channel_vector(t, name, c, dev)
    if post == "none" and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias need a post norm")
    _check_out(stats, "stats", torch.float32, rows * (2 if post == "none" else 4), dev)
    gates, gc, gio = _gate(gate, h.shape[:-1], rows, c, h.dtype, dev)
    for t, name in ((dx, "dx"), (df, "df")):
        if t is not None and t.shape != h.shape:
            raise ValueError(f"{name} must match h")
    lib = _library()
    need = _need("residual_norm_backward", rows, c, gates, gc, _POSTS[post], io)
    absent = set(skip)
    for name, t in (("dgate", gate), ("dbias", bias), ("dpost_weight", post_weight), ("dpost_bias", post_bias)):
        if t is None:
            absent.add(name)

    def launch(handle):
        gx = _wanted(absent, "dx", dx, h.shape, h.dtype, dev)
        gf = _wanted(absent, "df", df, h.shape, h.dtype, dev)
        gg = None if "dgate" in absent else torch.empty_like(gate)
        gs, gw, gb, gpw, gpb = (_wanted(absent, name, None, (c,), torch.float32, dev)
                                for name in ("dscale", "dweight", "dbias", "dpost_weight", "dpost_bias"))
        ws, wsp, wsn = _space(workspace, need, dev)
        st = lib.grkan_residual_norm_backward(f.data_ptr(), h.data_ptr(), _ptr(dh), _ptr(dz), stats.data_ptr(),
                                              _ptr(weight), _ptr(scale), _ptr(gate), _ptr(post_weight),
                                              _ptr(post_bias), _ptr(gx), _ptr(gf), _ptr(gs), _ptr(gg), _ptr(gw),
                                              _ptr(gb), _ptr(gpw), _ptr(gpb), rows, c, *lds, gates, gc, _NORMS[norm],
                                              _POSTS[post], io, gio, wsp, wsn, handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_residual_norm_backward")
        _written(dx, df)
        return gx, gf, gs, gg, gw, gb, gpw, gpb

    return _on_stream(stream, dev, launch)


class GRKANResidualNorm(torch.autograd.Function):
    """Autograd wrapper: (h, z) of ``grkan_residual_norm_forward``, ``apply(x, f, norm, weight, bias, scale, gate,
    post, post_weight, post_bias, eps)``."""

    @staticmethod
    def forward(ctx, x, f, norm="layer", weight=None, bias=None, scale=None, gate=None, post="none", post_weight=None,
                post_bias=None, eps=1e-5):
        h, z, stats = grkan_residual_norm_forward(x, f, norm, weight, bias, scale, gate, post, post_weight, post_bias,
                                                  eps)
        ctx.save_for_backward(f, h, stats, weight, bias, scale, gate, post_weight, post_bias)
        ctx.args = norm, post
        ctx.set_materialize_grads(False)
        return h, z

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dz):
        f, h, stats, weight, bias, scale, gate, post_weight, post_bias = ctx.saved_tensors
        norm, post = ctx.args
        needs = (*ctx.needs_input_grad, *(False,) * 9)
        if dh is None and dz is None:
            return (None,) * len(ctx.needs_input_grad)
        place = {"dx": 0, "df": 1, "dweight": 3, "dbias": 4, "dscale": 5, "dgate": 6, "dpost_weight": 8, "dpost_bias": 9}
        skip = [name for name, i in place.items() if not needs[i]]
        got = grkan_residual_norm_backward(f, h, None if dh is None else dh.contiguous(),
                                           None if dz is None else dz.contiguous(), stats, norm, weight, bias, scale,
                                           gate, post, post_weight, post_bias, skip=skip)
        got = dict(zip(_RESIDUAL_GRADS, got))
        out = [None] * 11
        for name, i in place.items():
            out[i] = got[name]
        for i, t in ((3, weight), (4, bias), (5, scale), (8, post_weight), (9, post_bias)):
            out[i] = _like(out[i], t) if t is not None else None
        return tuple(out[:len(ctx.needs_input_grad)])


# ---------------------------------------------------------------- AdamW

def _scalar(t, name: str, dtype, dev):
    if t.dtype != dtype or t.device != dev or t.numel() != 1:
        raise ValueError(f"{name} must be one {dtype} value on {dev}")
    return t.data_ptr()


_dtype, _size, _whole, _place, _at = (operator.attrgetter("dtype"), torch.Tensor.numel, torch.Tensor.is_contiguous,
                                      torch.Tensor.get_device, torch.Tensor.data_ptr)


def _all(want, of, tensors) -> bool:
    """Whether of(t) is `want` for all."""
    return all(got == want for got in map(of, tensors))


def _adamw_table(params, grads, masters, avgs, sqs, avg_scales, sq_scales, eight: bool, dev) -> array.array:
    """The tensors as an array of grkan_adamw_tensor_t, checked list by list (hundreds of tensors a step: a
    check costs as much as a small launch if it is made one tensor at a time)."""
    n, f32 = len(params), torch.float32
    state = F8 if eight else f32
    dtypes, counts = list(map(_dtype, params)), list(map(_size, params))
    held = [-(-k // BLOCK) * BLOCK for k in counts] if eight else counts
    scales = [k // BLOCK for k in held]
    for d in set(dtypes):
        if d not in _IO:
            raise TypeError(f"parameters must be float32 or bfloat16, got {d}")
    if list(map(_dtype, grads)) != dtypes or list(map(_size, grads)) != counts:
        raise ValueError("each gradient must have its parameter's size and dtype")
    if not (_all(state, _dtype, avgs) and _all(state, _dtype, sqs) and list(map(_size, avgs)) == held
            and list(map(_size, sqs)) == held):
        raise ValueError(f"avgs and sqs must be {state} of the parameters' sizes" + (", whole blocks of 128" if eight else ""))
    others = [params, grads, avgs, sqs]
    if eight:
        for t, name in ((avg_scales, "avg_scales"), (sq_scales, "sq_scales")):
            if not _all(f32, _dtype, t) or list(map(_size, t)) != scales:
                raise ValueError(f"{name} must be float32, one for each block of 128")
        others += [avg_scales, sq_scales]
    main = [0] * n
    if masters is not None:
        kept = [w for w in masters if w is not None]
        if not _all(f32, _dtype, kept) or any(w is not None and w.numel() != k for w, k in zip(masters, counts)):
            raise ValueError("masters must be float32 of their parameters' sizes")
        others.append(kept)
        main = [0 if w is None else w.data_ptr() for w in masters]
    if not _all(dev.index, _place, chain(*others)) or not all(map(_whole, chain(*others))):
        raise ValueError(f"all tensors must be contiguous and on {dev}")
    none = [0] * n
    rows = zip(map(_at, params), map(_at, grads), main, map(_at, avgs), map(_at, sqs),
               map(_at, avg_scales) if eight else none, map(_at, sq_scales) if eight else none, counts,
               map(_IO.__getitem__, dtypes))
    return array.array("q", chain.from_iterable(rows))


def grkan_adamw_step(params, grads, avgs, sqs, *, step, lr, beta1: float = 0.9, beta2: float = 0.999,
                     eps: float = 1e-8, weight_decay: float = 1e-2, masters=None, avg_scales=None, sq_scales=None,
                     grad_scale=None, seed: int = 0, stream=None) -> None:
    """One AdamW step over lists of tensors, in place (``grkan_adamw_step``).

    ``params`` and ``grads`` are contiguous float32 or bfloat16 tensors (a gradient in its parameter's dtype);
    ``masters``: the weights in float32 for some (None for the others), their parameter then being the rounded
    copy; where it is not, a program has written it since, and the parameter's value is stepped.  ``avgs`` and
    ``sqs`` are float32 tensors of the parameters' sizes, or, with ``avg_scales`` and ``sq_scales`` (float32, one
    for each 128 values), float8_e4m3fn codes of the first moment and of the second moment's root, whole blocks of
    128 (``grkan_adamw_state`` makes them).  ``step`` (from 1) and ``lr`` are numbers, or one int64 and one float32
    value on the device, which the kernel reads (and a captured graph reads again at each replay).  ``grad_scale``:
    one float32 value on the device that every gradient is multiplied with.  ``seed``: of the 8-bit states' rounding.

    What is written counts as modified in place: a backward that still needs it raises (a graph's replays
    write without being noticed)."""
    n = len(params)
    eight = avg_scales is not None or sq_scales is not None
    if eight and (avg_scales is None or sq_scales is None):
        raise ValueError("avg_scales and sq_scales come together")
    for name, got in (("grads", grads), ("avgs", avgs), ("sqs", sqs), ("masters", masters), ("avg_scales", avg_scales),
                      ("sq_scales", sq_scales)):
        if got is not None and len(got) != n:
            raise ValueError(f"{name} must be a list of {n}")
    if n == 0:
        return
    _on_gpu(params[0])
    dev = params[0].device
    table = _adamw_table(params, grads, masters, avgs, sqs, avg_scales, sq_scales, eight, dev)
    hyper = grkan_adamw_t(beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay, seed=seed & 0xFFFFFFFF)
    if isinstance(lr, torch.Tensor):
        hyper.lr_ptr = _scalar(lr, "lr", torch.float32, dev)
    else:
        hyper.lr = lr
    if isinstance(step, torch.Tensor):
        hyper.step_ptr = _scalar(step, "step", torch.int64, dev)
    else:
        hyper.step = step
    if grad_scale is not None:
        hyper.grad_scale = _scalar(grad_scale, "grad_scale", torch.float32, dev)
    lib = _library()

    def launch(handle):
        st = lib.grkan_adamw_step(table.buffer_info()[0], n, ctypes.byref(hyper), 8 if eight else 32, handle)
        if st != GRKAN_OK:
            raise GRKANError(st, "grkan_adamw_step")

    _on_stream(stream, dev, launch)
    kept = () if masters is None else (w for w in masters if w is not None)
    increment_version(chain(params, kept, avgs, sqs, avg_scales or (), sq_scales or ()))


def grkan_adamw_state(param: torch.Tensor, bits: int = 32):
    """(avg, sq, avg_scale, sq_scale) of a parameter before its first step; the scales None for 32 bits."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    if bits == 32:
        return (*(torch.zeros(param.numel(), dtype=torch.float32, device=param.device) for _ in range(2)), None, None)
    held = _up(param.numel(), BLOCK)
    # (a float8 zero is a byte of zeros)
    codes = (torch.zeros(held, dtype=torch.uint8, device=param.device).view(F8) for _ in range(2))
    return (*codes, *(torch.ones(held // BLOCK, dtype=torch.float32, device=param.device) for _ in range(2)))


class GRKANAdamW(torch.optim.Optimizer):
    """AdamW with one launch for up to 48 tensors, states in 32 bits or 8, and float32 masters of bfloat16
    parameters.

    Per parameter group: ``lr`` (a number, or one float32 value on the device), ``betas``, ``eps``,
    ``weight_decay``, ``bits`` (32 or 8), ``masters`` (keep bfloat16 parameters in float32 besides; what a program
    writes into a parameter between steps goes into its master with the next; without, parameters are stepped and
    rounded to nearest), ``seed`` (of the 8-bit states' rounding; each group adds its number).
    ``step(grad_scale=...)`` takes one float32 value on the device that every gradient is multiplied with.
    Parameters without a gradient are left as they are, and count no step.

    Steps are counted on the host, so a step is not captured into a graph (it would repeat its number):
    ``grkan_adamw_step`` with a step on the device is."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, bits=32, masters=True, seed=0):
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        if not isinstance(lr, torch.Tensor) and not lr >= 0.0:
            raise ValueError(f"lr must be at least 0, got {lr}")
        if len(betas) != 2 or not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError(f"betas must be two numbers in [0, 1), got {betas}")
        if not eps >= 0.0 or not weight_decay >= 0.0:
            raise ValueError(f"eps and weight_decay must be at least 0, got {eps} and {weight_decay}")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, bits=bits, masters=masters,
                                      seed=seed))

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        # (which casts states to their parameter's dtype: these have their own)
        saved = [i for g in state_dict["param_groups"] for i in g["params"]]
        held = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(saved, held):
            if i in state_dict["state"]:
                self.state[p] = {k: v.detach().clone().to(p.device) if isinstance(v, torch.Tensor) else v
                                 for k, v in state_dict["state"][i].items()}

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a captured step would repeat its number: capture grkan_adamw_step with step on the device")
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for at, group in enumerate(self.param_groups):
            runs = {}  # the tensors that are at the same step
            for index, p in enumerate(group["params"]):
                if p.grad is None:
                    continue
                state = self.state[p]
                if not state:
                    state["step"] = 0
                    state["avg"], state["sq"], state["avg_scale"], state["sq_scale"] = \
                        grkan_adamw_state(p, group["bits"])
                    state["master"] = p.detach().float().contiguous() \
                        if group["masters"] and p.dtype == torch.bfloat16 else None
                runs.setdefault((state["step"] + 1, p.device), []).append((p, state))
            for (step, _), run in runs.items():
                eight = run[0][1]["avg_scale"] is not None
                grkan_adamw_step(
                    [p.detach() for p, _ in run], [p.grad.detach().contiguous() for p, _ in run],
                    [s["avg"] for _, s in run], [s["sq"] for _, s in run], step=step, lr=group["lr"],
                    beta1=group["betas"][0], beta2=group["betas"][1], eps=group["eps"],
                    weight_decay=group["weight_decay"], masters=[s["master"] for _, s in run],
                    avg_scales=[s["avg_scale"] for _, s in run] if eight else None,
                    sq_scales=[s["sq_scale"] for _, s in run] if eight else None, grad_scale=grad_scale,
                    seed=group["seed"] + at)
                for _, state in run:  # (counted once it has run: a refused step may be tried again)
                    state["step"] = step
        return loss

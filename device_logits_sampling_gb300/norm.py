"""The join around a block (include/serve/arc_norm.h): the norm after it, its gate, the
scaled residual sum and the norm before the next one, in one pass."""
from __future__ import annotations

import struct

import torch

from . import serve
from .serve import want
from .workloads import DTYPE_F32

MAX_DIM = 32768
ACTIVATIONS = {None: 0, "sigmoid": 1}

_ROWS = struct.Struct("@PPPPPPPqqqqqqiiiiifff")  # arc_norm_rows


def _rows(x, shape, dev, name):
    """Row stride of a checked [rows, dim] tensor."""
    a, b = x.stride() if x.shape == shape else (0, 0)
    want(b == 1 or (a and shape[1] == 1), f"{name} must be [rows, dim], rows contiguous")
    want(x.get_device() == dev, "every tensor must be on x's device")
    return a if shape[0] > 1 else shape[1]


def _vector(x, dim, dev, name):
    want(x.shape == (dim,) and (x.stride(0) == 1 or dim == 1), f"{name} must be contiguous [dim]")
    want(x.get_device() == dev, "every tensor must be on x's device")


def join(x, y=None, weight=None, post_weight=None, gate=None, activation: str | None = None, alpha: float = 1.0,
         offset: float = 0.0, eps: float = 1e-6, h=None, n=None, dtype=None, next_norm: bool = True, stream=None,
         check: bool = True):
    """arc_norm_join: the residual stream x [rows, dim] (bfloat16, float16 or float32) after the block's output y
    [rows, dim] (bfloat16 or float16), and its norm.  Returns (h, n):

        u = y, normed with post_weight [dim] where given, times gate (or its sigmoid) where given
        h = x + alpha * u          of x's type
        n = rms_norm(h) * (offset + weight), before h is rounded, of y's type

    gate: [rows, dim] or [dim], of y's type.  weight, post_weight: of y's type or float32; weight None: the norm
    alone.  Without y only n is computed and h is x.  next_norm False: only h, and n is None.  h and n: outputs, new
    ones where None; h may be x, n may be y.  dtype: n's type where y is None and x is float32.  stream: where the
    call runs, the current stream where None; what the call makes for itself is made there."""
    shape, dev, xt = x.shape, x.get_device(), x.dtype
    want(len(shape) == 2, "x must be [rows, dim]")
    rows, dim = shape
    wide = xt == torch.float32
    if y is None:
        want(gate is None and post_weight is None and h is None, "gate, post_weight and h need y")
        want(next_norm, "without y there is the norm alone")
        kind = dtype or (xt if not wide else n.dtype if n is not None else torch.bfloat16)
    else:
        kind = y.dtype
        want(dtype is None or dtype == kind, "n has y's type")
    code = serve._CODES.get(kind)
    if code is None:
        raise TypeError(f"y and n must be bfloat16 or float16, not {kind}")
    if not wide and xt != kind:
        raise TypeError(f"x must be {kind} or float32, not {xt}")
    want(activation in ACTIVATIONS, f"activation must be one of {list(ACTIVATIONS)}")
    xs = _rows(x, shape, dev, "x")
    ys = gs = hs = ns = yp = gp = hp = np_ = wp = pp = 0
    if y is not None:
        ys, yp = _rows(y, shape, dev, "y"), y.data_ptr()
    if gate is not None:
        if gate.dtype != kind:
            raise TypeError(f"gate must be {kind}, not {gate.dtype}")
        if gate.dim() == 1:
            _vector(gate, dim, dev, "gate")
        else:
            gs = _rows(gate, shape, dev, "gate")
        gp = gate.data_ptr()
    wtype = None
    if weight is not None:
        _vector(weight, dim, dev, "weight")
        wtype, wp = weight.dtype, weight.data_ptr()
    if post_weight is not None:
        _vector(post_weight, dim, dev, "post_weight")
        if wtype is not None and post_weight.dtype != wtype:
            raise TypeError("weight and post_weight must have one type")
        wtype, pp = post_weight.dtype, post_weight.data_ptr()
    if wtype is not None and wtype != kind and wtype != torch.float32:
        raise TypeError(f"weights must be {kind} or float32, not {wtype}")
    serve.on_current_gpu(dev)
    if y is not None:
        if h is None:
            h = serve.new_output(x, (rows, dim), (dim, 1), xt, stream)
            hs = dim
        else:
            want(h.dtype == xt, "h must have x's type")
            hs = _rows(h, shape, dev, "h")
        hp = h.data_ptr()
    if next_norm:
        if n is None:
            n = serve.new_output(x, (rows, dim), (dim, 1), kind, stream)
            ns = dim
        else:
            want(n.dtype == kind, "n must have y's type")
            ns = _rows(n, shape, dev, "n")
        np_ = n.data_ptr()
    else:
        want(n is None, "n without next_norm")
    args = _ROWS.pack(x.data_ptr(), yp, gp, pp, wp, hp, np_, xs, ys, gs, hs, ns, rows, dim, DTYPE_F32 if wide else code, code,
                      DTYPE_F32 if wtype == torch.float32 else code, ACTIVATIONS[activation], alpha, offset, eps)
    rc = serve.load().arc_norm_join(args, serve.stream_of(stream, dev))
    if rc:
        serve.finish(rc, check)
    return (x if y is None else h), n

"""Products of a few rows with 4-bit weights and group scales (include/serve/arc_w4.h)."""
from __future__ import annotations

import struct

import torch

from . import serve
from .serve import want

MAX_ROWS = 256
FEW_ROWS = 8  # more rows need a workspace

_WEIGHT = struct.Struct("@PPPqqii")  # arc_w4_weight


def pack(q):
    """uint8 [outs, ins] of 0 .. 15 as uint8 [outs, ins / 2], two to a byte, the even one low."""
    return q[:, 0::2] | (q[:, 1::2] << 4)


def matvec(x, weight, scales, zeros=None, out=None, out_dtype=None, workspace=None, stream=None, check: bool = True):
    """arc_w4_matvec: x [rows, ins] (bfloat16 or float16, 1 .. 256 rows) times the transpose of
    (q - zero) * scale, weight uint8 [outs, ins / 2] (see pack), scales [outs, ins / group] of
    x's type with group 32, 64 or 128, zeros uint8 [outs, ins / group] or None for 8.  Returns
    out [rows, outs] of x's type, or float32 with out_dtype.  stream: where the call runs, the
    current stream where None; what the call makes for itself is made there."""
    want(x.dim() == 2 and weight.dim() == 2 and scales.dim() == 2, "x, weight and scales must be matrices")
    rows, ins = x.shape
    outs, groups = scales.shape
    xs, one = x.stride()
    want(one == 1, "rows of x must be contiguous")
    if weight.dtype != torch.uint8:
        raise TypeError(f"weight must be uint8, not {weight.dtype}")
    ws, one = weight.stride()
    want(weight.shape == (outs, ins // 2) and one == 1 and ins % 2 == 0, "weight must be [outs, ins / 2], rows contiguous")
    want(groups > 0 and ins % groups == 0 and scales.is_contiguous(), "scales must be contiguous [outs, ins / group]")
    if scales.dtype != x.dtype:
        raise TypeError("scales must have x's type")
    dev, zp = x.get_device(), 0
    if zeros is not None:
        want(zeros.shape == scales.shape and zeros.is_contiguous(), "zeros must be contiguous [outs, ins / group]")
        if zeros.dtype != torch.uint8:
            raise TypeError(f"zeros must be uint8, not {zeros.dtype}")
        want(zeros.get_device() == dev, "every tensor must be on x's device")
        zp = zeros.data_ptr()
    code = serve.dtype_code(x)
    want(weight.get_device() == dev and scales.get_device() == dev, "every tensor must be on x's device")
    serve.on_current_gpu(dev)
    if out is None:
        out = serve.new_output(x, (rows, outs), (outs, 1), out_dtype or x.dtype, stream)
        os = outs
    else:
        want(out.shape == (rows, outs) and out.stride(1) == 1, "out must be [rows, outs], rows contiguous")
        want(out_dtype is None or out.dtype == out_dtype, "out has another type than out_dtype")
        want(out.get_device() == dev, "every tensor must be on x's device")
        os = out.stride(0) if rows > 1 else outs
    w = _WEIGHT.pack(weight.data_ptr(), scales.data_ptr(), zp, ws if outs > 1 else ins // 2, outs, ins, ins // groups)
    lib = serve.load()
    wp, wn = 0, 0
    if rows > FEW_ROWS:
        if workspace is None:
            need = lib.arc_w4_workspace_bytes(w, rows)
            workspace = serve.new_workspace(x, need, False, stream)
        wp, wn = serve.workspace_of(workspace, dev)
    rc = lib.arc_w4_matvec(w, x.data_ptr(), rows, xs if rows > 1 else ins, code, out.data_ptr(), os,
                           serve.dtype_code(out, True), wp, wn, serve.stream_of(stream, dev))
    serve.finish(rc, check)
    return out

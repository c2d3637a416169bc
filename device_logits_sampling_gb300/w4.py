"""Products of a few rows with 4-bit weights and group scales (include/serve/arc_w4.h)."""
from __future__ import annotations

import ctypes

from . import sampler, serve
from .serve import want

MAX_ROWS = 256


def pack(q):
    """uint8 [outs, ins] of 0 .. 15 as uint8 [outs, ins / 2], two to a byte, the even one low."""
    return q[:, 0::2] | (q[:, 1::2] << 4)


def matvec(x, weight, scales, zeros=None, out=None, out_dtype=None, workspace=None, stream=None, check: bool = True):
    """arc_w4_matvec: x [rows, ins] (bfloat16 or float16, 1 .. 256 rows) times the transpose of
    (q - zero) * scale, weight uint8 [outs, ins / 2] (see pack), scales [outs, ins / group] of
    x's type with group 32, 64 or 128, zeros uint8 [outs, ins / group] or None for 8.  Returns
    out [rows, outs] of x's type, or float32 with out_dtype."""
    import torch

    want(x.dim() == 2 and weight.dim() == 2 and scales.dim() == 2, "x, weight and scales must be matrices")
    rows, ins = x.shape
    outs, groups = scales.shape
    want(x.stride(1) == 1, "rows of x must be contiguous")
    if weight.dtype != torch.uint8:
        raise TypeError(f"weight must be uint8, not {weight.dtype}")
    want(weight.shape == (outs, ins // 2) and weight.stride(1) == 1 and ins % 2 == 0,
         "weight must be [outs, ins / 2], rows contiguous")
    want(groups > 0 and ins % groups == 0 and scales.is_contiguous(), "scales must be contiguous [outs, ins / group]")
    if scales.dtype != x.dtype:
        raise TypeError("scales must have x's type")
    if zeros is not None:
        want(zeros.shape == scales.shape and zeros.is_contiguous(), "zeros must be contiguous [outs, ins / group]")
        if zeros.dtype != torch.uint8:
            raise TypeError(f"zeros must be uint8, not {zeros.dtype}")
    if out is None:
        out = torch.empty((rows, outs), dtype=out_dtype or x.dtype, device=x.device)
    else:
        want(out.shape == (rows, outs) and out.stride(1) == 1, "out must be [rows, outs], rows contiguous")
        want(out_dtype is None or out.dtype == out_dtype, "out has another type than out_dtype")
    for t in (weight, scales, zeros, out):
        want(t is None or t.device == x.device, "every tensor must be on x's device")
    w = serve.W4Weight(weight.data_ptr(), scales.data_ptr(), sampler._ptr(zeros),
                       weight.stride(0) if outs > 1 else weight.shape[1], outs, ins, ins // groups)
    lib = serve.load()
    ref = ctypes.addressof(w)
    need = lib.arc_w4_workspace_bytes(ref, rows)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    rc = lib.arc_w4_matvec(ref, x.data_ptr(), rows, x.stride(0) if rows > 1 else ins, serve.dtype_code(x), out.data_ptr(),
                           out.stride(0) if rows > 1 else outs, serve.dtype_code(out, f32=True),
                           sampler._ptr(workspace), 0 if workspace is None else workspace.numel(), serve.stream_of(stream, x.device))
    serve.finish(rc, check)
    return out

"""Edits of a step's logits before they are sampled (include/serve/arc_edit.h): penalties
for repeated ids, biases, and the bit mask of a grammar."""
from __future__ import annotations

import struct

import numpy as np
import torch

from . import serve
from .serve import want
from .workloads import DTYPE_BF16, DTYPE_F16, DTYPE_F32, ROW_PARAMS_DTYPE

ARC_EDIT_ERR_PARAM = 0x1
ARC_EDIT_ERR_HIST = 0x2
ARC_EDIT_ERR_BIAS = 0x4
ARC_EDIT_ERR_MASK = 0x8

_EDITS = struct.Struct("@PPPqPPPqPqqP")  # arc_logit_edits
_CODES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
_I32 = torch.int32


def pack_mask(allowed) -> np.ndarray:
    """Truth values [rows, V] as the mask's words, int32 [rows, ceil(V / 32)]: bit i % 32 of word i / 32."""
    a = np.asarray(allowed, dtype=bool)
    bits = np.zeros((a.shape[0], -(-a.shape[1] // 32) * 32), dtype=bool)
    bits[:, : a.shape[1]] = a
    return np.packbits(bits, axis=1, bitorder="little").view("<i4")


def _list(offsets, ids, B, dev, name):
    want(offsets.shape == (B + 1,) and offsets.is_contiguous(), f"{name}_offsets must be contiguous [rows + 1]")
    want(ids.dim() == 1 and ids.is_contiguous(), f"{name}_ids must be contiguous")
    if offsets.dtype != _I32 or ids.dtype != _I32:
        raise TypeError(f"{name}_offsets and {name}_ids must be int32")
    want(offsets.get_device() == dev and ids.get_device() == dev, "every tensor must be on the logits' device")


def edit_logits(logits, out=None, out_dtype=None, params=None, hist_offsets=None, hist_ids=None, bias_offsets=None,
                bias_ids=None, bias=None, allowed=None, allowed_rows=None, err_word=None, stream=None,
                check: bool = True):
    """arc_edit_logits: logits [rows, V] (bfloat16, float16 or float32, rows of any stride) with, in this order,

    * the penalties of params (the sampler's records, sampler.params_tensor) for the ids of each row's
      history, hist_ids[hist_offsets[r] : hist_offsets[r + 1]] (int32); a history edited here is not given to
      the sampler again
    * bias [entries] float32 added to the ids bias_ids[bias_offsets[r] : bias_offsets[r + 1]]; where a row
      lists an id more than once its last entry counts
    * -infinity for the ids whose bit in `allowed` int32 [masks, ceil(V / 32)] (see pack_mask) is 0;
      allowed_rows int32 [rows]: each row's mask, or -1 for none; its own where None

    Returns out: of the logits' type or float32 (out_dtype), new where None; out=logits edits in place.
    err_word int32 [1]: ARC_EDIT_ERR_* bits.  stream: where the call runs, the current stream where None."""
    want(logits.dim() == 2, "logits must be [rows, V]")
    B, V = logits.shape
    code = _CODES.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be bfloat16, float16 or float32, not {logits.dtype}")
    ls, one = logits.stride()
    want(one == 1 or V == 1, "rows of logits must be contiguous")
    dev = logits.get_device()
    hp = hi = bp = bi = bv = mp = mr = pp = 0
    hn = bn = ms = mn = 0
    if hist_offsets is not None or hist_ids is not None:
        want(hist_offsets is not None and hist_ids is not None and params is not None,
             "a history is hist_offsets, hist_ids and params")
        _list(hist_offsets, hist_ids, B, dev, "hist")
        want(params.is_contiguous() and params.numel() * params.element_size() >= B * ROW_PARAMS_DTYPE.itemsize,
             "params must hold a record for each row")
        want(params.get_device() == dev, "every tensor must be on the logits' device")
        hp, hn, pp = hist_offsets.data_ptr(), hist_ids.numel(), params.data_ptr()
        hi = hist_ids.data_ptr() if hn else hp  # (a list without an entry has no address, and is not read)
    if bias_offsets is not None or bias_ids is not None or bias is not None:
        want(bias_offsets is not None and bias_ids is not None and bias is not None,
             "biases are bias_offsets, bias_ids and bias")
        _list(bias_offsets, bias_ids, B, dev, "bias")
        want(bias.shape == bias_ids.shape and bias.is_contiguous(), "bias must have an entry for each of bias_ids")
        if bias.dtype != torch.float32:
            raise TypeError(f"bias must be float32, not {bias.dtype}")
        want(bias.get_device() == dev, "every tensor must be on the logits' device")
        bp, bn = bias_offsets.data_ptr(), bias.numel()
        bi, bv = (bias_ids.data_ptr(), bias.data_ptr()) if bn else (bp, bp)
    if allowed is not None:
        want(allowed.dim() == 2 and allowed.shape[1] >= -(-V // 32), "allowed must be [masks, ceil(V / 32)]")
        want(allowed.stride(1) == 1 or allowed.shape[1] == 1, "rows of allowed must be contiguous")
        if allowed.dtype != _I32:
            raise TypeError(f"allowed must be int32, not {allowed.dtype}")
        want(allowed.get_device() == dev, "every tensor must be on the logits' device")
        mp, mn = allowed.data_ptr(), allowed.shape[0]
        ms = allowed.stride(0) if mn > 1 else allowed.shape[1]
        if allowed_rows is not None:
            want(allowed_rows.shape == (B,) and allowed_rows.is_contiguous(), "allowed_rows must be contiguous [rows]")
            if allowed_rows.dtype != _I32:
                raise TypeError(f"allowed_rows must be int32, not {allowed_rows.dtype}")
            want(allowed_rows.get_device() == dev, "every tensor must be on the logits' device")
            mr = allowed_rows.data_ptr()
        else:
            want(mn >= B, "allowed must have a row for each row of logits")
    else:
        want(allowed_rows is None, "allowed_rows without allowed")
    serve.on_current_gpu(dev)
    if out is None:
        out = serve.new_output(logits, (B, V), (V, 1), out_dtype or logits.dtype, stream)
        os = V
    else:
        want(out.shape == (B, V) and (out.stride(1) == 1 or V == 1), "out must be [rows, V], rows contiguous")
        want(out_dtype is None or out.dtype == out_dtype, "out has another type than out_dtype")
        want(out.get_device() == dev, "every tensor must be on the logits' device")
        os = out.stride(0) if B > 1 else V
    if out.dtype != logits.dtype and out.dtype != torch.float32:
        raise TypeError(f"out must be {logits.dtype} or float32, not {out.dtype}")
    edits = _EDITS.pack(pp, hp, hi, hn, bp, bi, bv, bn, mp, ms, mn, mr)
    rc = serve.load().arc_edit_logits(logits.data_ptr(), B, V, ls if B > 1 else V, code, out.data_ptr(), os,
                                      _CODES[out.dtype], edits, serve.err_word_ptr(err_word, dev),
                                      serve.stream_of(stream, dev))
    serve.finish(rc, check)
    return out

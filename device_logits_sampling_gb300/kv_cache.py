"""Paged key/value cache in 8 bits (include/serve/arc_kv.h): appending a step's
tokens with the position rotation on the way, and attention over the cache.

Tensors are CUDA tensors used as device memory.  `positions` is the device
array that the decode-loop commit advances (decode.py), so append, attend, the
last projection (w4.py) and sampler.sample_batch / decode.sample_and_commit
replay as one captured step.
"""
from __future__ import annotations

import ctypes
import math
import struct

import numpy as np
import torch

from . import serve
from .serve import want

ARC_KV_ERR_PAGE = 0x1
ARC_KV_ERR_POSITION = 0x2
ARC_KV_ERR_NAN = 0x4
ARC_KV_ERR_OFFSETS = 0x8
ARC_KV_ERR_SCALE = 0x10
E4M3_MAX = 448.0
SCALE_EXP = 32  # page scales written by append lie in [2^-32, 2^32]
LAYOUTS = {"half": 0, "interleaved": 1}

# arc_kv_step, arc_kv_rows and arc_kv_query, packed for a call (a ctypes structure takes three times as long)
_STEP = struct.Struct("@PqPPqqii")
_ROWS = struct.Struct("@PPPPqqqqqqqqii")
_QUERY = struct.Struct("@PPqqqqiifi")
_I32 = torch.int32


class PagedCache:
    """CUDA tensors as a cache: keys and values as e4m3 codes [pages, heads, page_size, head_dim] (float8_e4m3fn or
    uint8; the last two dimensions contiguous) with fp32 scales [pages, heads]:
    value = code * scale.  page_size 16, 32, 64, 128 or 256; head_dim 64, 128 or 256."""

    def __init__(self, k, v, k_scale, v_scale):
        for x in (k, v):
            want(x.dim() == 4 and x.shape == k.shape, "k and v must be [pages, heads, page_size, head_dim]")
            if x.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError(f"k and v must be float8_e4m3fn or uint8, not {x.dtype}")
            want(x.stride() == k.stride(), "k and v must have the same strides")
        pages, heads, ps, d = k.shape
        want(k.stride(3) == 1 and k.stride(2) == d, "the rows of a page's head must be contiguous")
        for s in (k_scale, v_scale):
            want(s.shape == (pages, heads) and s.is_contiguous(), "scales must be contiguous [pages, heads]")
            if s.dtype != torch.float32:
                raise TypeError(f"scales must be float32, not {s.dtype}")
        want(len({x.device for x in (k, v, k_scale, v_scale)}) == 1, "the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, ps, d
        self.device = k.device
        self.index = k.get_device()
        self.default_scale = d ** -0.5
        self._c = serve.KvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0),
                                k.stride(1), pages, heads, ps, d)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, device="cuda"):
        """A cache whose pages hold nothing yet."""
        shape = (pages, heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    def attend_workspace(self, stream=None):
        """Zero-filled workspace for `attend` over caches of this shape (one per stream that uses it),
        made on the stream given, else on the current one."""
        n = int(serve.load().arc_kv_attend_workspace_bytes(self._ref))
        want(n > 0, "arc_kv_attend_workspace_bytes rejected the cache")
        return serve.new_workspace(self.k, n, True, stream)

    def shared_workspace(self, tokens: int, q_heads: int, stream=None):
        """Zero-filled workspace for `attend_shared` of up to so many new tokens over caches of this shape (one per
        stream that uses it), made on the stream given, else on the current one."""
        want(0 < q_heads < 1 << 31, "the heads must be positive and fit 32 bits")
        n = int(serve.load().arc_kv_attend_shared_workspace_bytes(self._ref, tokens, q_heads))
        want(n > 0, "arc_kv_attend_shared_workspace_bytes rejected the cache, the tokens or the heads")
        return serve.new_workspace(self.k, n, True, stream)


class Rope:
    """A position rotation: `turns` int64 [rot_dim / 2] on the device (64-bit fixed-point
    fractions of a turn per position, see rope_turns), the layout of the pairs ("half" or
    "interleaved") and the factor on the rotated values."""

    def __init__(self, turns, layout: str = "half", amplitude: float = 1.0):
        want(layout in LAYOUTS, f"layout must be one of {sorted(LAYOUTS)}")
        want(turns.dim() == 1 and turns.is_contiguous(), "turns must be contiguous [rot_dim / 2]")
        if turns.dtype != torch.int64:
            raise TypeError(f"turns must be int64, not {turns.dtype}")
        self.turns, self.layout, self.amplitude = turns, layout, float(amplitude)
        self.rot_dim = 2 * turns.numel()
        self._c = serve.RopeArgs(turns.data_ptr(), self.amplitude, self.rot_dim, LAYOUTS[layout], 0)
        self._ref = ctypes.addressof(self._c)


def rope_turns(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_length: int = 0, fast: float = 32.0, slow: float = 1.0):
    """(turns int64 [rot_dim / 2] on the host, amplitude) of a rotation.

    Pair i turns by base^(-2 i / rot_dim) radians a position.  For contexts `factor` times
    longer than those trained on:
      "linear"  every angle divided by the factor (position interpolation)
      "base"    the base raised so that the slowest pair turns `factor` times slower
      "parts"   pairs that turn less than `slow` times over original_length are
                interpolated, those that turn more than `fast` times are left alone, with a
                linear ramp between; amplitude 0.1 ln(factor) + 1 (Peng et al. 2023, "YaRN").  The
                ramp runs over the number of turns, as in the paper; where a model's own code ramps
                over the index of the pair instead, the pairs between turn differently: give that
                model's `turns` to Rope
    """
    want(rot_dim >= 0 and rot_dim % 2 == 0, "rot_dim must be even")
    want(scaling in (None, "linear", "base", "parts"), "scaling must be None, 'linear', 'base' or 'parts'")
    want(math.isfinite(base) and base > 1.0, "base must be above 1")
    want(scaling is None or (math.isfinite(factor) and factor >= 1.0), "factor must be at least 1")
    i = np.arange(rot_dim // 2, dtype=np.float64)
    amplitude = 1.0
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    freq = base ** (-2.0 * i / max(rot_dim, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        want(original_length > 0 and fast > slow > 0, "'parts' needs original_length > 0 and fast > slow > 0")
        turns = original_length * freq / (2.0 * math.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    return np.floor(freq / (2.0 * math.pi) * 2.0 ** 64).astype(np.uint64).astype(np.int64), amplitude


def _bad_heads(x, T, heads, dim, name):
    want(x.dim() == 3 and x.shape[0] == T and x.shape[2] == dim and (heads is None or x.shape[1] == heads),
         f"{name} must be [tokens, heads, head_dim] with head_dim {dim}" + ("" if heads is None else f", {heads} heads"))
    want(x.stride(2) == 1, f"the values of a head of {name} must be contiguous")


def _heads(x, T, heads, dim, name):
    """(token stride, head stride, heads) of a checked [T, heads, dim] tensor."""
    if x.dim() == 3:
        t, h, d = x.shape
        a, b, c = x.stride()
        if t == T and d == dim and c == 1 and (heads is None or h == heads):
            return a, b, h
    _bad_heads(x, T, heads, dim, name)
    raise ValueError(f"{name} has a shape that cannot be used")


def _step(cache, T, positions, page_table, row_offsets):
    """arc_kv_step as bytes."""
    want(page_table.dim() == 2, "page_table must be [sequences, pages]")
    B, pages = page_table.shape
    stride, one = page_table.stride()
    want(one == 1 or pages == 1, "rows of page_table must be contiguous")
    want(positions.shape == (B,) and positions.is_contiguous(), "positions must be contiguous [sequences]")
    offsets = 0
    if row_offsets is not None:
        want(row_offsets.shape == (B + 1,) and row_offsets.is_contiguous(), "row_offsets must be contiguous [sequences + 1]")
        if row_offsets.dtype != _I32:
            raise TypeError("row_offsets must be int32")
        want(row_offsets.get_device() == cache.index, "every tensor must be on the cache's device")
        offsets = row_offsets.data_ptr()
    else:
        want(T == B, "without row_offsets there is one new token for each sequence")
    if page_table.dtype != _I32 or positions.dtype != _I32:
        raise TypeError("page_table and positions must be int32")
    want(page_table.get_device() == cache.index and positions.get_device() == cache.index,
         "every tensor must be on the cache's device")
    return _STEP.pack(page_table.data_ptr(), stride if B > 1 else pages, positions.data_ptr(), offsets, B, T, pages, 0)


def append(cache: PagedCache, k, v, positions, page_table, q=None, q_out=None, rope: Rope | None = None,
           row_offsets=None, err_word=None, stream=None, check: bool = True):
    """arc_kv_append: store T new tokens' keys (rotated) and values, k and v [T, heads,
    head_dim] bfloat16 or float16 of any token and head strides; rotate q [T, q_heads,
    head_dim] into q_out (a new contiguous tensor where None; may be q itself), which is
    returned.  positions int32 [B]: tokens each sequence holds before these (negative:
    parked); page_table int32 [B, pages]; row_offsets int32 [B + 1] or None for one new
    token each; err_word int32 [1]: ARC_KV_ERR_* bits.  stream: as in `attend`."""
    T, dim, dev = k.shape[0], cache.head_dim, cache.index
    kt, kh, _ = _heads(k, T, cache.heads, dim, "k")
    vt, vh, _ = _heads(v, T, cache.heads, dim, "v")
    dtype, code = k.dtype, serve.dtype_code(k)
    want(v.dtype == dtype, "k and v must have one type")
    want(k.get_device() == dev and v.get_device() == dev, "every tensor must be on the cache's device")
    step = _step(cache, T, positions, page_table, row_offsets)
    serve.on_current_gpu(dev)
    qp = op = qt = qh = ot = oh = heads = 0
    if q is not None:
        qt, qh, heads = _heads(q, T, None, dim, "q")
        want(q.dtype == dtype and q.get_device() == dev, "q must have k's type and device")
        if q_out is None:
            q_out = serve.new_output(q, (T, heads, dim), (heads * dim, dim, 1), dtype, stream)
        elif q_out is not q:
            want(q_out.dtype == dtype and q_out.get_device() == dev, "q_out must have q's type and device")
        ot, oh, _ = _heads(q_out, T, heads, dim, "q_out")
        qp, op = q.data_ptr(), q_out.data_ptr()
    else:
        want(q_out is None, "q_out without q")
    if rope is not None:
        want(rope.turns.get_device() == dev, "every tensor must be on the cache's device")
    rows = _ROWS.pack(qp, k.data_ptr(), v.data_ptr(), op, qt, qh, kt, kh, vt, vh, ot, oh, heads, code)
    rc = serve.load().arc_kv_append(cache._ref, step, rows, None if rope is None else rope._ref,
                                    serve.err_word_ptr(err_word, dev), serve.stream_of(stream, dev))
    serve.finish(rc, check)
    return q_out


def attend(cache: PagedCache, q, positions, page_table, out=None, row_offsets=None, scale: float | None = None,
           window: int = 0, err_word=None, workspace=None, stream=None, check: bool = True, sinks: int = 0):
    """arc_kv_attend: attention of the step's tokens, q [T, q_heads, head_dim], over the cache
    that `append` has just extended (the same positions, page_table and row_offsets).  scale:
    head_dim ** -0.5 where None.  window > 0: each token sees its last `window` tokens, and the
    first `sinks` of its sequence (arc_kv_attend_sinks), alone.
    workspace: cache.attend_workspace(), made for the call where None.  Returns out.

    stream: where the call runs, the current stream where None.  What the call makes for itself (out,
    workspace) is made there; tensors given have to be ready there."""
    want(-1 << 31 <= sinks < 1 << 31, "sinks must fit 32 bits")
    T, dim, dev = q.shape[0], cache.head_dim, cache.index
    qt, qh, heads = _heads(q, T, None, dim, "q")
    code = serve.dtype_code(q)
    step = _step(cache, T, positions, page_table, row_offsets)
    want(q.get_device() == dev, "every tensor must be on the cache's device")
    serve.on_current_gpu(dev)
    if out is None:
        out = serve.new_output(q, (T, heads, dim), (heads * dim, dim, 1), q.dtype, stream)
        ot, oh = heads * dim, dim
    else:
        ot, oh, _ = _heads(out, T, heads, dim, "out")
        want(out.dtype == q.dtype and out.get_device() == dev, "out must have q's type and device")
    if workspace is None:
        workspace = cache.attend_workspace(stream)
    wp, wn = serve.workspace_of(workspace, dev)
    query = _QUERY.pack(q.data_ptr(), out.data_ptr(), qt, qh, ot, oh, heads, code,
                        cache.default_scale if scale is None else scale, window)
    err, handle = serve.err_word_ptr(err_word, dev), serve.stream_of(stream, dev)
    if sinks:
        rc = serve.load().arc_kv_attend_sinks(cache._ref, step, query, sinks, err, wp, wn, handle)
    else:
        rc = serve.load().arc_kv_attend(cache._ref, step, query, err, wp, wn, handle)
    serve.finish(rc, check)
    return out


def attend_shared(cache: PagedCache, q, positions, page_table, prefix, out=None, row_offsets=None,
                  scale: float | None = None, err_word=None, workspace=None, stream=None, check: bool = True):
    """arc_kv_attend_shared: `attend` for sequences that all begin with the same tokens, whose whole pages `prefix`
    int32 [pages] names: they are read once for the batch.  page_table keeps a sequence's pages in their places; the
    entries under the prefix are not read.  Every sequence's position lies at or past the prefix's end.  The prefix's scales
    lie in [2^-32, 2^32] (negative, NaN and larger ones set ARC_KV_ERR_SCALE) or, those of values, are 0; scale * q . k *
    log2(e) lies below 2^22 (rows beyond may be NaN).  workspace: cache.shared_workspace(tokens, q_heads), made for the call
    where None.  Returns out.  stream: as in `attend`."""
    T, dim, dev = q.shape[0], cache.head_dim, cache.index
    qt, qh, heads = _heads(q, T, None, dim, "q")
    code = serve.dtype_code(q)
    step = _step(cache, T, positions, page_table, row_offsets)
    want(q.get_device() == dev, "every tensor must be on the cache's device")
    want(prefix.dim() == 1 and prefix.is_contiguous(), "prefix must be contiguous [pages]")
    if prefix.dtype != _I32:
        raise TypeError("prefix must be int32")
    want(prefix.get_device() == dev, "every tensor must be on the cache's device")
    serve.on_current_gpu(dev)
    if out is None:
        out = serve.new_output(q, (T, heads, dim), (heads * dim, dim, 1), q.dtype, stream)
        ot, oh = heads * dim, dim
    else:
        ot, oh, _ = _heads(out, T, heads, dim, "out")
        want(out.dtype == q.dtype and out.get_device() == dev, "out must have q's type and device")
    if workspace is None:
        workspace = cache.shared_workspace(T, heads, stream)
    wp, wn = serve.workspace_of(workspace, dev)
    query = _QUERY.pack(q.data_ptr(), out.data_ptr(), qt, qh, ot, oh, heads, code,
                        cache.default_scale if scale is None else scale, 0)
    rc = serve.load().arc_kv_attend_shared(cache._ref, step, query, prefix.data_ptr(), prefix.numel(),
                                           serve.err_word_ptr(err_word, dev), wp, wn, serve.stream_of(stream, dev))
    serve.finish(rc, check)
    return out

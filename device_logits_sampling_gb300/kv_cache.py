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

import numpy as np

from . import sampler, serve
from .serve import want

ARC_KV_ERR_PAGE = 0x1
ARC_KV_ERR_POSITION = 0x2
ARC_KV_ERR_NAN = 0x4
ARC_KV_ERR_OFFSETS = 0x8
E4M3_MAX = 448.0
SCALE_EXP = 32  # page scales written by append lie in [2^-32, 2^32]
LAYOUTS = {"half": 0, "interleaved": 1}


class PagedCache:
    """Keys and values as e4m3 codes [pages, heads, page_size, head_dim] (float8_e4m3fn or
    uint8; the last two dimensions contiguous) with fp32 scales [pages, heads]:
    value = code * scale.  page_size 16, 32, 64, 128 or 256; head_dim 64, 128 or 256."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch

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
        self._c = serve.KvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0),
                                k.stride(1), pages, heads, ps, d)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, device="cuda"):
        """A cache whose pages hold nothing yet."""
        import torch

        shape = (pages, heads, page_size, head_dim)
        k, v = (torch.empty(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    def attend_workspace(self):
        """Zero-filled workspace for `attend` over caches of this shape (one per stream that uses it)."""
        import torch

        n = int(serve.load().arc_kv_attend_workspace_bytes(self._ref))
        want(n > 0, "arc_kv_attend_workspace_bytes rejected the cache")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)


class Rope:
    """A position rotation: `turns` int64 [rot_dim / 2] on the device (64-bit fixed-point
    fractions of a turn per position, see rope_turns), the layout of the pairs ("half" or
    "interleaved") and the factor on the rotated values."""

    def __init__(self, turns, layout: str = "half", amplitude: float = 1.0):
        import torch

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
                linear ramp between; amplitude 0.1 ln(factor) + 1 (Peng et al. 2023, "YaRN")
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


def _check_heads(x, T, heads, dim, name):
    want(x.dim() == 3 and x.shape[0] == T and x.shape[2] == dim and (heads is None or x.shape[1] == heads),
         f"{name} must be [tokens, heads, head_dim] with head_dim {dim}" + ("" if heads is None else f", {heads} heads"))
    want(x.stride(2) == 1, f"the values of a head of {name} must be contiguous")


def _step(cache, T, positions, page_table, row_offsets):
    import torch

    want(page_table.dim() == 2 and page_table.stride(1) == 1, "page_table must be [sequences, pages], rows contiguous")
    B = page_table.shape[0]
    want(positions.shape == (B,) and positions.is_contiguous(), "positions must be contiguous [sequences]")
    ints = [page_table, positions]
    if row_offsets is not None:
        want(row_offsets.shape == (B + 1,) and row_offsets.is_contiguous(), "row_offsets must be contiguous [sequences + 1]")
        ints.append(row_offsets)
    else:
        want(T == B, "without row_offsets there is one new token for each sequence")
    for x in ints:
        if x.dtype != torch.int32:
            raise TypeError("page_table, positions and row_offsets must be int32")
        want(x.device == cache.device, "every tensor must be on the cache's device")
    return serve.KvStep(page_table.data_ptr(), page_table.stride(0) if B > 1 else page_table.shape[1],
                        positions.data_ptr(), None if row_offsets is None else row_offsets.data_ptr(), B, T,
                        page_table.shape[1], 0)


def append(cache: PagedCache, k, v, positions, page_table, q=None, q_out=None, rope: Rope | None = None,
           row_offsets=None, err_word=None, stream=None, check: bool = True):
    """arc_kv_append: store T new tokens' keys (rotated) and values, k and v [T, heads,
    head_dim] bfloat16 or float16 of any token and head strides; rotate q [T, q_heads,
    head_dim] into q_out (a new contiguous tensor where None; may be q itself), which is
    returned.  positions int32 [B]: tokens each sequence holds before these (negative:
    parked); page_table int32 [B, pages]; row_offsets int32 [B + 1] or None for one new
    token each; err_word int32 [1]: ARC_KV_ERR_* bits."""
    import torch

    T = k.shape[0]
    _check_heads(k, T, cache.heads, cache.head_dim, "k")
    _check_heads(v, T, cache.heads, cache.head_dim, "v")
    want(k.dtype == v.dtype, "k and v must have one type")
    want(k.device == cache.device and v.device == cache.device, "every tensor must be on the cache's device")
    rows = serve.KvRows(None, k.data_ptr(), v.data_ptr(), None, 0, 0, k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                        0, 0, 0, serve.dtype_code(k))
    if q is not None:
        _check_heads(q, T, None, cache.head_dim, "q")
        want(q.dtype == k.dtype and q.device == cache.device, "q must have k's type and device")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif q_out is not q:
            _check_heads(q_out, T, q.shape[1], cache.head_dim, "q_out")
            want(q_out.dtype == q.dtype and q_out.device == q.device, "q_out must have q's type and device")
        rows.q, rows.q_out, rows.q_heads = q.data_ptr(), q_out.data_ptr(), q.shape[1]
        rows.q_token_stride, rows.q_head_stride = q.stride(0), q.stride(1)
        rows.out_token_stride, rows.out_head_stride = q_out.stride(0), q_out.stride(1)
    else:
        want(q_out is None, "q_out without q")
    if rope is not None:
        want(rope.turns.device == cache.device, "every tensor must be on the cache's device")
    step = _step(cache, T, positions, page_table, row_offsets)
    rc = serve.load().arc_kv_append(cache._ref, ctypes.addressof(step), ctypes.addressof(rows),
                                    None if rope is None else rope._ref, sampler._ptr(err_word), serve.stream_of(stream, cache.device))
    serve.finish(rc, check)
    return q_out


def attend(cache: PagedCache, q, positions, page_table, out=None, row_offsets=None, scale: float | None = None,
           window: int = 0, err_word=None, workspace=None, stream=None, check: bool = True):
    """arc_kv_attend: attention of the step's tokens, q [T, q_heads, head_dim], over the cache
    that `append` has just extended (the same positions, page_table and row_offsets).  scale:
    head_dim ** -0.5 where None.  window > 0: each token sees its last `window` tokens alone.
    workspace: cache.attend_workspace(), made for the call where None.  Returns out."""
    import torch

    T = q.shape[0]
    _check_heads(q, T, None, cache.head_dim, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _check_heads(out, T, q.shape[1], cache.head_dim, "out")
        want(out.dtype == q.dtype, "out must have q's type")
    want(q.device == cache.device and out.device == cache.device, "every tensor must be on the cache's device")
    if workspace is None:
        workspace = cache.attend_workspace()
    query = serve.KvQuery(q.data_ptr(), out.data_ptr(), q.stride(0), q.stride(1), out.stride(0), out.stride(1),
                          q.shape[1], serve.dtype_code(q), cache.head_dim ** -0.5 if scale is None else scale, int(window))
    step = _step(cache, T, positions, page_table, row_offsets)
    rc = serve.load().arc_kv_attend(cache._ref, ctypes.addressof(step), ctypes.addressof(query), sampler._ptr(err_word),
                                    workspace.data_ptr(), workspace.numel(), serve.stream_of(stream, cache.device))
    serve.finish(rc, check)
    return out

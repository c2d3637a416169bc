"""fp64 reference of the paged 8-bit cache: e4m3 rounding, append, attention.

Test infrastructure only; numpy on the host, loops over sequences and pages.
"""
import math

import numpy as np

E4M3_MAX = 448.0
SCALE_EXP = 32
ERR_PAGE, ERR_POSITION, ERR_NAN, ERR_SCALE = 1, 2, 4, 16


def decode_table() -> np.ndarray:
    """The 256 e4m3 values (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7F and 0xFF are NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if (c & 0x7F) == 0x7F else (-v if c & 0x80 else v)
    return out


TABLE = decode_table()
_MIDS = (TABLE[1:0x7F] + TABLE[:0x7E]) / 2


def encode(x) -> np.ndarray:
    """Nearest e4m3 codes of fp64 values: ties to the even code, magnitudes above 448 saturate, NaN counts as 0."""
    x = np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=1e300, neginf=-1e300)
    a = np.abs(x)
    i = np.searchsorted(_MIDS, a, side="left")
    tie = (i < len(_MIDS)) & (a == _MIDS[np.minimum(i, len(_MIDS) - 1)])
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    return (i + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    """Least e in [-32, 32] with amax <= 448 * 2^e."""
    e = -SCALE_EXP
    while e < SCALE_EXP and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e


def angles(turns, position: int) -> np.ndarray:
    """Radians of each pair: position * turns modulo 2^64, as a fraction of a turn."""
    frac = np.array([(int(position) * int(t)) % (1 << 64) for t in turns], dtype=object)
    return np.array([2.0 * math.pi * (int(f) / 2.0 ** 64) for f in frac])


def rotate(x, position: int, turns, amplitude: float, layout: str) -> np.ndarray:
    """x [..., head_dim] fp64 with its first 2 len(turns) values turned."""
    y = np.array(x, dtype=np.float64)
    n = len(turns)
    if n == 0:
        return y
    a = angles(turns, position)
    c, s = np.cos(a) * amplitude, np.sin(a) * amplitude
    one, two = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    with np.errstate(invalid="ignore"):
        p, q = np.array(y[..., one]), np.array(y[..., two])
        y[..., one] = p * c - q * s
        y[..., two] = q * c + p * s
    return y


def append(k, v, k_scale, v_scale, new_k, new_v, positions, table, offsets, turns=(), amplitude=1.0, layout="half") -> int:
    """Append to codes k, v [pages, heads, page_size, dim] and scales [pages, heads] in place; error bits."""
    pages, heads, ps, _ = k.shape
    err = 0
    for b in range(len(positions)):
        n = int(offsets[b + 1] - offsets[b])
        if positions[b] < 0:
            continue
        at, end, row = int(positions[b]), int(positions[b]) + n, int(offsets[b])
        while at < end:
            pi, slot = divmod(at, ps)
            take = min(ps - slot, end - at)
            if pi >= table.shape[1]:
                err |= ERR_POSITION
            elif not 0 <= table[b, pi] < pages:
                err |= ERR_PAGE
            else:
                p = int(table[b, pi])
                for h in range(heads):
                    for codes, scale, new, turn in ((k, k_scale, new_k, True), (v, v_scale, new_v, False)):
                        x = np.array(new[row:row + take, h], dtype=np.float64)
                        if turn:
                            x = np.stack([rotate(x[i], at + i, turns, amplitude, layout) for i in range(take)])
                        if np.isnan(x).any():
                            err |= ERR_NAN
                            x = np.where(np.isnan(x), 0.0, x)
                        now = 2.0 ** scale_exponent(float(np.abs(x).max()))
                        if slot:
                            old = float(scale[p, h])
                            if not 2.0 ** -SCALE_EXP <= old <= 2.0 ** SCALE_EXP:
                                err |= ERR_SCALE
                                continue
                            if now > old:
                                was = codes[p, h, :slot].copy()  # a NaN code stays one (without its sign)
                                again = encode(TABLE[was] * (old / now))
                                codes[p, h, :slot] = np.where((was & 0x7F) == 0x7F, 0x7F, again)
                            now = max(now, old)
                        scale[p, h] = now
                        codes[p, h, slot:slot + take] = encode(x / now)
            at, row = at + take, row + take
    return err


def gather(codes, scale, table_row, length: int, head: int) -> np.ndarray:
    """Values [length, dim] of one sequence's cached head."""
    ps = codes.shape[2]
    rows = [TABLE[codes[p, head]] * float(scale[p, head]) for p in table_row[: -(-length // ps)]]
    return np.concatenate(rows)[:length] if rows else np.zeros((0, codes.shape[3]))


def attend(k, v, k_scale, v_scale, q, positions, table, offsets, scale=None, window=0, sinks=0):
    """(out, spread) [T, q_heads, dim]: the attention, and sum_j p_j |v_j|, which bounds its rounding errors."""
    T, hq, d = q.shape
    heads, ps = k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, spread = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    for b in range(len(positions)):
        n = int(offsets[b + 1] - offsets[b])
        if positions[b] < 0 or n == 0:
            continue
        length = int(positions[b]) + n
        first = max(0, int(positions[b]) + 1 - window) if window else 0
        need = table[b, first // ps: -(-length // ps)]
        front = min(-(-sinks // ps), first // ps) if window else 0  # pages of first tokens before the window's
        need = np.concatenate([table[b, :front], need])
        if -(-length // ps) > table.shape[1] or (need < 0).any() or (need >= k.shape[0]).any():
            out[offsets[b]:offsets[b + 1]] = np.nan
            continue
        skip = (first // ps - front) * ps  # tokens between them that nobody sees
        for h in range(heads):
            kk = gather(k, k_scale, need, length - skip, h)
            vv = gather(v, v_scale, need, length - skip, h)
            for i in range(n):
                p = int(positions[b]) + i
                lo = max(0, p + 1 - window) if window else 0
                at = np.concatenate([np.arange(min(sinks, lo)), np.arange(lo, p + 1)])
                at = np.where(at < front * ps, at, at - skip)  # a window's token behind the front pages
                t = int(offsets[b]) + i
                grp = slice(h * (hq // heads), (h + 1) * (hq // heads))
                s = q[t, grp].astype(np.float64) @ kk[at].T * scale
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                out[t, grp], spread[t, grp] = w @ vv[at], w @ np.abs(vv[at])
    return out, spread

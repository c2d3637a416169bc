"""Reference of the logit edits: penalties, biases, mask.

Test infrastructure only; numpy on the host, loops over rows and list entries.  Each edit is one fp32
operation after another, rounded to nearest, so the result is the kernel's bit for bit."""
import numpy as np

ERR_PARAM, ERR_HIST, ERR_BIAS, ERR_MASK = 1, 2, 4, 8
F = np.float32


def _part(offsets, r, n):
    lo, hi = int(offsets[r]), int(offsets[r + 1])
    return (lo, hi, True) if 0 <= lo <= hi <= n else (0, 0, False)


def edit(logits, penalties=None, hist_offsets=None, hist_ids=None, bias_offsets=None, bias_ids=None, bias=None,
         allowed=None, allowed_rows=None):
    """(logits fp32 [B, V], error bits) of fp32 logits; penalties [B, 3]; allowed: truth values [masks, V]."""
    z = np.array(logits, dtype=F)
    B, V = z.shape
    err = 0
    with np.errstate(all="ignore"):
        for r in range(B):
            if hist_offsets is not None:
                lo, hi, ok = _part(hist_offsets, r, len(hist_ids))
                err |= 0 if ok else ERR_HIST
                rep, freq, pres = (F(p) for p in penalties[r])
                if not (rep > 0 and np.isfinite([rep, freq, pres]).all()):
                    err |= ERR_PARAM
                    hi = lo
                ids = np.asarray(hist_ids[lo:hi], dtype=np.int64)
                err |= ERR_HIST if ((ids < 0) | (ids >= V)).any() else 0
                for i, c in zip(*np.unique(ids[(ids >= 0) & (ids < V)], return_counts=True)):
                    x = z[r, i]
                    x = F(x / rep) if x > 0 else F(x * rep)
                    x = F(x - F(F(c) * freq))
                    z[r, i] = F(x - pres)
            if bias_offsets is not None:
                lo, hi, ok = _part(bias_offsets, r, len(bias_ids))
                err |= 0 if ok else ERR_BIAS
                last = {}
                for e in range(lo, hi):
                    if 0 <= bias_ids[e] < V:
                        last[int(bias_ids[e])] = F(bias[e])
                    else:
                        err |= ERR_BIAS
                for i, b in last.items():
                    z[r, i] = F(z[r, i] + b)
            if allowed is not None:
                m = r if allowed_rows is None else int(allowed_rows[r])
                if m >= len(allowed):
                    err |= ERR_MASK
                    z[r] = -np.inf
                elif m >= 0:
                    z[r, ~np.asarray(allowed[m], dtype=bool)] = -np.inf
    return z, err

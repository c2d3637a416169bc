"""fp64 reference of the join around a block: post norm, gate, scaled residual sum, norm.

Test infrastructure only; numpy on the host."""
import numpy as np


def rms(x, eps: float):
    """1 / rms of the rows of x."""
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def join(x, y=None, weight=None, post_weight=None, gate=None, sigmoid=False, alpha=1.0, offset=0.0, eps=1e-6):
    """(h, n, u): the sum, its norm, and what was added to x before alpha; all fp64 [rows, dim]."""
    x = np.asarray(x, dtype=np.float64)
    u = np.zeros_like(x) if y is None else np.array(y, dtype=np.float64)
    if post_weight is not None:
        u = u * rms(u, eps) * (offset + np.asarray(post_weight, dtype=np.float64))
    if gate is not None:
        g = np.asarray(gate, dtype=np.float64)
        with np.errstate(over="ignore"):
            u = u * (1.0 / (1.0 + np.exp(-g)) if sigmoid else g)
    h = x + alpha * u
    n = h * rms(h, eps)
    if weight is not None:
        n = n * (offset + np.asarray(weight, dtype=np.float64))
    return h, n, u

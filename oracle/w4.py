"""fp64 reference of the 4-bit products.  Test infrastructure only."""
import numpy as np


def unpack(weight) -> np.ndarray:
    """uint8 [outs, ins / 2] -> [outs, ins] of 0 .. 15, the low half of a byte first."""
    w = np.empty((weight.shape[0], 2 * weight.shape[1]), dtype=np.float64)
    w[:, 0::2], w[:, 1::2] = weight & 15, weight >> 4
    return w


def matvec(x, weight, scales, zeros=None):
    """(y, spread) [rows, outs]: the products, and sum_k |x_k| 15 s, which bounds the partial sums."""
    q = unpack(weight)
    group = q.shape[1] // scales.shape[1]
    s = np.repeat(scales.astype(np.float64), group, 1)
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)
    x = x.astype(np.float64)
    return x @ ((q - z) * s).T, np.abs(x) @ (15.0 * np.abs(s)).T

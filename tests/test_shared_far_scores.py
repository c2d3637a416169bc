"""attend_shared with scores far from 0, as large key scales give: exact where all of a row's lie below 2^22 (as powers of
two), NaN where its largest does not, and one or the other between; never a wrong number."""
import math

import numpy as np
import pytest

from oracle import kv_cache as ok
from test_attend_shared import run, shared_case


def check_far(c):
    """One token a sequence; (rows that have to be right, rows that have to be NaN)."""
    got = run(c, single=True).double().cpu().numpy()
    want, spread = ok.attend(c.k, c.v, c.ks, c.vs, c.q.double().numpy(), c.positions, c.table, c.offsets)
    group, front = c.q_heads // c.heads, len(c.prefix) * c.page
    near, far = np.zeros(got.shape[:2], bool), np.zeros(got.shape[:2], bool)
    for b in range(len(c.positions)):
        for h in range(c.heads):
            rows = slice(h * group, (h + 1) * group)
            k = ok.gather(c.k, c.ks, c.table[b], front, h)
            s = c.q[b, rows].double().numpy() @ k.T * (c.dim ** -0.5 * math.log2(math.e))
            near[b, rows] = (np.abs(s) < 2.0 ** 22 - 16).all(-1)
            far[b, rows] = np.abs(s.max(-1)) > 2.0 ** 22 + 16  # (the room above it, and fp32 roundings)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -25 * (c.positions.max() + 1) * 448.0 * c.vs.max()
    nan = np.isnan(got)
    assert nan[far].all() and not nan[near].any()
    assert (np.abs(got - want) <= tol)[~nan].all()
    return int(near.sum()), int(far.sum())


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads,group,front", [(64, 16, 2, 4, 60), (128, 64, 8, 4, 130), (256, 32, 4, 3, 200)])
@pytest.mark.parametrize("exponents", [(10, 11), (14, 15), (17, 18), (20, 21), (24, 25), (32, 33), (-9, 33)])
def test_large_key_scales(cuda_lib, dim, page, heads, group, front, exponents):
    c = shared_case(101, dim, page, heads, group, front, [5, 200, 31], [1] * 3)
    c.ks[:] = 2.0 ** c.rng.integers(*exponents, c.ks.shape)
    near, far = check_far(c)
    assert near + far > 0


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exponent", [8, 28])
def test_scores_far_below_zero(cuda_lib, dim, exponent):
    """Every score negative: keys against the query's direction."""
    import torch

    c = shared_case(102, dim, 16, 1, 2, 50, [9, 40], [1] * 2)
    c.q = torch.ones_like(c.q)
    c.k[:] = 0x80 | c.rng.integers(0x20, 0x78, c.k.shape, dtype=np.uint8)
    c.ks[:] = 2.0 ** exponent
    near, far = check_far(c)
    assert (near if exponent == 8 else far) == c.q[:, :, 0].numel()

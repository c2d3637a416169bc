"""Scales of a shared prefix's pages that append does not write: under value scales of 0 and below 2^-60 the values count as
zeros; negative, NaN and too large scales, of keys or values, are reported and spoil their head's rows."""
import numpy as np
import pytest

from device_logits_sampling_gb300 import kv_cache
from test_attend_shared import check, run, shared_case


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,front", [(64, 16, 37), (128, 16, 37), (128, 256, 5), (256, 16, 21), (256, 64, 5)])
@pytest.mark.parametrize("where", ["first", "first chunk", "middle", "last", "every other", "all but one", "all"])
def test_pages_of_scale_zero(cuda_lib, dim, page, front, where):
    """Their tokens keep their weights: the others' values count that much less."""
    c = shared_case(93, dim, page, 2, 3, front, [40, 3, None, 90], [1] * 4)
    c.ks[:] = 2.0 ** -9  # scores near one another: every page counts
    c.vs[c.prefix] = 2.0 ** c.rng.integers(-9, -2, (front, 2))
    at = {"first": [0], "first chunk": range(min(front, -(-128 // page))), "middle": [front // 2], "last": [front - 1],
          "every other": range(0, front, 2), "all but one": [i for i in range(front) if i != front - 2], "all": range(front)}[where]
    for zero in (0.0, 2.0 ** -100):
        c.vs[c.prefix[list(at)]] = zero
        check(c, single=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_head_of_scale_zero(cuda_lib, dim):
    """Zero scales of one cached head leave the other's alone; small scales stay exact beside them."""
    c = shared_case(94, dim, 16, 2, 2, 40, [7, 30], [1] * 2)
    c.vs[:] = 2.0 ** c.rng.integers(-30, -20, c.vs.shape)
    c.ks[:] = 2.0 ** -9
    c.vs[c.prefix[::3], 0] = 0
    check(c, single=True, exact_columns=True)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [-1.0, float("nan"), float("inf"), 2.0 ** 33])
def test_scales_out_of_range_are_reported(cuda_lib, which, value):
    import torch

    c = shared_case(95, 128, 32, 2, 2, 9, [7, None, 30], [1] * 3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(c, single=True, err_word=err)
    assert int(err) == 0
    getattr(c, which)[c.prefix[5], 1] = value
    got = run(c, single=True, err_word=err).float().cpu().numpy()
    assert int(err) == kv_cache.ARC_KV_ERR_SCALE
    assert np.isnan(got[[0, 2], 2:]).all() and np.isfinite(got[:, :2]).all() and (got[1] == 0).all()

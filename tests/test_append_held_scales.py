"""Pages that already hold tokens under a scale that append has not written: any number of [2^-32, 2^32] stays
where it need not grow, with the older codes as they are; a scale that grows takes the older values along; one
outside the range is reported, and the page left alone."""
import math

import numpy as np
import pytest

from test_kv_cache import Case, check_append
from oracle import kv_cache as ok

POSITIONS, PIECES = [3, 15, 16, 40, 7, 9, 0, -1], [2, 3, 1, 20, 1, 1, 5, 2]


def case(seed, single, dim=64, **kw):
    c = Case(seed, dim, 16, 2, 2, POSITIONS, [1] * 8 if single else PIECES, "bf16", **kw)
    rng = np.random.default_rng(seed)
    c.ks, c.vs = ((2.0 ** rng.integers(-12, 3, c.ks.shape) * (1.0 + rng.random(c.ks.shape))).astype(np.float32).astype(np.float64)
                  for _ in range(2))
    return c


def test_the_oracle_keeps_older_values():
    k = np.full((1, 1, 16, 4), 0x38, np.uint8)  # ones
    for scale, new, want in ((1.5, 1.5, 1.5), (1.5, 1000.0, 4.0), (2.0, 3.0, 2.0)):
        codes, s = k.copy(), np.full((1, 1), scale)
        x = np.full((1, 1, 4), new)
        assert ok.append(codes, k.copy(), s, np.ones((1, 1)), x, np.zeros_like(x), [3], np.zeros((1, 1), int), [0, 1]) == 0
        assert s[0, 0] == want
        got = ok.TABLE[codes[0, 0, :4]] * want
        assert np.abs(got[:3] / scale - 1.0).max() <= 2.0 ** -4 and np.abs(got[3] / new - 1.0).max() <= 2.0 ** -4
    for scale in (0.0, math.nan, math.inf, -1.0, 2.0 ** 33):
        codes, s = k.copy(), np.full((1, 1), scale)
        assert ok.append(codes, k.copy(), s, np.ones((1, 1)), x, x, [3], np.zeros((1, 1), int), [0, 1]) == ok.ERR_SCALE
        assert np.array_equal(codes, k)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("dim,rot,layout", [(64, 64, "half"), (128, 20, "half"), (64, 32, "interleaved"), (256, 0, "half")])
def test_any_scale_is_kept_or_grows(cuda_lib, single, dim, rot, layout):
    for seed in range(51, 55):
        check_append(case(seed, single, dim, rot=rot, layout=layout, amp=1.1), single=single)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
def test_the_older_tokens_keep_their_codes(cuda_lib, single):
    c = case(56, single)
    c.ks[:], c.vs[:] = 1.5, float(np.float32(1.9))  # what the device holds
    cache = check_append(c, single=single)
    p = c.table[0, 0]
    assert np.array_equal(cache.v[p, :, :3].cpu().numpy(), c.v[p, :, :3])
    assert cache.k_scale[p, 0].item() == 1.5


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
def test_scales_out_of_range_are_reported(cuda_lib, single):
    for bad in (0.0, math.nan, math.inf, -1.0, 2.0 ** 33, 2.0 ** -33):
        c = case(57, single)
        c.ks[c.table[0, 0], 1] = bad  # one head of a page that holds tokens
        c.vs[c.table[6, 0]] = bad     # a page whose first token is new: what it held does not matter
        before = c.k.copy()
        import torch
        from device_logits_sampling_gb300 import kv_cache

        cache, pos, table, offs = c.device()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv_cache.append(cache, c.nk.cuda(), c.nv.cuda(), pos, table, rope=c.rope(), row_offsets=None if single else offs,
                        err_word=err)
        ek, ev, eks, evs = c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy()
        want = ok.append(ek, ev, eks, evs, c.nk.double().numpy(), c.nv.double().numpy(), c.positions, c.table, c.offsets, c.turns,
                         1.0, c.layout)
        assert int(err.item()) == want == kv_cache.ARC_KV_ERR_SCALE
        got = cache.k.cpu().numpy()
        assert np.array_equal(got[c.table[0, 0], 1], before[c.table[0, 0], 1])
        for g, w in ((got, ek), (cache.v.cpu().numpy(), ev)):
            zero = (w & 0x7F) == 0  # the sign of a zero carries nothing
            assert np.array_equal(g & 0x7F, w & 0x7F) and np.array_equal(g[~zero], w[~zero])
        for g, w in ((cache.k_scale, eks), (cache.v_scale, evs)):
            assert np.array_equal(g.cpu().numpy(), w.astype(np.float32), equal_nan=True)

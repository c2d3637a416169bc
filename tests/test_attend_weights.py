"""Which tokens an attention output is made of: small weights, pages whose value scales are far apart, and long
sequences whose weights are all alike, so that every piece of the line and every join counts.

Tolerance: half a step of the output's type, and (2^-11 + 2^-12) sum p |v| (half a step of a weight as fp16, and
the fp32 scores). There is no absolute term: it holds where the scores of a step of 16 tokens (32 for heads of 64)
lie within 28 powers of two of the step's largest, which each case asserts."""
import math

import numpy as np
import pytest

from device_logits_sampling_gb300 import kv_cache
from oracle import kv_cache as ok


class Cache:
    """One or more sequences of `lengths` tokens, their pages in random order, one new token each."""

    def __init__(self, seed, dim, page, heads, group, lengths, news=None):
        self.rng = np.random.default_rng(seed)
        self.dim, self.page, self.heads, self.q_heads, self.lengths = dim, page, heads, heads * group, lengths
        self.news = news or [1] * len(lengths)
        need = [-(-n // page) for n in lengths]
        ids = self.rng.permutation(sum(need))
        self.table = np.zeros((len(lengths), max(need)), np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (sum(need), heads, page, dim)
        self.k, self.v = np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)
        self.ks, self.vs = np.ones(shape[:2]), np.ones(shape[:2])
        self.q = np.zeros((sum(self.news), self.q_heads, dim), np.float32)
        self.offsets = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        self.positions = np.array([n - m for n, m in zip(lengths, self.news)], np.int32)

    def at(self, b, token):
        return self.table[b, token // self.page], slice(None), token % self.page

    def check(self, dtype, window=0, most=None, span=28.0):
        import torch

        t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        q = torch.from_numpy(self.q).to(t)
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        f32 = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()  # noqa: E731
        cache = kv_cache.PagedCache(torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda(), f32(self.ks), f32(self.vs))
        single = all(n == 1 for n in self.news)
        got = kv_cache.attend(cache, q.cuda(), i32(self.positions), i32(self.table), window=window,
                              row_offsets=None if single else i32(self.offsets)).double().cpu().numpy()
        q = q.double().numpy()
        for b, n in enumerate(self.lengths):
            for h in range(self.heads):
                row = self.table[b, :-(-n // self.page)]
                kk, vv = (ok.gather(c, s, row, n, h) for c, s in ((self.k, self.ks), (self.v, self.vs)))
                for i in range(self.news[b]):
                    p = int(self.positions[b]) + i
                    lo = max(0, p + 1 - window) if window else 0
                    r, heads = int(self.offsets[b]) + i, slice(h * (self.q_heads // self.heads), (h + 1) * (self.q_heads // self.heads))
                    s = q[r, heads] @ kk[lo:p + 1].T * self.dim ** -0.5
                    step = 32 if self.dim == 64 else 16
                    steps = [s[:, j:j + step] / math.log(2.0) for j in range(0, s.shape[1], step)]
                    assert max(float((x.max(1) - x.min(1)).max()) for x in steps) <= span
                    w = np.exp(s - s.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    if most is not None:  # no few tokens carry the result
                        assert w.max() * s.shape[1] <= most
                    want, spread = w @ vv[lo:p + 1], w @ np.abs(vv[lo:p + 1])
                    tol = torch.finfo(t).eps / 2 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + torch.finfo(t).tiny
                    off = np.abs(got[r, heads] - want)
                    assert (off <= tol).all(), (b, h, i, float((off / tol).max()))
        return got


SHAPES = [(64, 16, 1), (64, 16, 16), (64, 64, 4), (128, 16, 5), (128, 64, 16), (256, 32, 3)]  # tiles of 8 and of 16 rows


def large_beside_small(dim, page, heads, group, lengths, apart):
    """Equal scores; every other page has a scale 2^apart times larger, set by one token's first value, and zeros
    elsewhere: the other values of the output are the small pages' alone."""
    c = Cache(1, dim, page, heads, group, lengths)
    small, large = 2.0 ** (-apart // 2), 2.0 ** (apart - apart // 2)
    for b in range(len(lengths)):
        for i in range(c.table.shape[1]):
            p = c.table[b, i]
            c.vs[p] = large if i % 2 else small
            if i % 2:
                c.v[p, :, 1, 0] = 0x7E  # 448
            else:
                c.v[p] = c.rng.integers(0x30, 0x41, c.v[p].shape)
    c.check("bf16", most=1.001)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,group", SHAPES)
@pytest.mark.parametrize("apart", [0, 14, 20, 22, 26, 40, 62])
def test_a_large_scale_beside_small_ones(cuda_lib, dim, page, group, apart):
    large_beside_small(dim, page, 2, group, [16 * page, 16 * page - 3], apart)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,group", [(64, 16, 128), (64, 64, 200), (128, 16, 128), (128, 64, 200), (256, 32, 120)])
@pytest.mark.parametrize("apart", [0, 26, 62])
def test_a_large_scale_beside_small_ones_in_one_warp(cuda_lib, dim, page, group, apart):
    """So many query heads that each warp of the launch takes ten and more steps in a row."""
    large_beside_small(dim, page, 1, group, [20001], apart)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,group", SHAPES)
def test_many_small_weights_count(cuda_lib, dim, page, group):
    """One token holds nearly all the weight, with a value of zero; 6,000 others, 2^-25.2 of it each, make the
    output."""
    c = Cache(2, dim, page, 1, group, [6000])
    c.q[:, :, 0] = 16.0
    c.v[:] = c.rng.integers(0x30, 0x41, c.v.shape)
    sink = c.at(0, 2777)
    c.k[sink][:, 0] = 0x38  # 1; the others' keys are 0: scores apart by 16 ks / sqrt(dim)
    c.ks[:] = float(np.float32(25.2 * math.log(2.0) * dim ** 0.5 / 16.0))
    c.v[sink] = 0
    c.check("bf16")
    c.check("fp16")


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,group", SHAPES)
@pytest.mark.parametrize("up", [True, False])
def test_scores_that_climb_and_fall(cuda_lib, dim, page, group, up):
    """From page to page scores rise (or fall) by two powers of two and value scales the other way, so that every
    page counts alike."""
    pages = 24
    c = Cache(3, dim, page, 1, group, [pages * page - 5])
    c.q[:, :, 0] = 1.0
    c.v[:] = c.rng.integers(0x30, 0x41, c.v.shape)
    c.k[..., 0] = 0x38
    for i in range(pages):
        p = c.table[0, i]
        c.ks[p] = float(np.float32((2.0 * (i if up else pages - 1 - i)) * math.log(2.0) * dim ** 0.5 + 2.0 ** -20))
        c.vs[p] = 2.0 ** ((-2 if up else 2) * i + (20 if up else -28))
    c.check("bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,group", [(64, 16, 4), (64, 64, 16), (128, 64, 1), (128, 16, 8), (128, 64, 16), (256, 32, 8)])
def test_long_and_all_alike(cuda_lib, dim, page, group):
    """A long sequence over all blocks of the launch: without a query its output is the mean of the values, and with
    scores within a few powers of two none of them stands out."""
    for lengths, window in (([30011], 0), ([20002], 5000), ([9001, 1, 4097, 17, 2600], 0)):
        c = Cache(4, dim, page, 1, group, lengths)
        c.v[:] = c.rng.integers(0, 0x7F, c.v.shape) | (c.rng.integers(0, 2, c.v.shape) << 7)
        c.vs[:] = 2.0 ** c.rng.integers(-9, -4, c.vs.shape)
        c.check("bf16", window=window, most=1.001)
        c.k[:] = c.rng.integers(0, 0x40, c.k.shape) | (c.rng.integers(0, 2, c.k.shape) << 7)
        c.ks[:] = 2.0 ** -2
        c.q[:] = c.rng.standard_normal(c.q.shape)
        c.check("fp16", window=window, most=60.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,group,window", [(64, 16, 2, 0), (64, 16, 4, 100), (128, 32, 3, 0), (128, 16, 16, 50), (256, 16, 2, 33)])
def test_several_tokens_all_alike(cuda_lib, dim, page, group, window):
    c = Cache(5, dim, page, 1, group, [3001, 40, 7, 500], news=[5, 9, 7, 1])
    c.v[:] = c.rng.integers(0, 0x7F, c.v.shape) | (c.rng.integers(0, 2, c.v.shape) << 7)
    c.vs[:] = 2.0 ** c.rng.integers(-20, 21, c.vs.shape)
    c.check("bf16", window=window, most=1.001)

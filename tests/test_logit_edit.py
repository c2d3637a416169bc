"""Logit edits against the oracle, whose fp32 operations are the kernel's: outputs have to be equal, bit for bit."""
import ctypes

import numpy as np
import pytest

from conftest import ROOT  # noqa: F401
from device_logits_sampling_gb300 import edit, sampler, serve, workloads
from oracle import edit as oe

FAKE = 0x1000


# ------------------------------------------------------------------ host
@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(serve.LIB_PATH):
        from device_logits_sampling_gb300 import build

        build.build_serve()
    return serve.load()


def test_refusals(lib):
    good = dict(params=FAKE, hist_offsets=FAKE, hist_ids=FAKE, hist_len=9, bias_offsets=FAKE, bias_ids=FAKE, bias=FAKE,
                bias_len=9, allowed=FAKE, allowed_stride=4, allowed_count=3, allowed_rows=None)

    def call(logits=FAKE, B=3, V=100, ld=104, dtype=1, out=2 * FAKE, out_ld=104, out_dtype=1, err=None, **kw):
        e = serve.LogitEdits(**{**good, **kw})
        return lib.arc_edit_logits(logits, B, V, ld, dtype, out, out_ld, out_dtype, ctypes.addressof(e), err, None)

    for kw, rc in [(dict(logits=None), -1), (dict(out=None), -1), (dict(hist_ids=None), -1), (dict(hist_offsets=None), -1),
                   (dict(params=None), -1), (dict(bias_ids=None), -1), (dict(bias=None), -1), (dict(bias_offsets=None), -1),
                   (dict(allowed=None, allowed_rows=FAKE), -1), (dict(dtype=3), -3), (dict(out_dtype=2), -3),
                   (dict(dtype=0, out_dtype=1), -3), (dict(B=0), -2), (dict(B=2 ** 31), -2), (dict(V=0), -2), (dict(V=2 ** 31), -2),
                   (dict(ld=99), -2), (dict(out_ld=99), -2), (dict(hist_len=-1), -2), (dict(bias_len=2 ** 31), -2),
                   (dict(allowed_stride=3), -2), (dict(allowed_count=2), -2), (dict(allowed_count=0, allowed_rows=FAKE), -2),
                   (dict(out=FAKE, out_ld=112), -6), (dict(out=FAKE, out_dtype=0), -6), (dict(logits=FAKE + 1), -4),
                   (dict(out=2 * FAKE + 2, out_dtype=0), -4), (dict(params=FAKE + 4), -4), (dict(bias=FAKE + 2), -4),
                   (dict(allowed=FAKE + 2), -4), (dict(err=FAKE + 2), -4)]:
        assert call(**kw) == rc, kw
    assert lib.arc_edit_logits(FAKE, 1, 1, 1, 1, FAKE, 1, 1, None, None, None) == -1


def test_python_refusals():
    import torch

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    z = torch.zeros(2, 40)
    ok = dict(bias_offsets=i32(0, 1, 1), bias_ids=i32(3), bias=torch.ones(1))
    m = torch.zeros(2, 2, dtype=torch.int32)
    for kw in [dict(hist_ids=i32(1)), dict(hist_offsets=i32(0, 0, 1), hist_ids=i32(1)), {**ok, "bias": None},
               {**ok, "bias": torch.ones(2)}, {**ok, "bias_offsets": i32(0, 1)}, dict(allowed=m[:, :1]), dict(allowed=m[:1]),
               dict(allowed_rows=i32(0, 1)), dict(allowed=m, allowed_rows=i32(0)), dict(allowed=m, out=z[:, :39]),
               dict(hist_offsets=i32(0, 0, 1), hist_ids=i32(1), params=torch.zeros(95, dtype=torch.uint8)),
               dict(allowed=m)]:  # the last: host tensors
        with pytest.raises(ValueError):
            edit.edit_logits(z, **kw)
    for kw in [{**ok, "bias": torch.ones(1, dtype=torch.float16)}, {**ok, "bias_ids": torch.tensor([3])},
               dict(allowed=m.long()), dict(allowed=m, allowed_rows=torch.tensor([0, 1]))]:
        with pytest.raises(TypeError):
            edit.edit_logits(z, **kw)
    with pytest.raises(TypeError):
        edit.edit_logits(z.double(), allowed=m)


def test_pack_mask():
    a = np.random.default_rng(0).random((3, 70)) < 0.5
    w = edit.pack_mask(a)
    assert w.shape == (3, 3) and w.dtype == np.int32
    i = np.arange(70)
    assert (((w[:, i // 32].astype(np.int64) >> (i % 32)) & 1) == a).all()


def test_the_oracle_by_hand():
    z, err = oe.edit([[2.0, -1.0, 0.5, 3.0]], [[2.0, 0.5, 0.25]], [0, 3], [0, 1, 1], [0, 2], [0, 0], [5.0, 1.0],
                     [[True, True, True, False]])
    assert z.tolist() == [[1.0 - 0.75 + 1.0, -2.0 - 1.25, 0.5, -np.inf]] and err == 0


# ------------------------------------------------------------------ GPU
def records(penalties):
    rows = workloads.make_params(len(penalties))
    for i, name in enumerate(("repetition", "frequency", "presence")):
        rows[name + "_penalty"] = [p[i] for p in penalties]
    return sampler.params_tensor(rows)


class Case:
    """Inputs of a call, on the host and on the GPU."""

    def __init__(self, B, V, kind="bfloat16", hist=0, bias=0, mask=None, pad=0, seed=0, shift=0):
        import torch

        rng = np.random.default_rng(seed)
        ld = V + pad
        self.flat = torch.from_numpy(rng.normal(0, 3, B * ld + shift).astype(np.float32)).to(getattr(torch, kind)).cuda()
        self.logits = self.flat[shift:].view(B, ld)[:, :V]
        self.kw, self.host = {}, {}
        if hist:
            n = [int(v) for v in rng.integers(0, hist + 1, B)]
            off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
            ids = (V * rng.random(off[-1]) ** 3).astype(np.int32)
            pen = [(float(np.float32(rng.uniform(0.8, 1.5))), float(np.float32(rng.uniform(-0.5, 0.5))),
                    float(np.float32(rng.uniform(-0.5, 0.5)))) for _ in range(B)]
            self.host.update(penalties=pen, hist_offsets=off, hist_ids=ids)
            self.kw.update(params=records(pen))
        if bias:
            n = [int(v) for v in rng.integers(0, bias + 1, B)]
            off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
            self.host.update(bias_offsets=off, bias_ids=rng.integers(0, min(V, 2 * bias), off[-1]).astype(np.int32),
                             bias=rng.normal(0, 4, off[-1]).astype(np.float32))
        for k in ("hist_offsets", "hist_ids", "bias_offsets", "bias_ids", "bias"):
            if k in self.host:
                self.kw[k] = torch.from_numpy(self.host[k]).cuda()
        if mask is not None:
            share = {"few": 0.02, "half": 0.5, "most": 0.98, "none": 0.0, "all": 1.0}[mask]
            on = rng.random((B, V)) < share
            self.host["allowed"] = on
            words = edit.pack_mask(on)
            words[:, -1] |= np.int32(-1) << np.int32((V - 1) % 32) << 1 if V % 32 else 0  # bits from V on mean nothing
            self.kw["allowed"] = torch.from_numpy(words).cuda()

    def want(self):
        return oe.edit(self.logits.float().cpu().numpy(), **self.host)

    def check(self, got, dtype=None, err=0):
        import torch

        z, e = self.want()
        z = torch.from_numpy(z).to(dtype or self.logits.dtype)
        assert torch.equal(got.cpu().view(torch.int16 if z.element_size() == 2 else torch.int32),
                           z.view(torch.int16 if z.element_size() == 2 else torch.int32))
        assert e == err


@pytest.mark.gpu
@pytest.mark.parametrize("V", (1, 7, 8, 31, 33, 1000, 8191, 8192, 8193, 16391, 100003))
@pytest.mark.parametrize("kind", ("bfloat16", "float16", "float32"))
def test_sizes(cuda_lib, V, kind):
    """Odd vocabularies put every row on another boundary."""
    import torch

    c = Case(3, V, kind, hist=50, bias=20, mask="half", seed=V)
    c.check(edit.edit_logits(c.logits, **c.kw))
    c.check(edit.edit_logits(c.logits, out_dtype=torch.float32, **c.kw), torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("hist,bias,mask", [(300, 0, None), (0, 300, None), (0, 0, "few"), (300, 40, None), (300, 0, "most"),
                                            (0, 40, "half"), (9000, 600, "most"), (5, 5, "none"), (5, 5, "all")])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 0), (8, 3)])
def test_forms(cuda_lib, hist, bias, mask, pad, shift):
    """Each edit alone and with the others; strided rows, an odd first address; in place; into a strided output of
    another alignment."""
    import torch

    c = Case(5, 20011, "float16", hist, bias, mask, pad, shift=shift)
    c.check(edit.edit_logits(c.logits, **c.kw))
    out = torch.full((5, 20100), 9.0, dtype=torch.float16, device="cuda")
    edit.edit_logits(c.logits, out=out[:, 21:20032], **c.kw)
    c.check(out[:, 21:20032].contiguous())
    assert (out[:, :21] == 9).all() and (out[:, 20032:] == 9).all()
    before, want = c.flat.clone(), c.want()[0]
    edit.edit_logits(c.logits, out=c.logits, **c.kw)
    assert torch.equal(c.logits.cpu().view(torch.int16), torch.from_numpy(want).half().view(torch.int16))
    keep = torch.ones_like(before, dtype=torch.bool)
    keep[shift:].view(5, -1)[:, :20011] = False
    assert torch.equal(c.flat[keep], before[keep])  # nothing beside the rows


@pytest.mark.gpu
def test_allowed_rows(cuda_lib):
    """A mask for several rows, none for others, one that does not exist."""
    import torch

    c = Case(6, 3001, "bfloat16", mask="half")
    rows = [2, -1, 2, 0, 6, -7]
    c.host["allowed_rows"] = rows
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = edit.edit_logits(c.logits, **c.kw, allowed_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"), err_word=err)
    c.check(got, err=edit.ARC_EDIT_ERR_MASK)
    assert int(err) == edit.ARC_EDIT_ERR_MASK and torch.isinf(got[4]).all()
    wide = torch.full((9, 200), -1, dtype=torch.int32, device="cuda")  # masks of a padded pool
    wide[:6, :94] = c.kw["allowed"]
    c.host["allowed_rows"] = rows = [0, 1, 2, 3, 4, 5]
    c.check(edit.edit_logits(c.logits, allowed=wide, allowed_rows=torch.tensor(rows, dtype=torch.int32, device="cuda")))


@pytest.mark.gpu
def test_wrong_ids_offsets_and_penalties(cuda_lib):
    import torch

    c = Case(8, 500, "float32", hist=30, bias=30, seed=3)
    h = c.host
    h["hist_ids"][[0, 1, 5]] = [-1, 500, 2 ** 31 - 1]
    h["bias_ids"][[0, 1, 5]] = [500, -2 ** 31, 501]
    for name, bits in (("hist", edit.ARC_EDIT_ERR_HIST), ("bias", edit.ARC_EDIT_ERR_BIAS)):
        off = h[name + "_offsets"].copy()
        off[3], off[6] = off[4] + 1, 2 ** 31 - 1  # descends; past the list
        h[name + "_offsets"] = off
    h["penalties"][0] = (0.0, 0.1, 0.1)
    h["penalties"][1] = (float("nan"), 0.1, 0.1)
    h["penalties"][7] = (1.0, float("inf"), 0.1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {k: torch.from_numpy(h[k]).cuda() for k in ("hist_offsets", "hist_ids", "bias_offsets", "bias_ids", "bias")}
    got = edit.edit_logits(c.logits, **kw, params=records(h["penalties"]), err_word=err)
    c.check(got, err=7)
    assert int(err) == 7


@pytest.mark.gpu
def test_special_values(cuda_lib):
    """NaN and infinite logits and biases; a NaN that the mask takes out is gone."""
    import torch

    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[nan, nan, inf, -inf, -inf, -0.0, 3e38, 1.0]], device="cuda")
    h = dict(penalties=[(1.5, 0.5, 0.25)], hist_offsets=[0, 4], hist_ids=[1, 2, 3, 5], bias_offsets=[0, 4], bias_ids=[4, 5, 6, 7],
             bias=[inf, -inf, 3e38, nan], allowed=np.array([[0, 1, 1, 1, 1, 1, 1, 1]], dtype=bool))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = edit.edit_logits(z, params=records(h["penalties"]), hist_offsets=i32(h["hist_offsets"]), hist_ids=i32(h["hist_ids"]),
                           bias_offsets=i32(h["bias_offsets"]), bias_ids=i32(h["bias_ids"]),
                           bias=torch.tensor(h["bias"], device="cuda"), allowed=torch.from_numpy(edit.pack_mask(h["allowed"])).cuda())
    want = oe.edit(z.cpu().numpy(), **h)[0]
    assert np.array_equal(got.cpu().numpy(), want, equal_nan=True) and got[0, 0] == -inf


@pytest.mark.gpu
def test_empty_lists(cuda_lib):
    import torch

    c = Case(2, 300)
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = edit.edit_logits(c.logits, params=records([(1.5, 1, 1)] * 2), hist_offsets=z, hist_ids=none, bias_offsets=z,
                           bias_ids=none, bias=none.float())
    assert torch.equal(got, c.logits)


@pytest.mark.gpu
def test_many_rows(cuda_lib):
    """More rows than a grid's second dimension has."""
    import torch

    B = 65535 + 70
    z = torch.randn(B, 40, device="cuda")
    on = torch.rand(3, 40, device="cuda") < 0.5
    rows = torch.arange(B, device="cuda", dtype=torch.int32) % 4 - 1
    mask = torch.from_numpy(edit.pack_mask(on.cpu().numpy())).cuda()
    got = edit.edit_logits(z, allowed=mask, allowed_rows=rows)
    keep = (rows < 0)[:, None] | on[rows.clamp(min=0).long()]
    assert torch.equal(got, torch.where(keep, z, torch.full((), -float("inf"), device="cuda")))


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_lib):
    import torch

    stride = (1 << 30) + 5
    big = torch.empty(2 * stride + 100, dtype=torch.bfloat16, device="cuda")
    z = big.as_strided((3, 100), (stride, 1))
    c = Case(3, 100, hist=20, bias=5, mask="half")
    z.copy_(c.logits)
    c.check(edit.edit_logits(z, **c.kw))
    edit.edit_logits(z, out=z, **c.kw)
    c.check(z.contiguous())


@pytest.mark.gpu
def test_edited_logits_are_sampled_as_edited(cuda_lib):
    """Edits, then the sampler, replayed as one graph: penalties edited in give the tokens that the sampler's own
    give, greedy tokens obey the mask, and a row without an allowed id is degenerate."""
    import torch

    B, V = 16, 5000
    c = Case(B, V, "float32", hist=400, seed=5)
    pen = [(p[0], p[1], p[2]) for p in c.host["penalties"]]
    rows = workloads.make_params(B)
    for i, name in enumerate(("repetition", "frequency", "presence")):
        rows[name + "_penalty"] = [p[i] for p in pen]
    rows["temperature"], rows["seed"] = [0.0, 0.8] * (B // 2), range(B)
    params = sampler.params_tensor(rows)
    a, b = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    sampler.sample_batch(c.logits, params, a, hist_offsets=c.kw["hist_offsets"], hist_ids=c.kw["hist_ids"])
    kw = {**c.kw, "params": params}
    sampler.sample_batch(edit.edit_logits(c.logits, **kw), params, b)
    assert torch.equal(a, b)
    on = np.random.default_rng(1).random((B, V)) < 0.01
    on[3] = False
    mask = torch.from_numpy(edit.pack_mask(on)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(c.logits), sampler.workspace_tensor(B, V, sampler._dtype_code(c.logits))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        edit.edit_logits(c.logits, out=out, allowed=mask, **kw)
        sampler.sample_batch(out, params, b, err_word=err, workspace=ws)
    for _ in range(3):
        c.logits.copy_(torch.randn(B, V, device="cuda"))
        graph.replay()
        t = b.cpu().numpy()
        assert int(err) == sampler.ARC_ERR_DEGENERATE and t[3] == 0
        assert all(on[r, t[r]] for r in range(B) if r != 3)
        z = oe.edit(c.logits.cpu().numpy(), **c.host, allowed=on)[0]
        assert all(t[r] == int(np.argmax(z[r])) for r in range(0, B, 2))


@pytest.mark.gpu
def test_another_stream(cuda_lib):
    import torch

    c = Case(64, 50000, hist=100, bias=10, mask="half")
    want = edit.edit_logits(c.logits, **c.kw).cpu()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = edit.edit_logits(c.logits, **c.kw, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,V", [(1, 5001), (3, 40000)])
def test_long_lists(cuda_lib, rows, V):
    """A history of a million ids, most of them one id, and thousands of biases that name one id over and over, beside
    short rows."""
    import torch

    rng = np.random.default_rng(8)
    c = Case(rows, V, "float32", mask="most", seed=8)
    long_hist = np.where(rng.random((1 << 20) + 77) < 0.7, 4321, rng.integers(0, V, (1 << 20) + 77)).astype(np.int32)
    long_bias = rng.integers(0, 700, 9001).astype(np.int32)
    hist = [long_hist] + [rng.integers(0, V, 50).astype(np.int32) for _ in range(rows - 1)]
    bias = [rng.integers(0, V, 3).astype(np.int32) for _ in range(rows - 1)] + [long_bias]
    for name, lists in (("hist", hist), ("bias", bias)):
        c.host[name + "_offsets"] = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
        c.host[name + "_ids"] = np.concatenate(lists)
    c.host["bias"] = rng.normal(0, 4, len(c.host["bias_ids"])).astype(np.float32)
    c.host["penalties"] = [(1.1, float(np.float32(1e-5)), 0.25)] * rows
    kw = {k: torch.from_numpy(c.host[k]).cuda() for k in ("hist_offsets", "hist_ids", "bias_offsets", "bias_ids", "bias")}
    kw.update(c.kw, params=records(c.host["penalties"]))
    c.check(edit.edit_logits(c.logits, **kw))
    want = c.want()[0]
    edit.edit_logits(c.logits, out=c.logits, **kw)
    assert np.array_equal(c.logits.cpu().numpy(), want)

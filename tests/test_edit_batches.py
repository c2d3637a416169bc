"""edit_logits on batches whose blocks have two groups of ids a thread (lists, and more than 2,621,440 logits), against the
oracle, bit for bit."""
import numpy as np
import pytest

from device_logits_sampling_gb300 import edit
from test_logit_edit import Case, records

SLICE = 4096  # ids of a block, and of each of its two groups half


def batch(rows, V, kind, mask, pad=0, shift=0, seed=0):
    """Ids at the ends of every slice and group, wherever a row's first boundary shifts them, beside drawn ones."""
    import torch

    c = Case(rows, V, kind, mask=mask, pad=pad, shift=shift, seed=seed)
    rng = np.random.default_rng(seed + 1)
    ends = np.unique(np.concatenate([np.arange(0, V, SLICE // 2) + d for d in range(-9, 10)] + [[V - 1]]))
    ends = ends[(ends >= 0) & (ends < V)]
    for name, most in (("hist", 600), ("bias", 200)):
        lists = [np.concatenate([rng.choice(ends, len(ends) // 3), rng.integers(0, V, rng.integers(0, most))]) if rng.random() < 0.9
                 else np.zeros(0, int) for _ in range(rows)]
        c.host[name + "_offsets"] = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
        c.host[name + "_ids"] = np.concatenate(lists).astype(np.int32)
    c.host["bias"] = rng.normal(0, 4, len(c.host["bias_ids"])).astype(np.float32)
    c.host["penalties"] = [tuple(float(np.float32(x)) for x in (rng.uniform(0.8, 1.5), rng.uniform(-0.5, 0.5), rng.uniform(-0.5, 0.5)))
                           for _ in range(rows)]
    for k in ("hist_offsets", "hist_ids", "bias_offsets", "bias_ids", "bias"):
        c.kw[k] = torch.from_numpy(c.host[k]).cuda()
    c.kw["params"] = records(c.host["penalties"])
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("rows,V,pad", [(64, 50003, 0), (30, 100003, 5), (24, 129280, 0)])
@pytest.mark.parametrize("kind", ("bfloat16", "float16", "float32"))
@pytest.mark.parametrize("mask", ("half", "most", None))
def test_batches(cuda_lib, rows, V, pad, kind, mask):
    import torch

    c = batch(rows, V, kind, mask, pad, seed=V)
    c.check(edit.edit_logits(c.logits, **c.kw))
    c.check(edit.edit_logits(c.logits, out_dtype=torch.float32, **c.kw), torch.float32)
    want = torch.from_numpy(c.want()[0]).to(c.logits.dtype)
    edit.edit_logits(c.logits, out=c.logits, **c.kw)
    bits = torch.int32 if kind == "float32" else torch.int16
    assert torch.equal(c.logits.cpu().contiguous().view(bits), want.view(bits))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,shift", [("bfloat16", 3), ("float32", 1)])
def test_another_stream_and_an_odd_address(cuda_lib, kind, shift):
    import torch

    c = batch(64, 50000, kind, "half", shift=shift)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = edit.edit_logits(c.logits, **c.kw, stream=side)
    side.synchronize()
    c.check(got)

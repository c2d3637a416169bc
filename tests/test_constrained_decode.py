"""The operators of a step together, as examples/constrained_decode.py uses them: norms joined with residual sums,
attention behind a shared instruction or within a window with first tokens, logits edited before they are sampled."""
import os
import sys

import pytest

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 4), (20, 3)])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_replayed_steps_are_the_eager_ones(cuda_lib, window, sinks, temperature):
    import constrained_decode as cd

    kw = dict(batch=6, steps=20, window=window, sinks=sinks, temperature=temperature)
    replayed, model, allowed = cd.generate(graph=True, **kw)
    eager, _, _ = cd.generate(graph=False, **kw)
    assert replayed.tolist() == eager.tolist() and int(model.err.item()) == 0
    for b in range(6):
        if b % 3:
            assert all(allowed[b % 3 - 1, t] for t in replayed[:, b])
        assert 7 not in replayed[:, b]  # its bias is -100
    assert len({tuple(replayed[:, b]) for b in range(6)}) > 1


@pytest.mark.gpu
def test_shared_and_plain_attention_give_the_same_step(cuda_lib):
    """One forward pass of a batch behind the instruction, with the prefix read once and with each sequence's own
    attention over its whole table: activations of unit size whose two computations round in bf16 after every product."""
    import constrained_decode as cd
    import torch

    _, model, _ = cd.generate(batch=5, steps=4, front=9, graph=False)
    ids = torch.arange(5, device="cuda", dtype=torch.int32)
    # (the shortest prompt has 3 tokens, and 4 steps came after it: the next one is the eighth)
    pos = torch.full((5,), 9 * cd.PAGE + 7, dtype=torch.int32, device="cuda")
    keep = [t.clone() for c in model.caches for t in (c.k, c.v, c.k_scale, c.v_scale)]
    out = []
    for shared in (True, False):
        for t, k in zip((t for c in model.caches for t in (c.k, c.v, c.k_scale, c.v_scale)), keep):
            t.copy_(k)
        out.append(model.forward(ids, pos, shared=shared).float())
    # the attentions differ by a bf16 step (2^-8) of their values here and there; two layers of projections with
    # weights that keep the size of their input add such differences up like the square root of their number
    assert (out[0] - out[1]).abs().max() <= 2.0 ** -8 * 16 and (out[0] - out[1]).norm() <= 2.0 ** -8 * 2 * out[0].norm()

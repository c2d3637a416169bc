"""The decode loop of examples/paged_decode.py: replayed and eager steps give the same
tokens, and its logits are those of an fp64 evaluation of the same model over the oracle's
cache."""
import os
import sys

import numpy as np
import pytest

from conftest import ROOT
from oracle import kv_cache as ok
from oracle import w4 as ow

sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_replayed_steps_are_eager_steps(cuda_lib, temperature):
    import paged_decode as pd

    a, m = pd.generate(batch=6, steps=24, graph=True, temperature=temperature)
    b, _ = pd.generate(batch=6, steps=24, graph=False, temperature=temperature)
    assert a.shape == (25, 6) and np.array_equal(a, b)
    assert (a >= 0).all() and (a < pd.VOCAB).all() and int(m.err.item()) == 0
    assert len(set(a.reshape(-1).tolist())) > 10


@pytest.mark.gpu
def test_logits_against_the_oracle(cuda_lib):
    """Activations are rounded to bf16 at some twenty places on the way (2^-8 each, of values of size 1) and the
    cached codes follow the rounded ones: 10% of the logits' size bounds both."""
    import paged_decode as pd
    import torch

    batch = 3
    texts = pd.prompts(batch)
    model = pd.Model(batch, 40)
    offsets = np.concatenate([[0], np.cumsum([len(t) for t in texts])])
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    flat = [t for text in texts for t in text]
    got = model.logits(model.forward(i32(flat), i32([0] * batch), row_offsets=i32(offsets))).double().cpu().numpy()

    host = lambda w: (w[0].cpu().numpy(), w[1].double().cpu().numpy())  # noqa: E731
    mul = lambda x, w: ow.matvec(x, *host(w))[0]  # noqa: E731
    norm = lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)  # noqa: E731
    x = model.embed.double().cpu().numpy()[flat]
    table = model.table.cpu().numpy()
    pages = table.size
    T = len(flat)
    where = np.concatenate([np.arange(len(t)) for t in texts])
    for layer in model.layers:
        qkv = mul(norm(x), layer["qkv"]).reshape(T, -1, pd.DIM)
        q, k, v = qkv[:, :pd.Q_HEADS], qkv[:, pd.Q_HEADS:pd.Q_HEADS + pd.KV_HEADS], qkv[:, pd.Q_HEADS + pd.KV_HEADS:]
        kc, vc = (np.zeros((pages, pd.KV_HEADS, pd.PAGE, pd.DIM), np.uint8) for _ in range(2))
        ks, vs = (np.ones((pages, pd.KV_HEADS)) for _ in range(2))
        assert ok.append(kc, vc, ks, vs, k, v, [0] * batch, table, offsets, model.turns, model.amplitude) == 0
        q = np.stack([ok.rotate(q[t], int(where[t]), model.turns, model.amplitude, "half") for t in range(T)])
        o, _ = ok.attend(kc, vc, ks, vs, q, [0] * batch, table, offsets)
        x = x + mul(o.reshape(T, -1), layer["out"])
        gate, up = np.split(mul(norm(x), layer["up"]), 2, axis=1)
        x = x + mul(gate / (1.0 + np.exp(-gate)) * up, layer["down"])
    want = mul(norm(x), model.head)
    assert np.linalg.norm(got - want) <= 0.1 * np.linalg.norm(want)

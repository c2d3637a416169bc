"""Decode steps of a batch behind one shared instruction, or of endless streams, with edited logits.

    python examples/constrained_decode.py [--batch 8] [--steps 32] [--window 0] [--sinks 4]

The small model of paged_decode.py, with its residual sums and norms joined (norm.join).  The instruction's tokens go
into the cache once; every sequence's page table begins with its pages, and attend_shared reads them once for the batch.
With a window the batch are streams that see their first tokens and their last ones alone (attend with sinks).  Each
step's logits are edited before they are sampled: penalties for the ids of the prompt, a bias, and the ids that a
"grammar" allows.  A step replays as one CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import paged_decode  # noqa: E402
from device_logits_sampling_gb300 import decode, edit, kv_cache, norm, sampler, workloads  # noqa: E402
from paged_decode import DIM, HIDDEN, KV_HEADS, PAGE, Q_HEADS, VOCAB, project  # noqa: E402


class Model(paged_decode.Model):
    """The model behind an instruction of `front` pages that its sequences share; each has `length` tokens of its own."""

    def __init__(self, batch: int, length: int, front: int, window: int = 0, sinks: int = 0, seed: int = 0):
        super().__init__(batch, length, seed)
        g = torch.Generator().manual_seed(seed + 1)
        own = self.table.shape[1]
        pages = front + batch * own
        self.caches = [kv_cache.PagedCache.empty(pages, KV_HEADS, PAGE, DIM) for _ in self.layers]
        ids = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.prefix = ids[:front].contiguous()
        self.table = torch.cat([self.prefix.expand(batch, -1), ids[front:].reshape(batch, own)], 1).contiguous()
        self.window, self.sinks = window, sinks
        self.gains = [[(1.0 + 0.1 * torch.randn(HIDDEN, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
                      for _ in self.layers]
        self.last_gain = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.shared_space = self.caches[0].shared_workspace(max(batch * own * PAGE, front * PAGE), Q_HEADS)

    def attend(self, cache, q, positions, table, row_offsets, shared: bool):
        kw = dict(row_offsets=row_offsets, err_word=self.err)
        if shared and not self.window:
            return kv_cache.attend_shared(cache, q, positions, table, self.prefix, workspace=self.shared_space, **kw)
        return kv_cache.attend(cache, q, positions, table, workspace=self.workspace, window=self.window, sinks=self.sinks, **kw)

    def forward(self, ids, positions, row_offsets=None, table=None, shared: bool = True):
        """Normed activations [T, HIDDEN] of the tokens ids [T]; the caches grow by them."""
        table = self.table if table is None else table
        x = self.embed[ids.long()]
        _, n = norm.join(x, weight=self.gains[0][0])
        for i, (layer, cache) in enumerate(zip(self.layers, self.caches)):
            qkv = project(n, layer["qkv"]).unflatten(1, (Q_HEADS + 2 * KV_HEADS, DIM))
            q, k, v = qkv.split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
            q = kv_cache.append(cache, k, v, positions, table, q=q, rope=self.rope, row_offsets=row_offsets, err_word=self.err)
            o = self.attend(cache, q, positions, table, row_offsets, shared)
            x, n = norm.join(x, project(o.flatten(1), layer["out"]), weight=self.gains[i][1])
            gate, up = project(n, layer["up"]).chunk(2, dim=1)
            y = project(torch.nn.functional.silu(gate) * up, layer["down"])
            following = self.gains[i + 1][0] if i + 1 < len(self.layers) else self.last_gain
            x, n = norm.join(x, y, weight=following)
        return n

    def logits(self, n):
        return project(n, self.head, out_dtype=torch.float32)


def generate(batch: int = 8, steps: int = 32, front: int = 3, window: int = 0, sinks: int = 4, graph: bool = True,
             temperature: float = 0.0, seed: int = 0):
    """Tokens [steps + 1, batch] that follow the instruction and the prompts, the model, and which ids were allowed."""
    texts = paged_decode.prompts(batch)
    model = Model(batch, max(map(len, texts)) + steps + 1, front, window, sinks, seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(seed + 2)
    # the instruction, once: a sequence of its own on the shared pages
    n = front * PAGE
    model.forward(torch.randint(0, VOCAB, (n,), generator=g).cuda(), i32([0]), i32([0, n]), table=model.prefix[None].contiguous(),
                  shared=False)
    offsets = [0]
    for t in texts:
        offsets.append(offsets[-1] + len(t))
    x = model.forward(i32([t for text in texts for t in text]), i32([n] * batch), row_offsets=i32(offsets))

    allowed = np.random.default_rng(seed).random((2, VOCAB)) < 0.3
    edits = dict(allowed=torch.from_numpy(edit.pack_mask(allowed)).cuda(), allowed_rows=i32([b % 3 - 1 for b in range(batch)]),
                 hist_offsets=i32(offsets), hist_ids=i32([t for text in texts for t in text]),
                 bias_offsets=i32(range(batch + 1)), bias_ids=i32([7] * batch),
                 bias=torch.full((batch,), -100.0, device="cuda"), err_word=model.err)
    rows = workloads.make_params(batch)
    rows["temperature"], rows["seed"] = temperature, range(batch)
    rows["repetition_penalty"], rows["presence_penalty"] = 1.1, 0.2
    params = sampler.params_tensor(rows)
    ids, out = i32([0] * batch), i32([0] * batch)
    positions = i32([n + len(t) - 1 for t in texts])  # the commit makes it the next token's
    head = torch.zeros(2, dtype=torch.int64, device="cuda")
    ring = decode.Ring(batch * (steps + 1))
    limit = model.table.shape[1] * PAGE

    def sample(x):
        logits = model.logits(x)
        edit.edit_logits(logits, out=logits, params=params, **edits)
        decode.sample_and_commit(logits, params, out, ids, positions, limit, ring, head, autoinc=True)

    sample(x[i32(offsets[1:]).long() - 1])

    def step():
        sample(model.forward(ids, positions))

    if graph and steps:
        # the first launches set kernel attributes: one eager step, then put back what it advanced
        state = (ids, positions, head, params, *(t for c in model.caches for t in (c.k, c.v, c.k_scale, c.v_scale)))
        kept = [t.clone() for t in state]
        step()
        for t, k in zip(state, kept):
            t.copy_(k)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        run = captured.replay
    else:
        run = step
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        run()
    end.record()
    torch.cuda.synchronize()
    tokens = ring.drain(batch * (steps + 1))["token"].reshape(steps + 1, batch)
    ring.close()
    model.us_per_step = start.elapsed_time(end) * 1e3 / max(steps, 1)
    return tokens, model, allowed


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0, help="tokens that a stream sees besides its first ones; 0: all")
    ap.add_argument("--sinks", type=int, default=4)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--eager", action="store_true", help="launch each step instead of replaying a graph")
    a = ap.parse_args()
    tokens, model, _ = generate(a.batch, a.steps, window=a.window, sinks=a.sinks, graph=not a.eager, temperature=a.temperature)
    for b in range(min(a.batch, 4)):
        print(f"sequence {b}: {tokens[:, b].tolist()}")
    print(f"{model.us_per_step:.1f} us a step of {a.batch} sequences, error bits {int(model.err.item())}")


if __name__ == "__main__":
    main()

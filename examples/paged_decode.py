"""A decode loop on one GPU with every step on the device: 4-bit projections, keys
and values appended to a paged 8-bit cache with the rotation on the way, attention
over it, the last projection's logits sampled and committed, and the whole step
replayed as a CUDA graph.

    python examples/paged_decode.py [--batch 8] [--steps 32]

The model is small and its weights are random: what it shows is how the calls fit
together.  Prompts go in as ragged pieces (row_offsets), then each replay reads the
positions and token ids that the last one's commit left in device memory.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from device_logits_sampling_gb300 import decode, kv_cache, sampler, w4, workloads  # noqa: E402

VOCAB, HIDDEN, INNER, LAYERS, GROUP = 2048, 256, 512, 2, 64
Q_HEADS, KV_HEADS, DIM, PAGE = 8, 2, 64, 16


def weight(outs: int, ins: int, g) -> tuple:
    """A random 4-bit matrix whose products keep the size of their input."""
    q = torch.randint(0, 16, (outs, ins), generator=g, dtype=torch.uint8)
    s = (0.5 + torch.rand(outs, ins // GROUP, generator=g)) / (4.6 * ins ** 0.5)
    return w4.pack(q).cuda(), s.to(torch.bfloat16).cuda()


def norm(x):
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def project(x, w, **kw):
    """Products of any number of rows, w4.MAX_ROWS at a time (prompts)."""
    if len(x) <= w4.MAX_ROWS:
        return w4.matvec(x, *w, **kw)
    return torch.cat([w4.matvec(p, *w, **kw) for p in x.split(w4.MAX_ROWS)])


class Model:
    def __init__(self, batch: int, length: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.batch, self.length = batch, length
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g).to(torch.bfloat16).cuda()
        self.head = weight(VOCAB, HIDDEN, g)
        self.layers = [dict(qkv=weight((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN, g), out=weight(HIDDEN, Q_HEADS * DIM, g),
                            up=weight(2 * INNER, HIDDEN, g), down=weight(HIDDEN, INNER, g)) for _ in range(LAYERS)]
        pages = -(-length // PAGE)
        self.caches = [kv_cache.PagedCache.empty(batch * pages, KV_HEADS, PAGE, DIM) for _ in range(LAYERS)]
        self.table = torch.randperm(batch * pages, generator=g).to(torch.int32).reshape(batch, pages).cuda()
        self.turns, self.amplitude = kv_cache.rope_turns(DIM)
        self.rope = kv_cache.Rope(torch.from_numpy(self.turns).cuda(), layout="half", amplitude=self.amplitude)
        self.workspace = self.caches[0].attend_workspace()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward(self, ids, positions, row_offsets=None):
        """Activations [T, HIDDEN] of the tokens ids [T]; the caches grow by them."""
        x = self.embed[ids.long()]
        for layer, cache in zip(self.layers, self.caches):
            qkv = project(norm(x), layer["qkv"]).unflatten(1, (Q_HEADS + 2 * KV_HEADS, DIM))
            q, k, v = qkv.split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
            q = kv_cache.append(cache, k, v, positions, self.table, q=q, rope=self.rope, row_offsets=row_offsets,
                                err_word=self.err)
            o = kv_cache.attend(cache, q, positions, self.table, row_offsets=row_offsets, workspace=self.workspace,
                                err_word=self.err)
            x = x + project(o.flatten(1), layer["out"])
            gate, up = project(norm(x), layer["up"]).chunk(2, dim=1)
            x = x + project(torch.nn.functional.silu(gate) * up, layer["down"])
        return x

    def logits(self, x):
        return project(norm(x), self.head, out_dtype=torch.float32)


def prompts(batch: int, seed: int = 1) -> list:
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, VOCAB, (3 + 5 * b % 23,), generator=g).tolist() for b in range(batch)]


def generate(batch: int = 8, steps: int = 32, graph: bool = True, temperature: float = 0.0, seed: int = 0):
    """Tokens [steps + 1, batch] that follow the prompts, and the model.  The first comes from the
    prompts' last logits, the others from decode steps."""
    texts = prompts(batch)
    length = max(map(len, texts)) + steps + 1
    model = Model(batch, length, seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets = [0]
    for t in texts:
        offsets.append(offsets[-1] + len(t))
    x = model.forward(i32([t for text in texts for t in text]), i32([0] * batch), row_offsets=i32(offsets))

    rows = workloads.make_params(batch)
    rows["temperature"], rows["seed"] = temperature, range(batch)
    params = sampler.params_tensor(rows)
    ids, out = i32([0] * batch), i32([0] * batch)
    positions = i32([len(t) - 1 for t in texts])  # the commit makes it the next token's
    head = torch.zeros(2, dtype=torch.int64, device="cuda")
    ring = decode.Ring(batch * (steps + 1))

    def sample(x):
        decode.sample_and_commit(model.logits(x), params, out, ids, positions, length, ring, head, autoinc=True)

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
    records = ring.drain(batch * (steps + 1))
    tokens = records["token"].reshape(steps + 1, batch)
    ring.close()
    model.us_per_step = start.elapsed_time(end) * 1e3 / max(steps, 1)
    return tokens, model


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--eager", action="store_true", help="launch each step instead of replaying a graph")
    a = ap.parse_args()
    tokens, model = generate(a.batch, a.steps, not a.eager, a.temperature)
    for b in range(min(a.batch, 4)):
        print(f"sequence {b}: {tokens[:, b].tolist()}")
    print(f"{model.us_per_step:.1f} us a step of {a.batch} sequences, error bits {int(model.err.item())}")


if __name__ == "__main__":
    main()

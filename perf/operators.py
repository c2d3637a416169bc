"""What a decode step does around the sampler, as measurable cases.

Three operators on the GPU, each in its plain form (elementary torch operations)
and, where `own` is set, through this package's kernels:

* append: rotate a step's queries and keys by their positions and put the keys
  and values into a paged cache of 8-bit floats (e4m3) with one power-of-two
  scale for each page and head; a page whose scale has to grow is rewritten.
* attend: attention of the new tokens over that cache, grouped heads, causal,
  optionally within a window.
* w4: products of a few rows with a matrix of 4-bit weights and group scales.

A case is a dict of plain values; lengths and row counts follow from the case,
the seed only shuffles them and draws the values.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
SCALE_EXP = 32  # page scales lie in [2^-32, 2^32]
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's decode step: a single token enters the cache
        dict(name="append one token", op="append", batch=1, new=1, pos_lo=1000, pos_hi=1000, q_heads=32, kv_heads=8,
             dim=128, rot=128, layout="half", stretch=1.0, page=64, type="bf16"),
        # a served batch at the sampler's batch size, one token a sequence, part of each head rotated
        dict(name="append a batch", op="append", batch=256, new=1, pos_lo=5, pos_hi=4095, q_heads=32, kv_heads=8,
             dim=64, rot=32, layout="interleaved", stretch=1.0, page=16, type="fp16"),
        # prompts taken in: ragged pieces far into a long context with stretched positions
        dict(name="append prompts", op="append", batch=5, new=3277, pos_lo=3, pos_hi=400000, q_heads=32, kv_heads=8,
             dim=128, rot=128, layout="half", stretch=8.0, page=64, type="bf16"),
        # one user, a short conversation: latency
        dict(name="attend one short", op="attend", batch=1, new=1, len_lo=777, len_hi=777, q_heads=32, kv_heads=8,
             dim=128, page=64, window=0, type="bf16"),
        # one user, a book in the context: few rows, a long axis
        dict(name="attend one long", op="attend", batch=1, new=1, len_lo=200003, len_hi=200003, q_heads=32, kv_heads=8,
             dim=128, page=64, window=0, type="bf16"),
        # a served batch of very different lengths, small pages
        dict(name="attend a batch", op="attend", batch=256, new=1, len_lo=1, len_hi=4096, q_heads=64, kv_heads=8,
             dim=128, page=16, window=0, type="bf16"),
        # drafted tokens checked together, each head looking back over a window
        dict(name="attend drafts", op="attend", batch=48, new=5, len_lo=100, len_hi=8192, q_heads=32, kv_heads=8,
             dim=64, page=32, window=2048, type="fp16"),
        # a full server: long contexts, five query heads to a cached one
        dict(name="attend large", op="attend", batch=64, new=1, len_lo=4096, len_hi=32768, q_heads=40, kv_heads=8,
             dim=128, page=128, window=0, type="bf16"),
        # a projection of one token
        dict(name="w4 one row", op="w4", rows=1, outs=4096, ins=4096, group=128, zeros=False, type="bf16", out="bf16"),
        # the last projection of one token: the logits that the sampler reads
        dict(name="w4 head one row", op="w4", rows=1, outs=129280, ins=4096, group=64, zeros=False, type="bf16",
             out="fp32"),
        # a few drafted tokens through an odd-sized projection with zero points
        dict(name="w4 few rows", op="w4", rows=7, outs=11007, ins=4096, group=32, zeros=True, type="fp16", out="fp16"),
        # the last projection of the sampler's batch
        dict(name="w4 head batch", op="w4", rows=256, outs=129280, ins=4096, group=128, zeros=False, type="bf16",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "w4"])
    if op == "w4":
        while True:
            group = rng.choice([32, 64, 128])
            c = dict(op="w4", rows=_log(rng, 1, 256), outs=_log(rng, 300, 129280),
                     ins=group * _log(rng, max(1, 256 // group), 16384 // group), group=group,
                     zeros=rng.random() < 0.4, type=rng.choice(["bf16", "fp16"]), out=rng.choice(["same", "fp32"]))
            c["out"] = c["type"] if c["out"] == "same" else "fp32"
            if c["outs"] * c["ins"] <= 129280 * 4096:
                return c
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        while True:
            new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 8000)])
            hi = _log(rng, 10, 500000)
            c = dict(op="append", batch=_log(rng, 1, 512), new=new, pos_lo=rng.randint(0, hi), pos_hi=hi,
                     q_heads=kv * group, kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]),
                     layout=rng.choice(["half", "interleaved"]), stretch=rng.choice([1.0, 1.0, 4.0, 32.0]), page=page,
                     type=rng.choice(["bf16", "fp16"]))
            if sum(_news(c)) * (group + 2) * kv * dim <= 8200 * 48 * 128:
                return c
    while True:
        hi = _log(rng, 1, 250000)
        new = rng.choice([1, 1, 1, rng.randint(2, 8)])
        c = dict(op="attend", batch=_log(rng, 1, 512), new=new, len_lo=max(1, min(hi, rng.randint(1, hi))), len_hi=hi,
                 q_heads=kv * group, kv_heads=kv, dim=dim, page=page, window=rng.choice([0, 0, 0, _log(rng, 16, 8192)]),
                 type=rng.choice(["bf16", "fp16"]))
        held = c["batch"] * (hi + page) * kv * dim
        if held <= 64 * 32768 * 8 * 128 and held * group * new <= 64 * 32768 * 40 * 128:
            return c


def _spread(lo, hi, n):
    """n whole numbers of [lo, hi], spread over their logarithm by a golden-ratio sequence; the last one is hi."""
    at = [(0.5 + 0.6180339887498949 * i) % 1.0 for i in range(n - 1)] + [1.0]
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** f)) - 1 for f in at]


def _news(c):
    """New tokens of each sequence: one each, drafts of 1 .. new tokens, or pieces of new / 3 .. new tokens."""
    if c["new"] == 1:
        return [1] * c["batch"]
    if c["new"] <= 8:  # drafts: 1 .. new
        return [1 + (i * 7 + c["new"] - 1) % c["new"] for i in range(c["batch"])]
    return [max(1, v) for v in _spread(c["new"] // 3, c["new"], c["batch"])]


# ------------------------------------------------------------------ inputs
def _rope(c, device):
    """Angles per position of the rotated pairs, in radians (float64) and as 64-bit fixed-point
    fractions of a turn; positions stretched by interpolation, with the amplitude that goes with it."""
    r = c["rot"]
    inv = 10000.0 ** (-2.0 * np.arange(r // 2, dtype=np.float64) / r) / c["stretch"]
    turns = np.floor(inv / (2.0 * math.pi) * 2.0 ** 64).astype(np.uint64).astype(np.int64)
    amp = float(np.float32(1.0 + 0.1 * math.log(c["stretch"])))
    return torch.from_numpy(inv).to(device), torch.from_numpy(turns).to(device), amp


def _pages(c, lens, first, g):
    """A shuffled page table [B, most] for the pages of tokens first .. lens (others -1), and the pages in all."""
    dev = "cuda"
    lens_t = torch.tensor(lens, dtype=torch.int64)
    first_t = torch.tensor(first, dtype=torch.int64)
    a, b = first_t // c["page"], (lens_t + c["page"] - 1) // c["page"]
    most = int(b.max())
    j = torch.arange(most)[None, :]
    used = (j >= a[:, None]) & (j < b[:, None])
    n = int(used.sum())
    total = n + n // 8 + 1
    perm = torch.randperm(total, generator=g, device=dev)[:n].to(torch.int32)
    table = torch.full((c["batch"], most), -1, dtype=torch.int32, device=dev)
    table[used.to(dev)] = perm
    return table, total


def _cache(c, total, g):
    """Keys and values as a server holds them: e4m3 values near 1 times their page's power-of-two scale."""
    shape = (total, c["kv_heads"], c["page"], c["dim"])
    out = []
    for lo, hi in ((-7, -5), (-8, -4)):
        e = torch.randint(lo, hi + 1, shape[:2], generator=g, device="cuda")
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        x *= torch.exp2(-e.to(torch.float32) - (1.0 if lo == -8 else 0.0)).to(torch.bfloat16)[:, :, None, None]
        out += [x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), torch.exp2(e.to(torch.float32))]
        del x
    k, ks, v, vs = out
    return k, v, ks, vs


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[c["type"]]
    st = {"case": c}
    if c["op"] == "w4":
        n, k, grp = c["outs"], c["ins"], c["group"]
        st["x"] = torch.randn(c["rows"], k, generator=g, device="cuda").to(t)
        st["weight"] = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        st["scales"] = (torch.rand(n, k // grp, generator=g, device="cuda") * 0.01 + 0.002).to(t)
        st["zeros"] = (torch.randint(0, 16, (n, k // grp), generator=g, device="cuda", dtype=torch.uint8)
                       if c["zeros"] else None)
        return st
    order = torch.randperm(c["batch"], generator=torch.Generator().manual_seed(seed))
    news = [_news(c)[i] for i in order.tolist()]
    offsets = [0]
    for n in news:
        offsets.append(offsets[-1] + n)
    T, hq, hkv, d = offsets[-1], c["q_heads"], c["kv_heads"], c["dim"]
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    if c["op"] == "append":
        pos = [_spread(c["pos_lo"], c["pos_hi"], c["batch"])[i] for i in order.tolist()]
        lens = [p + n for p, n in zip(pos, news)]
        st["table"], total = _pages(c, lens, pos, g)  # pages before the new tokens' first are no longer held
        st["inv"], st["turns"], st["amp"] = _rope(c, "cuda")
        qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda").to(t)  # one projection's output
        st["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        st["keys"] = qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d))
        st["values"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    else:
        lens = [_spread(c["len_lo"], c["len_hi"], c["batch"])[i] for i in order.tolist()]
        lens = [max(a, n) for a, n in zip(lens, news)]
        pos = [a - n for a, n in zip(lens, news)]
        st["table"], total = _pages(c, lens, [0] * c["batch"], g)
        st["q"] = (2.0 * torch.randn(T, hq, d, generator=g, device="cuda")).to(t)
    st["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    st["k"], st["v"], st["ks"], st["vs"] = _cache(c, total, g)
    # slots past a sequence's last token hold whatever was there: NaN codes here
    ends = torch.tensor(lens if c["op"] == "attend" else pos, device="cuda")
    last = ends // c["page"]
    part = ends % c["page"] != 0
    ids = st["table"].gather(1, last.clamp(max=st["table"].shape[1] - 1)[:, None])[:, 0].long()[part]
    stale = torch.arange(c["page"], device="cuda")[None, :] >= (ends % c["page"])[part][:, None]
    for x in (st["k"], st["v"]):
        b = x.view(torch.uint8)
        b[ids] = torch.where(stale[:, None, :, None], torch.full_like(b[:1, :1, :1, :1], 0x7F), b[ids])
    return st


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, inv, amp, rot, layout):
    """Rotate the first `rot` values of each head of x [T, H, D] (float64) by the angles of pos [T]."""
    angle = pos.to(torch.float64)[:, None] * inv[None, :]
    c, s = (amp * torch.cos(angle))[:, None, :], (amp * torch.sin(angle))[:, None, :]
    y = x.clone()
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _e4m3(y):
    """Round float64 values to e4m3 (ties to even, saturating)."""
    a = y.abs().clamp(max=E4M3_MAX)
    step = torch.exp2((torch.frexp(a)[1] - 1).clamp(min=-6).to(torch.float64) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), y).to(torch.float32).to(torch.float8_e4m3fn)


def _append_half(cache, scale, x, page, slot, fresh_from):
    """Put x [T, H, D] (float64) at (page, slot) [T] of cache [P, H, ps, D] with scale [P, H]; `fresh_from` [P] is
    the first new slot of a page (page size where there is none)."""
    P, H, ps, D = cache.shape
    amax = torch.zeros(P, H, dtype=torch.float64, device=x.device)
    amax = amax.scatter_reduce(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax / E4M3_MAX)
    need = torch.where(m == 0.5, e - 1, e).clamp(-SCALE_EXP, SCALE_EXP)
    need = torch.where(amax == 0, torch.full_like(need, -SCALE_EXP), need)
    old = torch.frexp(scale)[1] - 1
    touched = (fresh_from < ps)[:, None]
    grown = torch.where(touched, torch.where((fresh_from > 0)[:, None], torch.maximum(old, need), need), old)
    older = torch.arange(ps, device=x.device)[None, :] < fresh_from[:, None]
    redo = (touched & (grown > old) & (fresh_from > 0)[:, None])[:, :, None, None] & older[:, None, :, None]
    down = torch.exp2((old - grown).to(torch.float64))[:, :, None, None]
    again = _e4m3(cache.to(torch.float32).to(torch.float64) * down)
    cache.view(torch.uint8).copy_(torch.where(redo, again.view(torch.uint8), cache.view(torch.uint8)))
    scale.copy_(torch.exp2(grown.to(torch.float32)))
    new = _e4m3(x * torch.exp2(-grown.to(torch.float64))[page][:, :, None])
    cache.view(torch.uint8)[page, :, slot] = new.view(torch.uint8)


def _append(st):
    c = st["case"]
    T = st["q"].shape[0]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(st["offsets"][1:].contiguous(), t.to(torch.int32), right=True)
    pos = st["pos"][seq].long() + t - st["offsets"][seq].long()
    page, slot = st["table"][seq, pos // c["page"]].long(), pos % c["page"]
    fresh = torch.full((st["k"].shape[0],), c["page"], dtype=torch.int64, device="cuda").scatter_reduce(0, page, slot, "amin")
    turn = lambda x: _rotate(x.to(torch.float64), pos, st["inv"], st["amp"], c["rot"], c["layout"])  # noqa: E731
    _append_half(st["k"], st["ks"], turn(st["keys"]), page, slot, fresh)
    _append_half(st["v"], st["vs"], st["values"].to(torch.float64), page, slot, fresh)
    return {"q": turn(st["q"]).to(st["q"].dtype), "k": st["k"], "v": st["v"], "k_scale": st["ks"], "v_scale": st["vs"]}


def _gather(x, scale, table):
    """[B, H, L, D] float32 values of a paged cache."""
    B, n = table.shape
    y = x.view(torch.uint8)[table].view(torch.float8_e4m3fn).to(torch.float32) * scale[table][..., None, None]
    return y.transpose(1, 2).reshape(B, x.shape[1], n * x.shape[2], x.shape[3])


def _attend(st):
    c = st["case"]
    T, hq, d = st["q"].shape
    hkv, B = c["kv_heads"], c["batch"]
    grp, n = hq // hkv, max(_news(c))
    table = st["table"].long().clamp(min=0)
    k, v = _gather(st["k"], st["ks"], table), _gather(st["v"], st["vs"], table)
    off = st["offsets"].long()
    i = torch.arange(n, device="cuda")
    tok = (off[:-1, None] + i[None, :]).clamp(max=T - 1)
    q = st["q"].to(torch.float32)[tok].reshape(B, n, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * grp, d)
    s = (q @ k.transpose(2, 3)) * d ** -0.5
    at = (st["pos"].long()[:, None] + i[None, :]).repeat_interleave(grp, 1)[:, None, :, None]
    j = torch.arange(k.shape[2], device="cuda")
    seen = j <= at
    if c["window"]:
        seen = seen & (j > at - c["window"])
    s = torch.where(seen, s, torch.full((), -math.inf, device="cuda"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    held = j[None, :] < (st["pos"].long() + off[1:] - off[:-1])[:, None]
    v = torch.where(held[:, None, :, None], v, torch.zeros((), device="cuda"))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, torch.zeros((), device="cuda"))
    o = o.reshape(B, hkv, n, grp, d).permute(0, 2, 1, 3, 4).reshape(B, n, hq, d)
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(st["offsets"][1:].contiguous(), t.to(torch.int32), right=True)
    return o[seq, t - off[seq]].to(st["q"].dtype)


def _w4(st):
    c = st["case"]
    n, k, grp = c["outs"], c["ins"], c["group"]
    w = torch.stack([st["weight"] & 15, st["weight"] >> 4], -1).reshape(n, k // grp, grp).to(torch.float32)
    w -= 8.0 if st["zeros"] is None else st["zeros"].to(torch.float32)[:, :, None]
    w *= st["scales"].to(torch.float32)[:, :, None]
    return (st["x"].to(torch.float32) @ w.reshape(n, k).T).to(TYPES[c["out"]])


def _own(st):
    """The calls of a program that keeps its cache, rotation and workspace."""
    c = st["case"]
    if c["op"] == "w4":
        from device_logits_sampling_gb300 import w4

        return w4.matvec(st["x"], st["weight"], st["scales"], zeros=st["zeros"], out_dtype=TYPES[c["out"]])
    from device_logits_sampling_gb300 import kv_cache

    if "cache" not in st:
        st["cache"] = kv_cache.PagedCache(st["k"], st["v"], st["ks"], st["vs"])
        if c["op"] == "append":
            st["rope"] = kv_cache.Rope(st["turns"], layout=c["layout"], amplitude=st["amp"])
        else:
            st["workspace"] = st["cache"].attend_workspace()
    offsets = None if c["new"] == 1 else st["offsets"]
    if c["op"] == "append":
        q = kv_cache.append(st["cache"], st["keys"], st["values"], st["pos"], st["table"], q=st["q"], rope=st["rope"],
                            row_offsets=offsets)
        return {"q": q, "k": st["k"], "v": st["v"], "k_scale": st["ks"], "v_scale": st["vs"]}
    return kv_cache.attend(st["cache"], st["q"], st["pos"], st["table"], row_offsets=offsets, window=c["window"],
                           workspace=st["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "w4": _w4}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "w4":
        m, n, k, grp = c["rows"], c["outs"], c["ins"], c["group"]
        out = 4 if c["out"] == "fp32" else 2
        return {"bytes": n * k // 2 + n * (k // grp) * (3 if c["zeros"] else 2) + m * k * 2 + m * n * out,
                "flops": 2 * m * n * k}
    news = _news(c)
    T, hq, hkv, d = sum(news), c["q_heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        pages = sum(-(-n // c["page"]) for n in news)
        return {"bytes": T * (2 * hq + 2 * hkv) * d * 2 + T * 2 * hkv * d + pages * (2 * hkv * 4 + 4),
                "flops": T * (hq + hkv) * c["rot"] * 3 + T * 2 * hkv * d * 2}
    lens = [max(a, n) for a, n in zip(_spread(c["len_lo"], c["len_hi"], c["batch"]), news)]
    w = c["window"] or max(lens)
    read = sum(min(a, w + n - 1) for a, n in zip(lens, news))
    seen = sum(sum(min(a - n + i + 1, w) for i in range(n)) for a, n in zip(lens, news))
    return {"bytes": read * hkv * d * 2 + sum(-(-a // c["page"]) for a in lens) * (8 * hkv + 4) + T * hq * d * 4,
            "flops": 4 * seen * hq * d}


# ------------------------------------------------------------------ 64 bits
def _exact_append(st):
    c = st["case"]
    host = lambda x: x.to(torch.float64).cpu().numpy()  # noqa: E731
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    mids = (codes[1:] + codes[:-1]) / 2

    def nearest(y):  # the codes ascend with their value, an even code is an even mantissa
        a = np.abs(y)
        i = np.searchsorted(mids, a, side="left")
        j = np.minimum(i, len(mids) - 1)
        return np.copysign(codes[np.where((a == mids[j]) & (i < len(mids)) & (i % 2 == 1), i + 1, i)], y)

    def exponent(m):
        e = -SCALE_EXP
        while e < SCALE_EXP and m > E4M3_MAX * 2.0 ** e:
            e += 1
        return e

    offs, pos, table = st["offsets"].cpu().numpy(), st["pos"].cpu().numpy(), st["table"].cpu().numpy()
    inv, r, ps = host(st["inv"]), c["rot"], c["page"]
    where = np.concatenate([p + np.arange(n, dtype=np.int64) for p, n in zip(pos, np.diff(offs))]).astype(np.float64)
    turn = np.exp(1j * (where[:, None] * inv[None, :]))[:, None, :] * st["amp"]

    def rotated(x):
        x = host(x)
        one, two = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
        z = (x[..., one] + 1j * x[..., two]) * turn
        x[..., one], x[..., two] = z.real, z.imag
        return x

    new = {"k": rotated(st["keys"]), "v": host(st["values"])}
    out = {"q": torch.from_numpy(rotated(st["q"]))}
    for name, scale in (("k", "ks"), ("v", "vs")):
        held, sc, x = host(st[name].to(torch.float32)), host(st[scale]), new[name]
        for b in range(c["batch"]):
            at, end = int(pos[b]), int(pos[b]) + int(offs[b + 1] - offs[b])
            row = int(offs[b])
            while at < end:
                p, s = int(table[b, at // ps]), at % ps
                n = min(ps - s, end - at)
                for h in range(c["kv_heads"]):
                    e = exponent(np.abs(x[row:row + n, h]).max())
                    if s:
                        was = int(math.log2(sc[p, h]))
                        e = max(e, was)
                        if e > was:
                            held[p, h, :s] = nearest(held[p, h, :s] * 2.0 ** (was - e))
                    sc[p, h] = 2.0 ** e
                    held[p, h, s:s + n] = nearest(x[row:row + n, h] * 2.0 ** -e)
                at, row = at + n, row + n
        out[name], out[name + "_scale"] = torch.from_numpy(held), torch.from_numpy(sc)
    return out


def _exact_attend(st):
    c = st["case"]
    offs, pos = st["offsets"].tolist(), st["pos"].tolist()
    hkv, d, ps = c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        n = offs[b + 1] - offs[b]
        length = pos[b] + n
        start = max(0, pos[b] + 1 - c["window"]) // ps if c["window"] else 0
        pages = st["table"][b, start: -(-length // ps)].long()
        kv = []
        for x, s in ((st["k"], st["ks"]), (st["v"], st["vs"])):
            y = x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(torch.float64) * s[pages].to(torch.float64)[..., None, None]
            kv.append(y.permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, : length - start * ps])
        for i in range(n):
            p = pos[b] + i
            lo = max(0, p + 1 - c["window"]) - start * ps if c["window"] else 0
            hi = p + 1 - start * ps
            q = st["q"][offs[b] + i].to(torch.float64).reshape(hkv, -1, d)
            w = torch.softmax(torch.einsum("hgd,hld->hgl", q, kv[0][:, lo:hi]) / math.sqrt(d), -1)
            out[offs[b] + i] = torch.einsum("hgl,hld->hgd", w, kv[1][:, lo:hi]).reshape(-1, d)
    return out


def _exact_w4(st):
    c = st["case"]
    x, parts = st["x"].to(torch.float64), []
    for a in range(0, c["outs"], 8192):
        b = st["weight"][a:a + 8192].to(torch.int16)
        q = torch.empty(b.shape[0], c["ins"], dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = b % 16, b // 16
        z = 8 if st["zeros"] is None else st["zeros"][a:a + 8192].to(torch.float64).repeat_interleave(c["group"], 1)
        parts.append(x @ ((q - z) * st["scales"][a:a + 8192].to(torch.float64).repeat_interleave(c["group"], 1)).T)
    return torch.cat(parts, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        # the page loop runs on the host: about 20 seconds at twice this
        return _exact_append(st) if sum(_news(case)) * case["kv_heads"] * case["dim"] <= 1 << 24 else None
    return _exact_attend(st) if case["op"] == "attend" else _exact_w4(st)

"""More of what a decode step does around the sampler, as measurable cases.

Four operators on the GPU, each in its plain form (elementary torch operations)
and, where `own` is set, through this package's kernels:

* edit: logits before the sampler: penalties for ids of each row's history, a few
  biases, and a bit mask of the ids that a grammar allows.
* sinks: attention of new tokens over the paged 8-bit cache within a window, with a
  sequence's first tokens always visible.
* shared: the same attention, causal, of a batch whose sequences begin with the
  same long prefix.
* norm: the join around a block: norm after it, gate, scaled residual sum, norm
  before the next one.

A case is a dict of plain values; lengths and row counts follow from the case,
the seed only shuffles them and draws the values.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's constrained decode step inside a free text: most ids allowed, a page of text behind it
        dict(name="edit one row", op="edit", rows=1, vocab=129280, hist=2000, bias=30, mask="most", place="new",
             type="bf16", out="bf16"),
        # the sampler's batch: histories and biases of very different lengths, a grammar on three rows in four
        dict(name="edit a batch", op="edit", rows=256, vocab=129280, hist=4096, bias=300, mask="mixed", place="new",
             type="bf16", out="bf16"),
        # a grammar alone, written into the logits where they are; an odd vocabulary
        dict(name="mask in place", op="edit", rows=100, vocab=100003, hist=0, bias=0, mask="mixed", place="same",
             type="fp32", out="fp32"),
        # one user far into an endless stream: latency
        dict(name="sinks one", op="sinks", batch=1, new=1, len_lo=300001, len_hi=300001, q_heads=32, kv_heads=8, dim=128,
             page=64, window=4096, sinks=4, type="bf16"),
        # a served batch of streams, some shorter than their window, small pages
        dict(name="sinks a batch", op="sinks", batch=256, new=1, len_lo=5, len_hi=50000, q_heads=32, kv_heads=8, dim=128,
             page=16, window=4096, sinks=64, type="bf16"),
        # drafted tokens of streams, heads of 64
        dict(name="sinks drafts", op="sinks", batch=48, new=5, len_lo=1000, len_hi=100000, q_heads=32, kv_heads=8, dim=64,
             page=32, window=8000, sinks=130, type="fp16"),
        # a few users behind a short instruction: latency
        dict(name="shared few", op="shared", batch=4, new=1, prefix=1024, own_lo=1, own_hi=300, q_heads=32, kv_heads=8,
             dim=128, page=64, type="bf16"),
        # a served batch behind a long document
        dict(name="shared batch", op="shared", batch=64, new=1, prefix=32768, own_lo=1, own_hi=2048, q_heads=32,
             kv_heads=8, dim=128, page=64, type="bf16"),
        # drafted tokens behind instructions of an odd number of small pages, heads of 64
        dict(name="shared drafts", op="shared", batch=32, new=4, prefix=8208, own_lo=4, own_hi=700, q_heads=32,
             kv_heads=8, dim=64, page=16, type="fp16"),
        # a full server, every request behind the same instructions and examples
        dict(name="shared large", op="shared", batch=256, new=1, prefix=16384, own_lo=1, own_hi=1024, q_heads=64,
             kv_heads=8, dim=128, page=32, type="bf16"),
        # one token's residual sum and the next norm: latency
        dict(name="norm one token", op="norm", rows=1, dim=4096, stream="bf16", type="bf16", post=False, gate="none",
             alpha=1.0, offset=0.0),
        # prompts: 32-bit residual stream, a norm on both sides, a learned gate for each token
        dict(name="norm prompts", op="norm", rows=8191, dim=5120, stream="fp32", type="bf16", post=True, gate="sigmoid",
             alpha=0.22, offset=1.0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["edit", "sinks", "shared", "norm"])
    half = rng.choice(["bf16", "fp16"])
    if op == "norm":
        while True:
            c = dict(op="norm", rows=_log(rng, 1, 16384), dim=_log(rng, 64, 16384), stream=rng.choice([half, "fp32"]),
                     type=half, post=rng.random() < 0.5, gate=rng.choice(["none", "none", "channel", "token", "sigmoid"]),
                     alpha=rng.choice([1.0, round(rng.uniform(0.05, 2.0), 3)]), offset=rng.choice([0.0, 1.0]))
            if rng.random() < 0.8:
                c["dim"] = max(64, c["dim"] // 64 * 64)
            if c["rows"] * c["dim"] <= 8191 * 5120:
                return c
    if op == "edit":
        while True:
            place = rng.choice(["new", "new", "same"])
            t = rng.choice(["bf16", "fp16", "fp32"])
            c = dict(op="edit", rows=_log(rng, 1, 512), vocab=_log(rng, 1000, 200000),
                     hist=rng.choice([0, _log(rng, 1, 8000)]), bias=rng.choice([0, _log(rng, 1, 300)]),
                     mask=rng.choice(["none", "few", "most", "mixed"]), place=place, type=t, out=rng.choice([t, "fp32"]))
            if place == "same":  # the mask alone gives the same result however often it is applied
                c.update(hist=0, bias=0, out=t, mask=rng.choice(["few", "most", "mixed"]))
            if c["hist"] == 0 and c["bias"] == 0 and c["mask"] == "none":
                c["mask"] = "mixed"
            if c["rows"] * c["vocab"] * (2 if c["out"] == "fp32" else 1) <= 256 * 129280:
                return c
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    new = rng.choice([1, 1, 1, rng.randint(2, 8)])
    head = dict(q_heads=kv * group, kv_heads=kv, dim=dim, page=page, type=half)
    if op == "sinks":
        while True:
            hi = _log(rng, 10, 200000)
            c = dict(op="sinks", batch=_log(rng, 1, 256), new=new, len_lo=max(1, min(hi, rng.randint(1, hi))), len_hi=hi,
                     **head, window=_log(rng, 16, 8192), sinks=_log(rng, 1, 300))
            # (the pages between the sinks and the window are no longer held)
            if work(c)["bytes"] <= 850e6 and work(c)["flops"] <= 13.5e9:
                return c
    while True:
        own_hi = _log(rng, 8, 2048)
        c = dict(op="shared", batch=_log(rng, 1, 256), new=new, prefix=page * _log(rng, 1, max(1, 65536 // page)),
                 own_lo=rng.randint(1, own_hi), own_hi=own_hi, **head)
        if work(c)["bytes"] <= 850e6 and work(c)["flops"] <= 138e9:
            return c


def _spread(lo, hi, n):
    """n whole numbers of [lo, hi], spread over their logarithm by a golden-ratio sequence; the last one is hi."""
    at = [(0.5 + 0.6180339887498949 * i) % 1.0 for i in range(n - 1)] + [1.0]
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** f)) - 1 for f in at]


def _news(c):
    """New tokens of each sequence: one each, or drafts of 1 .. new tokens."""
    return [1 + (i * 7 + c["new"] - 1) % c["new"] for i in range(c["batch"])]


def _counts(most, rows):
    """Entries of each row's list: none for some, up to `most`."""
    return [0] * rows if most == 0 else _spread(0 if rows > 1 else most, most, rows)


# ------------------------------------------------------------------ inputs
def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _mask_of(c, g):
    """Allowed ids as bits, [rows, ceil(vocab / 32)] int32, and the mask's row of each logits row (-1: no mask)."""
    n, v = c["rows"], c["vocab"]
    kinds = {"few": ["few"], "most": ["most"], "mixed": ["few", "most", "none", "half"]}[c["mask"]]
    share = {"few": 40.0 / v, "most": 0.97, "half": 0.5, "none": 1.0}
    p = torch.tensor([share[kinds[i % len(kinds)]] for i in range(n)], device="cuda")
    words = -(-v // 32)
    bits = torch.rand(n, words * 32, generator=g, device="cuda") < p[:, None]
    bits = bits.view(n, words, 32).to(torch.int64) << torch.arange(32, device="cuda")
    packed = bits.sum(-1)
    packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
    rows = torch.tensor([-1 if kinds[i % len(kinds)] == "none" else i for i in range(n)], dtype=torch.int32, device="cuda")
    return packed, rows


def _prepare_edit(c, g, seed):
    n, v = c["rows"], c["vocab"]
    st = {"case": c}
    st["logits"] = (3.0 * torch.randn(n, v, generator=g, device="cuda")).to(TYPES[c["type"]])
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()
    rng = np.random.default_rng(seed)
    hist = [_counts(c["hist"], n)[i] for i in order]
    bias = [min(v, _counts(c["bias"], n)[i]) for i in order]
    # text repeats itself: ids follow a power law over a shuffled vocabulary
    ids = (v * rng.random(sum(hist)) ** 4).astype(np.int64) * 7919 % v
    st["hist_offsets"] = torch.tensor(_offsets(hist), dtype=torch.int32, device="cuda")
    st["hist_ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    bids = np.concatenate([rng.choice(v, k, replace=False) for k in bias]) if sum(bias) else np.zeros(0, np.int64)
    st["bias_offsets"] = torch.tensor(_offsets(bias), dtype=torch.int32, device="cuda")
    st["bias_ids"] = torch.from_numpy(bids.astype(np.int32)).cuda()
    st["bias"] = torch.from_numpy(rng.uniform(-8.0, 8.0, sum(bias)).astype(np.float32)).cuda()
    penalties = np.stack([rng.uniform(1.0, 1.3, n), rng.uniform(0.0, 0.5, n), rng.uniform(0.0, 0.5, n)], 1).astype(np.float32)
    st["penalties_host"], st["penalties"] = penalties, torch.from_numpy(penalties).cuda()
    st["allowed"], st["allowed_rows"] = (None, None) if c["mask"] == "none" else _mask_of(c, g)
    return st


def _prepare_norm(c, g):
    n, d, t = c["rows"], c["dim"], TYPES[c["type"]]
    make = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    st = {"case": c, "x": (4.0 * make(n, d)).to(TYPES[c["stream"]]), "y": make(n, d).to(t)}
    st["weight"] = (1.0 - c["offset"] + 0.2 * make(d)).to(t)
    st["post"] = (1.0 - c["offset"] + 0.2 * make(d)).to(t) if c["post"] else None
    st["gate"] = None if c["gate"] == "none" else (make(d) if c["gate"] == "channel" else make(n, d)).to(t)
    return st


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


def _lengths(c):
    """Tokens that each sequence holds with the new ones, in the order of the case."""
    news = _news(c)
    if c["op"] == "sinks":
        return [max(a, n) for a, n in zip(_spread(c["len_lo"], c["len_hi"], c["batch"]), news)]
    return [c["prefix"] + max(a, n) for a, n in zip(_spread(c["own_lo"], c["own_hi"], c["batch"]), news)]


def _prepare_attend(c, g, seed):
    ps, B = c["page"], c["batch"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    news = [_news(c)[i] for i in order]
    lens = [_lengths(c)[i] for i in order]
    pos = [a - n for a, n in zip(lens, news)]
    st = {"case": c, "offsets": torch.tensor(_offsets(news), dtype=torch.int32, device="cuda"),
          "pos": torch.tensor(pos, dtype=torch.int32, device="cuda")}
    # pages held: those of the sinks and of the window, or those behind the prefix; the others are -1
    last = (torch.tensor(lens) + ps - 1) // ps
    most = int(last.max())
    j = torch.arange(most)[None, :]
    if c["op"] == "sinks":
        first = (torch.tensor(pos) + 1 - c["window"]).clamp(min=0) // ps
        held = (j < last[:, None]) & ((j >= first[:, None]) | (j < -(-c["sinks"] // ps)))
        front = 0
    else:
        front = c["prefix"] // ps
        held = (j < last[:, None]) & (j >= front)
    n = int(held.sum()) + front
    total = n + n // 8 + 1
    perm = torch.randperm(total, generator=g, device="cuda")[:n].to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    table[held.cuda()] = perm[front:]
    if front:
        st["prefix"] = perm[:front].contiguous()
        table[:, :front] = st["prefix"]
    st["table"] = table
    st["q"] = (2.0 * torch.randn(sum(news), c["q_heads"], c["dim"], generator=g, device="cuda")).to(TYPES[c["type"]])
    st["k"], st["v"], st["ks"], st["vs"] = _cache(c, total, g)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "edit":
        return _prepare_edit(case, g, seed)
    return _prepare_norm(case, g) if case["op"] == "norm" else _prepare_attend(case, g, seed)


# ------------------------------------------------------------------ plain forms
def _edit(st):
    c = st["case"]
    n, v = c["rows"], c["vocab"]
    z = st["logits"].to(torch.float32)
    rows = torch.arange(n, device="cuda")
    if c["hist"]:
        at = torch.repeat_interleave(rows, (st["hist_offsets"][1:] - st["hist_offsets"][:-1]).long(), output_size=len(st["hist_ids"]))
        count = torch.zeros(n, v, device="cuda").index_put_((at, st["hist_ids"].long()),
                                                            torch.ones((), device="cuda"), accumulate=True)
        rep, freq, pres = (st["penalties"][:, i:i + 1] for i in range(3))
        hit = torch.where(z > 0, z / rep, z * rep) - count * freq - pres
        z = torch.where(count > 0, hit, z)
    if c["bias"]:
        at = torch.repeat_interleave(rows, (st["bias_offsets"][1:] - st["bias_offsets"][:-1]).long(), output_size=len(st["bias_ids"]))
        z = z + torch.zeros(n, v, device="cuda").index_put_((at, st["bias_ids"].long()), st["bias"])
    if st["allowed"] is not None:
        ids = torch.arange(v, device="cuda")
        on = (st["allowed"][:, ids // 32] >> (ids % 32).to(torch.int32)) & 1
        z = torch.where((on == 1) | (st["allowed_rows"] < 0)[:, None], z, torch.full((), -math.inf, device="cuda"))
    if c["place"] == "same":
        return st["logits"].copy_(z)
    return z.to(TYPES[c["out"]])


def _rms(x, weight, offset):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (offset + weight.to(torch.float32))


def _norm(st):
    c = st["case"]
    u = st["y"].to(torch.float32)
    if st["post"] is not None:
        u = _rms(u, st["post"], c["offset"])
    if st["gate"] is not None:
        gate = st["gate"].to(torch.float32)
        u = u * (1.0 / (1.0 + torch.exp(-gate)) if c["gate"] == "sigmoid" else gate)
    h = st["x"].to(torch.float32) + c["alpha"] * u
    return {"h": h.to(TYPES[c["stream"]]), "n": _rms(h, st["weight"], c["offset"]).to(TYPES[c["type"]])}


def _gather(x, scale, table):
    """[B, H, L, D] float32 values of a paged cache."""
    B, n = table.shape
    y = x.view(torch.uint8)[table].view(torch.float8_e4m3fn).to(torch.float32) * scale[table][..., None, None]
    return y.transpose(1, 2).reshape(B, x.shape[1], n * x.shape[2], x.shape[3])


def _padded(st):
    """Queries as [B, H, tokens * group, D] float32, and each row's position [B, 1, tokens * group, 1]."""
    c = st["case"]
    T, hq, d = st["q"].shape
    hkv, B, n = c["kv_heads"], c["batch"], c["new"]
    off = st["offsets"].long()
    i = torch.arange(n, device="cuda")
    tok = (off[:-1, None] + i[None, :]).clamp(max=T - 1)
    q = st["q"].to(torch.float32)[tok].reshape(B, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)
    at = (st["pos"].long()[:, None] + i[None, :]).repeat_interleave(hq // hkv, 1)[:, None, :, None]
    return q, at


def _flat(st, o):
    """[T, q_heads, D] of the query's type, from the padded rows."""
    c = st["case"]
    T, hq, d = st["q"].shape
    off = st["offsets"].long()
    o = o.reshape(c["batch"], c["kv_heads"], c["new"], -1, d).permute(0, 2, 1, 3, 4).reshape(c["batch"], c["new"], hq, d)
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(st["offsets"][1:].contiguous(), t.to(torch.int32), right=True)
    return o[seq, t - off[seq]].to(st["q"].dtype)


def _sinks(st):
    c = st["case"]
    off = st["offsets"].long()
    end = st["pos"].long() + off[1:] - off[:-1]
    # the tokens that a sequence holds: its sinks, then its window from the first page that a row sees
    ps = c["page"]
    front = -(-c["sinks"] // ps)
    first = (st["pos"].long() + 1 - c["window"]).clamp(min=0) // ps
    width = (c["window"] + c["new"]) // ps + 2
    j = torch.arange(width, device="cuda")
    pages = torch.cat([torch.arange(front, device="cuda").expand(c["batch"], -1), first[:, None] + j[None, :]], 1)
    again = torch.arange(front + width, device="cuda")[None, :] >= front
    twice = again & (pages < front)
    table = st["table"].long().gather(1, pages.clamp(max=st["table"].shape[1] - 1)).clamp(min=0)
    k, v = _gather(st["k"], st["ks"], table), _gather(st["v"], st["vs"], table)
    token = (pages[:, :, None] * ps + torch.arange(ps, device="cuda")).reshape(c["batch"], 1, 1, -1)
    q, at = _padded(st)
    seen = (token <= at) & ((token > at - c["window"]) | (token < c["sinks"]))
    seen = seen & ~twice.repeat_interleave(ps, 1)[:, None, None, :] & (token < end[:, None, None, None])
    s = torch.where(seen, (q @ k.transpose(2, 3)) * c["dim"] ** -0.5, torch.full((), -math.inf, device="cuda"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return _flat(st, torch.where(total > 0, (p @ v) / total, torch.zeros((), device="cuda")))


def _shared(st):
    c = st["case"]
    front = c["prefix"] // c["page"]
    q, at = _padded(st)
    B, H, R, D = q.shape
    front_pages = st["prefix"].long()[None]
    k0, v0 = _gather(st["k"], st["ks"], front_pages), _gather(st["v"], st["vs"], front_pages)
    table = st["table"].long()[:, front:].clamp(min=0)
    k1, v1 = _gather(st["k"], st["ks"], table), _gather(st["v"], st["vs"], table)
    rows = q.transpose(0, 1).reshape(H, B * R, D)
    s0 = (rows @ k0[0].transpose(1, 2)) * D ** -0.5
    s1 = (q @ k1.transpose(2, 3)) * D ** -0.5
    token = c["prefix"] + torch.arange(s1.shape[-1], device="cuda")
    s1 = torch.where(token <= at, s1, torch.full((), -math.inf, device="cuda"))
    m = torch.maximum(s0.amax(-1, keepdim=True).reshape(H, B, R, 1).transpose(0, 1), s1.amax(-1, keepdim=True))
    p0 = torch.exp(s0 - m.transpose(0, 1).reshape(H, B * R, 1))
    p1 = torch.exp(s1 - m)
    total = p0.sum(-1).reshape(H, B, R, 1).transpose(0, 1) + p1.sum(-1, keepdim=True)
    o = (p0 @ v0[0]).reshape(H, B, R, D).transpose(0, 1) + p1 @ v1
    return _flat(st, o / total)


def _own(st):
    """The calls of a program that keeps its cache, records and workspace."""
    c = st["case"]
    if c["op"] == "edit":
        from device_logits_sampling_gb300 import edit, sampler, workloads

        if "params" not in st:  # the records that the sampler reads too
            rows = workloads.make_params(c["rows"])
            for i, name in enumerate(("repetition", "frequency", "presence")):
                rows[name + "_penalty"] = st["penalties_host"][:, i]
            st["params"] = sampler.params_tensor(rows)
        kw = {}
        if c["hist"]:
            kw.update(params=st["params"], hist_offsets=st["hist_offsets"], hist_ids=st["hist_ids"])
        if c["bias"]:
            kw.update(bias_offsets=st["bias_offsets"], bias_ids=st["bias_ids"], bias=st["bias"])
        if st["allowed"] is not None:
            kw.update(allowed=st["allowed"], allowed_rows=st["allowed_rows"])
        if c["place"] == "same":
            return edit.edit_logits(st["logits"], out=st["logits"], **kw)
        return edit.edit_logits(st["logits"], out_dtype=TYPES[c["out"]], **kw)
    if c["op"] == "norm":
        from device_logits_sampling_gb300 import norm

        h, n = norm.join(st["x"], st["y"], weight=st["weight"], post_weight=st["post"], gate=st["gate"],
                         activation="sigmoid" if c["gate"] == "sigmoid" else None, alpha=c["alpha"], offset=c["offset"],
                         eps=1e-6)
        return {"h": h, "n": n}
    from device_logits_sampling_gb300 import kv_cache

    if "cache" not in st:
        st["cache"] = kv_cache.PagedCache(st["k"], st["v"], st["ks"], st["vs"])
        st["workspace"] = (st["cache"].attend_workspace() if c["op"] == "sinks"
                           else st["cache"].shared_workspace(st["q"].shape[0], c["q_heads"]))
    offsets = None if c["new"] == 1 else st["offsets"]
    if c["op"] == "sinks":
        return kv_cache.attend(st["cache"], st["q"], st["pos"], st["table"], row_offsets=offsets, window=c["window"],
                               sinks=c["sinks"], workspace=st["workspace"])
    return kv_cache.attend_shared(st["cache"], st["q"], st["pos"], st["table"], st["prefix"], row_offsets=offsets,
                                  workspace=st["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"edit": _edit, "sinks": _sinks, "shared": _shared, "norm": _norm}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def _visible(c, length, new):
    """(tokens that any new token of a sequence sees, pairs of new token and seen token)."""
    w, s = c["window"], c["sinks"]
    first = max(0, length - new + 1 - w)  # of the first new token's window
    union = length - first + min(s, first)
    pairs = 0
    for p in range(length - new, length):
        lo = max(0, p + 1 - w)
        pairs += p + 1 - lo + min(s, lo)
    return union, pairs


def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "edit":
        n, v = c["rows"], c["vocab"]
        hist, bias = sum(_counts(c["hist"], n)), sum(_counts(c["bias"], n))
        mask = 0 if c["mask"] == "none" else n * (-(-v // 32) * 4 + 4)
        return {"bytes": n * v * (size[c["type"]] + size[c["out"]]) + hist * 4 + bias * 8 + n * 16 + mask,
                "flops": 4 * hist + bias}
    if c["op"] == "norm":
        n, d = c["rows"], c["dim"]
        gate = {"none": 0, "channel": d * 2}.get(c["gate"], n * d * 2)
        return {"bytes": n * d * (2 * size[c["stream"]] + 4) + gate + d * (4 if c["post"] else 2),
                "flops": n * d * (5 + (3 if c["post"] else 0) + (0 if c["gate"] == "none" else 1))}
    news, lens = _news(c), _lengths(c)
    T, hq, hkv, d = sum(news), c["q_heads"], c["kv_heads"], c["dim"]
    if c["op"] == "sinks":
        seen = [_visible(c, a, n) for a, n in zip(lens, news)]
        read, pairs = sum(u for u, _ in seen), sum(p for _, p in seen)
    else:
        behind = [a - c["prefix"] for a in lens]
        read = c["prefix"] + sum(behind)
        pairs = T * c["prefix"] + sum(n * a - n * (n - 1) // 2 for a, n in zip(behind, news))
    return {"bytes": read * hkv * d * 2 + -(-read // c["page"]) * (8 * hkv + 4) + T * hq * d * 4, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ 64 bits
def _exact_edit(st):
    c = st["case"]
    out = torch.empty(st["logits"].shape, dtype=torch.float64, device="cuda")
    ho, bo = st["hist_offsets"].tolist(), st["bias_offsets"].tolist()
    shift = torch.arange(32, dtype=torch.int32, device="cuda")
    for r in range(c["rows"]):
        z = st["logits"][r].to(torch.float64)
        if c["hist"] and ho[r + 1] > ho[r]:
            ids, count = torch.unique(st["hist_ids"][ho[r]:ho[r + 1]].long(), return_counts=True)
            rep, freq, pres = (float(p) for p in st["penalties_host"][r])
            x = z[ids]
            z[ids] = torch.where(x > 0, x / rep, x * rep) - freq * count.to(torch.float64) - pres
        if c["bias"] and bo[r + 1] > bo[r]:
            z[st["bias_ids"][bo[r]:bo[r + 1]].long()] += st["bias"][bo[r]:bo[r + 1]].to(torch.float64)
        if st["allowed"] is not None and int(st["allowed_rows"][r]) >= 0:
            word = st["allowed"][int(st["allowed_rows"][r])]
            off = ((word[:, None] >> shift[None, :]) & 1).reshape(-1)[: c["vocab"]] == 0
            z[off] = -math.inf
        out[r] = z
    return out


def _exact_norm(st):
    c = st["case"]
    f = lambda x: x.to(torch.float64)  # noqa: E731
    scale = lambda x: (x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()  # noqa: E731
    y = f(st["y"])
    if st["post"] is not None:
        y = y / scale(y) * (f(st["post"]) + c["offset"])
    if st["gate"] is not None:
        y = y * (torch.sigmoid(f(st["gate"])) if c["gate"] == "sigmoid" else f(st["gate"]))
    h = f(st["x"]) + c["alpha"] * y
    return {"h": h, "n": h / scale(h) * (f(st["weight"]) + c["offset"])}


def _exact_attend(st):
    c = st["case"]
    offs, pos = st["offsets"].tolist(), st["pos"].tolist()
    hkv, d, ps = c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")

    def tokens(b, at):
        """Keys and values [H, n, D] of the sequence's tokens at the positions `at`."""
        page, slot = st["table"][b][at // ps].long(), at % ps
        return [(x.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).to(torch.float64)
                 * s[page].to(torch.float64)[..., None]).transpose(0, 1) for x, s in ((st["k"], st["ks"]), (st["v"], st["vs"]))]

    for b in range(c["batch"]):
        for i in range(offs[b + 1] - offs[b]):
            p = pos[b] + i
            lo = max(0, p + 1 - c["window"]) if c["op"] == "sinks" else 0
            at = torch.arange(lo, p + 1, device="cuda")
            if lo:
                at = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), at])
            k, v = tokens(b, at)
            q = st["q"][offs[b] + i].to(torch.float64).reshape(hkv, -1, d)
            w = torch.softmax(torch.einsum("hgd,hld->hgl", q, k) / math.sqrt(d), -1)
            out[offs[b] + i] = torch.einsum("hgl,hld->hgd", w, v).reshape(-1, d)
    return out


def exact(case, seed):
    # the attention in 64 bits takes about 20 seconds at twice this
    if case["op"] in ("sinks", "shared") and work(case)["flops"] > 8e9:
        return None
    st = prepare(case, seed)
    if case["op"] == "edit":
        return _exact_edit(st)
    return _exact_norm(st) if case["op"] == "norm" else _exact_attend(st)

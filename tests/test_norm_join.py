"""The join around a block against the fp64 oracle, its refusals, and its calls on other streams and in graphs.

What an output may be off by, beside half a step of its type.  A sum of squares of positive terms: 64 fused
products in a thread and 10 levels of a tree, 74 roundings of 2^-24 of the sum, 2^-17.7; its root half of that,
with 2^-22 of rsqrtf and 2^-24 for each product.  The sigmoid: exp of a fp32 argument |g| log2(e) rounded, (2 + 2 |g|)
2^-23, and two roundings.  All in all u is within E = 2^-17 + |g| 2^-22 of itself; h within E |alpha u| + 2^-23 (|x| + |alpha u|);
n within that times its factor, plus (E + the relative error that h's leave in its mean square) of itself."""
import numpy as np
import pytest

from conftest import ROOT  # noqa: F401
from device_logits_sampling_gb300 import norm, serve
from oracle import norm as on

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
    import ctypes
    import math

    good = dict(x=FAKE, y=FAKE, gate=FAKE, post_weight=FAKE, weight=FAKE, h=2 * FAKE, n=3 * FAKE, x_stride=64, y_stride=64,
                gate_stride=0, h_stride=64, n_stride=64, rows=4, dim=64, stream_dtype=1, dtype=1, weight_dtype=1,
                activation=0, alpha=1.0, offset=0.0, eps=1e-6)
    for kw, rc in [(dict(x=None), -1), (dict(h=None, n=None), -1), (dict(y=None), -1), (dict(y=None, gate=None), -1),
                   (dict(dtype=0), -3), (dict(dtype=7), -3), (dict(stream_dtype=2), -3), (dict(weight_dtype=2), -3),
                   (dict(rows=0), -2), (dict(rows=2 ** 31), -2), (dict(dim=0), -2), (dict(dim=32769), -2),
                   (dict(x_stride=63), -2), (dict(y_stride=1), -2), (dict(gate_stride=32), -2), (dict(h_stride=-64), -2),
                   (dict(n_stride=0), -2), (dict(h=FAKE, h_stride=128), -6), (dict(n=FAKE, n_stride=128), -6),
                   (dict(activation=2), -6), (dict(activation=-1), -6), (dict(alpha=math.nan), -6), (dict(alpha=math.inf), -6),
                   (dict(offset=math.inf), -6), (dict(eps=0.0), -6), (dict(eps=-1.0), -6), (dict(eps=math.nan), -6),
                   (dict(x=FAKE + 1), -4), (dict(n=FAKE + 1), -4), (dict(stream_dtype=0, x=FAKE + 2), -4),
                   (dict(weight_dtype=0, weight=FAKE + 2), -4)]:
        assert lib.arc_norm_join(ctypes.addressof(serve.NormRows(**{**good, **kw})), None) == rc, kw
    assert lib.arc_norm_join(None, None) == -1


def test_python_refusals():
    import torch

    bf = torch.bfloat16
    x, y, w = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    for kw in [dict(y=y[:3]), dict(y=y.T), dict(y=y, weight=w[:32]), dict(y=y, gate=y[:2]), dict(gate=y), dict(post_weight=w),
               dict(y=y, activation="tanh"), dict(y=y, next_norm=False, n=y), dict(next_norm=False), dict(h=x),
               dict(y=y, dtype=torch.float16), dict(y=y)]:  # the last: host tensors
        with pytest.raises(ValueError):
            norm.join(x, **kw)
    for kw in [dict(y=y.float()), dict(y=y.half()), dict(y=y, weight=w.half()), dict(y=y, gate=y.half()),
               dict(y=y, weight=w, post_weight=w.float())]:
        with pytest.raises(TypeError):
            norm.join(x, **kw)


# ------------------------------------------------------------------ GPU
TYPES = ("bfloat16", "float16")


def case(rows, dim, kind="bfloat16", stream=None, post=True, gate=None, wide=False, pad=0, seed=0):
    """Tensors of a call: rows of `pad` more values than are used."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    t = getattr(torch, kind)
    make = lambda n, ty, s=1.0: (s * torch.randn(n, dim + pad, generator=g, device="cuda")).to(ty)[:, :dim]  # noqa: E731
    one = lambda ty: torch.randn(dim, generator=g, device="cuda").to(ty)  # noqa: E731
    kw = dict(y=make(rows, t), weight=one(torch.float32 if wide else t))
    if post:
        kw["post_weight"] = one(torch.float32 if wide else t)
    if gate == "channel":
        kw["gate"] = one(t)
    elif gate:
        kw["gate"] = make(rows, t, 3.0)
    if gate == "sigmoid":
        kw["activation"] = "sigmoid"
    return make(rows, getattr(torch, stream or kind), 2.0), kw


def wide(t):
    return None if t is None else t.double().cpu().numpy()


def check(x, kw, got, alpha=1.0, offset=0.0, eps=1e-6):
    import torch

    h, n, u = on.join(wide(x), wide(kw.get("y")), wide(kw.get("weight")), wide(kw.get("post_weight")), wide(kw.get("gate")),
                      kw.get("activation") == "sigmoid", alpha, offset, eps)
    E = 2.0 ** -17
    if kw.get("activation") == "sigmoid":
        E = E + np.abs(wide(kw["gate"])) * 2.0 ** -22
    au = np.abs(alpha * u)
    eh = E * au + 2.0 ** -23 * (np.abs(wide(x)) + au) if kw.get("y") is not None else 0.0 * au
    if kw.get("y") is not None:
        tol = eh + torch.finfo(got[0].dtype).eps / 2 * (np.abs(h) + eh) + 2.0 ** -25
        assert (np.abs(wide(got[0]) - h) <= tol).all(), np.max(np.abs(wide(got[0]) - h) / tol)
    if got[1] is not None:
        f = on.rms(h, eps)
        w = np.abs(offset + wide(kw["weight"])) if kw.get("weight") is not None else 1.0
        rel = 2.0 ** -17 + f * np.sqrt(np.mean(eh * eh, axis=-1, keepdims=True))
        en = f * w * eh + np.abs(n) * rel
        tol = en + torch.finfo(got[1].dtype).eps / 2 * (np.abs(n) + en) + 2.0 ** -25
        assert (np.abs(wide(got[1]) - n) <= tol).all(), np.max(np.abs(wide(got[1]) - n) / tol)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 8), (3, 7), (1, 4096), (5, 2048), (2, 2049), (200, 64), (301, 257), (153, 1000),
                                      (400, 1024), (2, 5120), (7, 5003), (3, 16384), (2, 16385), (2, 16392), (1, 32768),
                                      (2, 32767)])
@pytest.mark.parametrize("kind,stream", [("bfloat16", None), ("float16", "float32")])
def test_sizes(cuda_lib, rows, dim, kind, stream):
    x, kw = case(rows, dim, kind, stream, gate="sigmoid", seed=dim)
    check(x, kw, norm.join(x, **kw, alpha=0.3, offset=1.0), alpha=0.3, offset=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("stream", (None, "float32"))
@pytest.mark.parametrize("post", (False, True))
@pytest.mark.parametrize("gate", (None, "channel", "token", "sigmoid"))
@pytest.mark.parametrize("wide_weights,pad", [(False, 0), (True, 8), (False, 3)])
def test_forms(cuda_lib, kind, stream, post, gate, wide_weights, pad):
    x, kw = case(9, 1320, kind, stream, post, gate, wide_weights, pad)
    check(x, kw, norm.join(x, **kw, alpha=-1.5, eps=1e-3), alpha=-1.5, eps=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(9800, 1032), (40000, 72)])  # more rows than the grid has blocks or warps
def test_rows_in_turn(cuda_lib, rows, dim):
    x, kw = case(rows, dim, gate="token")
    check(x, kw, norm.join(x, **kw))


@pytest.mark.gpu
def test_parts(cuda_lib):
    """The norm alone, the sum alone, no weights, outputs given and in place, a gate row for all."""
    import torch

    x, kw = case(6, 520, "bfloat16", "float32")
    h, n = norm.join(x, weight=kw["weight"], offset=1.0)
    assert h is x
    check(x, dict(weight=kw["weight"]), (h, n), offset=1.0)
    check(x, {}, norm.join(x, dtype=torch.bfloat16))
    full = norm.join(x, **kw)
    h, n = norm.join(x, **kw, next_norm=False)
    assert n is None and torch.equal(h, full[0])
    y = kw.pop("y")
    out = torch.full((6, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    norm.join(x, y, **kw, n=out[:, 40:560])
    assert torch.equal(out[:, 40:560], full[1]) and (out[:, :40] == 7).all() and (out[:, 560:] == 7).all()
    g = torch.randn(1, 520, device="cuda").to(torch.bfloat16)
    a, b = norm.join(x, y, gate=g.expand(6, -1), **kw), norm.join(x, y, gate=g[0], **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x2, y2 = x.clone(), y.clone()
    h, n = norm.join(x2, y2, **kw, h=x2, n=y2)
    assert h is x2 and n is y2 and torch.equal(h, full[0]) and torch.equal(n, full[1])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(4, 2048), (300, 64)])
def test_a_bad_row_is_alone(cuda_lib, rows, dim):
    """NaN, infinite and zero rows; the others keep their bits."""
    import torch

    x, kw = case(rows, dim)
    want = norm.join(x, **kw)
    x[1, 3], kw["y"][2, 5] = float("nan"), float("inf")
    x[0], kw["y"][0] = 0, 0
    h, n = norm.join(x, **kw)
    assert torch.isnan(n[1]).all() and torch.isnan(n[2]).any()
    assert (h[0] == 0).all() and (n[0] == 0).all()
    assert torch.equal(h[3:], want[0][3:]) and torch.equal(n[3:], want[1][3:])


@pytest.mark.gpu
def test_streams_and_graphs(cuda_lib):
    import torch

    x, kw = case(64, 4096, gate="token")
    want = norm.join(x, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # the current stream is busy: nothing of the call may wait for it
    got = norm.join(x, **kw, stream=side)
    side.synchronize()
    assert torch.equal(got[0].cpu(), want[0].cpu()) and torch.equal(got[1].cpu(), want[1].cpu())
    h, n = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm.join(x, **kw, h=h, n=n)
        norm.join(h, n, weight=kw["weight"], h=h, n=n)
    for i in range(2):
        x.add_(1)
        graph.replay()
        a = norm.join(x, **kw)
        a = norm.join(a[0], a[1], weight=kw["weight"])
        assert torch.equal(a[0], h) and torch.equal(a[1], n)


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_lib):
    """Row 2 of these lies more than 2^31 values behind the first."""
    import torch

    stride = (1 << 30) + 8
    big = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 64), (stride, 1))
    src, kw = case(3, 64)
    x.copy_(src)
    want = norm.join(src, **kw)
    h, n = norm.join(x, **kw, h=x)
    assert torch.equal(h, want[0]) and torch.equal(n, want[1])

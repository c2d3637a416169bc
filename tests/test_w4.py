"""Products with 4-bit weights (include/serve/arc_w4.h) against the fp64 oracle, and their refusals.

Products are exact and sums fp32, so an output may be off by half a step of its
type and by one fp32 rounding (2^-23, tensor-core sums truncate) of the partial
sums for each 16 products, group and joined part: (ins / 16 + 2 ins / group + 16)
2^-23 sum_k |x_k| 15 s."""
import ctypes
import math
import os

import numpy as np
import pytest

from device_logits_sampling_gb300 import serve, w4
from oracle import w4 as ow


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(serve.LIB_PATH):
        from device_logits_sampling_gb300 import build

        build.build_serve()
    return serve.load()


FAKE = 0x1000


def test_refusals(lib):
    good = dict(q=FAKE, scales=FAKE, zeros=None, row_bytes=512, outs=100, ins=1024, group=128)

    def call(weight=good, x=FAKE, rows=2, xs=1024, xt=1, y=FAKE, ys=100, yt=1):
        w = serve.W4Weight(**weight)
        return lib.arc_w4_matvec(ctypes.addressof(w), x, rows, xs, xt, y, ys, yt, FAKE, 1 << 40, None)

    for kw, rc in [(dict(q=None), -1), (dict(scales=None), -1), (dict(group=16), -5), (dict(group=256), -5), (dict(outs=0), -2),
                   (dict(outs=1 << 31), -2), (dict(ins=0), -2), (dict(ins=1000), -2), (dict(ins=65536, row_bytes=32768), -2),
                   (dict(row_bytes=496), -2), (dict(row_bytes=520), -4), (dict(q=FAKE + 8), -4), (dict(scales=FAKE + 1), -4)]:
        assert call(weight={**good, **kw}) == rc, kw
    for kw, rc in [(dict(x=None), -1), (dict(y=None), -1), (dict(xt=0), -3), (dict(xt=9), -3), (dict(yt=2), -3), (dict(yt=5), -3),
                   (dict(rows=0), -2), (dict(rows=257), -2), (dict(xs=1023), -2), (dict(ys=99), -2), (dict(x=FAKE + 1), -4),
                   (dict(y=FAKE + 2, yt=0), -4)]:
        assert call(**kw) == rc, kw
    assert lib.arc_w4_matvec(None, FAKE, 1, 1024, 1, FAKE, 100, 1, None, 0, None) == -1
    assert lib.arc_w4_workspace_bytes(None, 1) == 0


def test_python_refusals():
    import torch

    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    w, s = torch.zeros(10, 128, dtype=torch.uint8), torch.zeros(10, 2, dtype=torch.bfloat16)
    for kw in (dict(x=x[0]), dict(x=x[:, ::2]), dict(weight=w[:9]), dict(weight=w[:, :64]), dict(scales=s[0]),
               dict(scales=torch.zeros(10, 3, dtype=torch.bfloat16)), dict(zeros=torch.zeros(10, 1, dtype=torch.uint8)),
               dict(out=torch.zeros(3, 9)), dict(out=torch.zeros(3, 10), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            w4.matvec(**{**dict(x=x, weight=w, scales=s), **kw})
    for kw in (dict(weight=w.float()), dict(scales=s.float()), dict(zeros=torch.zeros(10, 2)), dict(x=x.float(), scales=s.float())):
        with pytest.raises(TypeError):
            w4.matvec(**{**dict(x=x, weight=w, scales=s), **kw})


def test_oracle_pins():
    import torch

    q = np.arange(32, dtype=np.uint8).reshape(1, 32) % 16
    packed = w4.pack(torch.from_numpy(q)).numpy()
    assert np.array_equal(ow.unpack(packed)[0], q[0].astype(float))
    x = np.zeros((1, 32))
    x[0, 5] = 2.0
    y, spread = ow.matvec(x, packed, np.full((1, 1), 0.5))
    assert y[0, 0] == 2.0 * (5 - 8) * 0.5 and spread[0, 0] == 15.0
    assert ow.matvec(x, packed, np.full((1, 1), 0.5), np.full((1, 1), 3))[0][0, 0] == 2.0


def check(rows, outs, ins, group, dtype, zeros=False, f32=False, seed=0, pad=0, xpad=0, ypad=0, x=None, factor=1.0):
    import torch

    g = torch.Generator().manual_seed(seed)
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    if x is None:
        x = (torch.randn(rows, ins, generator=g) * factor).to(t)
    weight = torch.randint(0, 256, (outs, ins // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(outs, ins // group, generator=g) - 0.3) * 0.02).to(t)
    z = torch.randint(0, 16, (outs, ins // group), generator=g, dtype=torch.uint8) if zeros else None
    dw = torch.full((outs, ins // 2 + pad), 0xAB, dtype=torch.uint8, device="cuda")
    dw[:, : ins // 2] = weight
    dx = torch.full((rows, ins + xpad), math.nan, dtype=t, device="cuda")
    dx[:, :ins] = x
    ty = torch.float32 if f32 else t
    dy = torch.full((rows, outs + ypad), 77.0, dtype=ty, device="cuda")
    got = w4.matvec(dx[:, :ins], dw[:, : ins // 2], scales.cuda(), zeros=None if z is None else z.cuda(), out=dy[:, :outs])
    torch.cuda.synchronize()
    assert bool((dy[:, outs:] == 77.0).all())
    want, spread = ow.matvec(x.double().numpy(), weight.numpy(), scales.double().numpy(), None if z is None else z.numpy())
    got = got.double().cpu().numpy()
    eps = torch.finfo(ty).eps / 2
    tol = eps * np.abs(want) + (ins / 16 + 2 * ins / group + 16) * 2.0 ** -23 * spread + (2.0 ** -25 if ty == torch.float16 else 0.0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300))))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16])
def test_few_rows(cuda_lib, dtype, group, rows):
    check(rows, 333, 768, group, dtype, zeros=rows % 2 == 0, f32=rows in (1, 9), seed=rows)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group", [("bf16", 128), ("fp16", 64), ("bf16", 32)])
@pytest.mark.parametrize("rows", [17, 31, 32, 33, 64, 100, 128, 129, 200, 255, 256])
def test_many_rows(cuda_lib, dtype, group, rows):
    check(rows, 457, 1152 if rows % 2 else 256, group, dtype, zeros=rows % 3 == 0, f32=rows % 4 == 0, seed=rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5, 16, 24, 200])
@pytest.mark.parametrize("outs,ins,group", [(1, 32, 32), (15, 64, 64), (16, 128, 128), (17, 96, 32), (129, 4096, 128), (64, 32768, 128),
                                            (130, 13312, 64), (2049, 160, 32)])
def test_odd_sizes(cuda_lib, rows, outs, ins, group):
    check(rows, outs, ins, group, "bf16", zeros=True, f32=True, seed=outs)
    check(rows, outs, ins, group, "fp16", seed=ins)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 40])
def test_strides(cuda_lib, rows):
    for pad, xpad, ypad in ((16, 0, 0), (48, 8, 1), (0, 1, 3), (0, 3, 0)):
        check(rows, 150, 512, 64, "bf16", pad=pad, xpad=xpad, ypad=ypad)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [4, 20])
def test_values(cuda_lib, rows):
    import torch

    for factor in (1e4, 1e-4, 1e-30, 1e30):
        check(rows, 70, 512, 128, "bf16", f32=True, factor=factor)
    check(rows, 70, 512, 128, "fp16", f32=True, factor=1e-6)
    check(rows, 70, 512, 128, "fp16", f32=True, factor=1e4)
    # rows of very different size, values of one row 2^30 apart, zeros
    x = torch.randn(rows, 512).to(torch.bfloat16)
    x[0] *= 2.0 ** 60
    x[1, ::2] *= 2.0 ** -30
    x[2] = 0.0
    check(rows, 70, 512, 64, "bf16", f32=True, x=x)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [4, 20])
def test_not_finite(cuda_lib, rows):
    """An infinite or NaN value spoils its own row alone."""
    import torch

    x = torch.randn(rows, 256).to(torch.bfloat16)
    x[1, 17], x[3, 200] = math.nan, math.inf
    w = torch.full((40, 128), 0x99, dtype=torch.uint8, device="cuda")  # every weight 1
    y = w4.matvec(x.cuda(), w, torch.ones(40, 2, dtype=torch.bfloat16, device="cuda"), out_dtype=torch.float32).cpu()
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[3]).any())
    ok = [r for r in range(rows) if r not in (1, 3)]
    assert bool(torch.isfinite(y[ok]).all())


@pytest.mark.gpu
def test_weights_past_32_bits(cuda_lib):
    import torch

    outs, ins = 270000, 32768
    w = torch.zeros(outs, ins // 2, dtype=torch.uint8, device="cuda")
    assert w.numel() > 1 << 32
    w[-1] = 0x99
    s = torch.ones(outs, ins // 128, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(1, ins, dtype=torch.bfloat16, device="cuda")
    y = w4.matvec(x, w, s, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert y[0, -1].item() == ins and y[0, -2].item() == -8.0 * ins and y[0, 0].item() == -8.0 * ins


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 16, 64])
def test_streams_and_graphs(cuda_lib, rows):
    import torch

    x = torch.randn(rows, 1024, device="cuda").to(torch.bfloat16)
    w = torch.randint(0, 256, (500, 512), device="cuda", dtype=torch.uint8)
    s = torch.rand(500, 8, device="cuda").to(torch.bfloat16)
    want = w4.matvec(x, w, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = w4.matvec(x, w, s)
    side.synchronize()
    assert torch.equal(want, b)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.matvec(x, w, s, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)

"""4-bit products of 1 to 8 rows whose blocks take many tiles of outputs one after another, with rare joins:
a warp's scales are written again for each tile, so every repeat has to give the same bits, and each output
the value that a product of its weight row alone gives."""
import pytest

from device_logits_sampling_gb300 import w4


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,outs,ins,group", [(1, 70001, 512, 32), (8, 60000, 768, 64), (3, 50003, 4096, 128), (5, 30001, 256, 32)])
def test_every_repeat_has_the_same_bits(cuda_lib, rows, outs, ins, group, zeros):
    import torch

    g = torch.Generator(device="cuda").manual_seed(rows + outs)
    x = torch.randn(rows, ins, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(0, 256, (outs, ins // 2), generator=g, device="cuda", dtype=torch.uint8)
    # scales that double from one row to the next, eight rows long: a neighbour's or an older tile's shows
    s = (2.0 ** (torch.arange(outs, device="cuda") % 8 - 8.0))[:, None].expand(outs, ins // group).to(torch.bfloat16).contiguous()
    z = torch.randint(0, 16, (outs, ins // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    outputs = [w4.matvec(x, w, s, zeros=z, out_dtype=torch.float32) for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(outputs[0], y) for y in outputs[1:])
    q = torch.stack([w & 15, w >> 4], -1).reshape(outs, ins).double()
    q -= 8.0 if z is None else z.double().repeat_interleave(group, 1)
    sums = s.double().repeat_interleave(group, 1)
    want, spread = x.double() @ (q * sums).T, x.double().abs() @ (15.0 * sums).T
    # half a step of fp32 and one fp32 rounding (2^-23, tensor-core sums truncate) for each 16 products, group and
    # joined part
    tol = 2.0 ** -24 * want.abs() + (ins / 16 + 2 * ins / group + 16) * 2.0 ** -23 * spread
    assert bool(((outputs[0].double() - want).abs() <= tol).all())

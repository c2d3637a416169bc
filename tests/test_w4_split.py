"""4-bit products whose inner dimension is split over a cluster (few outputs, long inner dimension): the
block's sums are written over the memory that its last products read x from, so every repeat has to
give the first one's bits, and the first one the oracle's values."""
import numpy as np
import pytest

from device_logits_sampling_gb300 import w4
from oracle import w4 as ow


@pytest.mark.gpu
@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("rows", [129, 192, 256])
@pytest.mark.parametrize("outs,ins", [(4096, 11008), (640, 4224), (300, 1152), (1000, 8704)])  # odd and even shares
def test_every_repeat_has_the_same_bits(cuda_lib, rows, outs, ins, group):
    import torch

    g = torch.Generator(device="cuda").manual_seed(rows + outs)
    x = torch.randn(rows, ins, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(0, 256, (outs, ins // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(outs, ins // group, generator=g, device="cuda") * 0.01 + 0.002).to(torch.bfloat16)
    outputs = [w4.matvec(x, w, s, out_dtype=torch.float32) for _ in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(outputs[0], y) for y in outputs[1:])
    some = np.linspace(0, outs - 1, 97).astype(int)
    want, spread = ow.matvec(x.double().cpu().numpy(), w.cpu().numpy()[some], s.double().cpu().numpy()[some])
    got = outputs[0][:, torch.from_numpy(some).cuda()].double().cpu().numpy()
    # half a step of fp32 and one fp32 rounding (2^-23, tensor-core sums truncate) for each 16 products, group and
    # joined part
    tol = 2.0 ** -24 * np.abs(want) + (ins / 16 + 2 * ins / group + 16) * 2.0 ** -23 * spread
    assert (np.abs(got - want) <= tol).all()

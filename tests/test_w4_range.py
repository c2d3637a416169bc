"""4-bit products of rows near the ends of the 16-bit types' ranges: the factors that rows are scaled by, and
the products' unit of 2^-24, are powers of two that must not push a normal output out of fp32's normal range."""
import pytest

import test_w4


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 4, 8, 9, 20, 200])
@pytest.mark.parametrize("factor", [1e-36, 3e-37, 1e34])
def test_tiny_and_huge_rows(cuda_lib, rows, factor):
    import torch

    test_w4.check(rows, 70, 512, 128, "bf16", f32=True, factor=factor)
    # few distinct values, none of which loses bits as bf16: weights times scales of 1, outputs far above 2^-126
    x = torch.full((rows, 4352), 1.5) * factor
    test_w4.check(rows, 40, 4352, 128, "bf16", f32=True, x=x.to(torch.bfloat16))


@pytest.mark.gpu
def test_eight_and_nine_rows_agree(cuda_lib):
    """Two kernels meet at eight rows; a weight of 1 times a single value is that value's exact product."""
    import torch
    from device_logits_sampling_gb300 import w4

    w = torch.full((33, 256), 0x99, dtype=torch.uint8, device="cuda")
    s = torch.full((33, 4), 2.0 ** -6, dtype=torch.bfloat16, device="cuda")
    for e in (-118, -110, -60, 0, 60, 110):
        x = torch.zeros(9, 512, dtype=torch.bfloat16, device="cuda")
        x[:, 5] = 1.3671875 * 2.0 ** e
        few, many = w4.matvec(x[:8], w, s, out_dtype=torch.float32), w4.matvec(x, w, s, out_dtype=torch.float32)
        want = torch.full((8, 33), 1.3671875 * 2.0 ** (e - 6), dtype=torch.float32, device="cuda")
        assert torch.equal(few, want) and torch.equal(many[:8], want), e

"""Keys whose rotation ends inside a thread's sixteen values, or between two threads': NaN and infinite values past
its end are stored as those of any other key are (as 0, and as the largest code), beside values that turn."""
import math

import pytest

from test_kv_cache import Case, check_append

SHAPES = [(64, 20, "half"), (64, 20, "interleaved"), (128, 50, "half"), (128, 50, "interleaved"), (256, 254, "interleaved"),
          (256, 254, "half"), (64, 32, "half"), (64, 0, "half")]


def keys_with(value, dim, rot, layout, single):
    c = Case(41, dim, 16, 2, 2, [0, 5, 16, 40], [1] * 4 if single else [2, 3, 1, 20], "bf16", rot=rot, layout=layout)
    for t in range(len(c.nk)):
        c.nk[t, t % 2, rot + t % (dim - rot)] = value
    c.nk[0, 0, dim - 1] = value
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("dim,rot,layout", SHAPES)
def test_nan_past_the_rotation(cuda_lib, dim, rot, layout, single):
    check_append(keys_with(math.nan, dim, rot, layout, single), single=single, err_want=4)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("dim,rot,layout", SHAPES)
def test_infinite_past_the_rotation(cuda_lib, dim, rot, layout, single):
    for value in (math.inf, -math.inf):
        check_append(keys_with(value, dim, rot, layout, single), single=single)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
def test_infinite_keys_without_a_rotation(cuda_lib, single):
    import torch
    from device_logits_sampling_gb300 import kv_cache

    n = 3
    cache = kv_cache.PagedCache.empty(8, 1, 16, 64)
    k = torch.ones(n, 1, 64, device="cuda", dtype=torch.float16)
    k[1, 0, 7], k[2, 0, 63] = math.inf, -math.inf
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    pos, offs = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n + 1, dtype=torch.int32, device="cuda")
    kv_cache.append(cache, k, k, pos, table, row_offsets=None if single else offs)
    torch.cuda.synchronize()
    for codes in (cache.k, cache.v):
        codes = codes.view(torch.uint8)[:n, 0, 0].cpu()
        assert codes[1, 7] == 0x7E and codes[2, 63] == 0xFE
        assert not ((codes & 0x7F) == 0x7F).any()

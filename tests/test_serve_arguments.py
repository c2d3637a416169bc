"""Whole numbers that do not fit the 32 bits of the C calls are refused, not cut."""
import pytest

from device_logits_sampling_gb300 import kv_cache


def small_cache():
    import torch

    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.ones(4, 2)
    return kv_cache.PagedCache(k, k.clone(), s, s.clone())


@pytest.mark.parametrize("sinks", [1 << 31, 1 << 32, (1 << 32) + 4, -(1 << 32), -(1 << 31) - 1])
def test_sinks(sinks):
    import torch

    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="sinks"):
        kv_cache.attend(small_cache(), x, pos, table, window=8, sinks=sinks)


@pytest.mark.parametrize("heads", [(1 << 32) + 8, 1 << 32, 1 << 31, -(1 << 32) + 8])
def test_heads_of_a_workspace(heads):
    with pytest.raises(ValueError, match="heads"):
        small_cache().shared_workspace(3, heads)

"""The Python binding of the attention's cache refuses numbers that the C
argument blocks cannot hold (no GPU).
"""
import pytest
import torch

from linear_attention_serving_delta_gb300 import kda


@pytest.mark.parametrize("page_size", [(1 << 32) + 16, (1 << 31), -(1 << 32) + 16])
def test_page_sizes_past_32_bits(page_size):
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    free, count = torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="page_size"):
        kda.KvPlan(torch.tensor([0, 4]), 4, table, lens, free, count, page_size=page_size)
    with pytest.raises(ValueError, match="page_size"):
        kda.KvRelease(torch.zeros(1, dtype=torch.int32), table, lens, free, count, page_size=page_size)


def test_numbers_that_fit():
    assert kda._i32("x", (1 << 31) - 1) == (1 << 31) - 1 and kda._i32("x", -(1 << 31)) == -(1 << 31)
    with pytest.raises(ValueError):
        kda._i32("max_seqlen", -(1 << 32))

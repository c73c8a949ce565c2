"""Integers past 32 bits are refused, not passed on without their upper bits."""
import pytest
import torch

import weight_only_int4_w4a16_amd as w


@pytest.mark.parametrize("value", [2 ** 32 + 16, 2 ** 31, -2 ** 31 - 1, 2 ** 70])
def test_page_size_and_window_past_32_bits(value):
    ints = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="page_size must fit"):
        w.page_tables(ints, ints, ints[None], ints, value, max_tokens=4)
    with pytest.raises(ValueError, match="window must fit"):
        w.paged_attention(q, cache, cache, ints[None], ints, window=value)


def test_what_is_no_integer():
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        w.page_tables(ints, ints, ints[None], ints, 16.0, max_tokens=4)

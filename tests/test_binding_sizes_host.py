"""Numbers that do not fit the C calls' 32-bit integers are refused by name: ctypes would pass their
low 32 bits on, and a limit of 2^32 + 64 tokens would become one of 64."""
import pytest
import torch

import decode_attention_stief_b200 as stief
from decode_attention_stief_b200 import _binding


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 64, -2 ** 31 - 1])
def test_limits_past_32_bits(value):
    i = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros((2, 64, 48), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="page_size does not fit 32 bits"):
        stief.stief_plan_pages(i, i, i.view(2, 2), i, i[:1], None, None, None, None, i[:1], i, value)
    with pytest.raises(ValueError, match="max_seq_len does not fit 32 bits"):
        stief.stief_decode_shared_paged(b, b, i.view(2, 2), i, b, i, value, 0.1)
    with pytest.raises(ValueError, match="max_q_len does not fit 32 bits"):
        stief.stief_prefill_attention(b, b, b, i, i, b, value, 0.1)


def test_sizes_past_32_bits():
    assert _binding._sizes("f", -2 ** 31, 0, 2 ** 31 - 1) == (-2 ** 31, 0, 2 ** 31 - 1)
    for sizes in ((5, 2 ** 31), (2 ** 32 + 3,), (-2 ** 31 - 1, 1)):
        with pytest.raises(ValueError, match="f: a size does not fit 32 bits"):
            _binding._sizes("f", *sizes)

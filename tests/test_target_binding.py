"""CPU checks of the target side's binding: numbers that the C call would take
cut down to 32 bits."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from target_ref import paged_case


def test_numbers_beyond_32_bits_are_refused():
    c = paged_case(1, torch.bfloat16, 64, 4, 2, 16, [3, 2], [5, 0], device="cpu")
    args = (c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    for kw in (dict(window=2**32 + 7), dict(window=-2**31 - 1), dict(max_len=-2**33)):
        with pytest.raises(ValueError, match="32 bits"):
            df2.paged_attention(*args, **kw)
    # an estimate may be as large as it likes
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.paged_attention(*args, max_len=2**40)
    wide = torch.zeros(1).expand(1, 2, 2**32 + 10)
    with pytest.raises(ValueError, match="32 bits"):
        df2.verify(wide, torch.zeros((1, 1), dtype=torch.int32), temperature=0.0)

"""What the 4-bit cache's binding refuses before anything is launched."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_bit_gb300 as sdv
from speculative_decoding_tree_bit_gb300 import _build


@pytest.fixture(scope="module")
def M():
    _build.build()
    sdv.lib()
    from speculative_decoding_tree_bit_gb300 import model
    return model


def rows16(n, heads, dim=128):
    return torch.zeros(n, heads, dim, dtype=torch.bfloat16)


def test_slopes_and_starts_too_short_are_refused(M):
    """They are read by query head and by request."""
    c = M.KV4Cache(np.zeros((3, 1)), 1, 2, 128, 64, device="cpu")
    rows, q, lse = M.RequestRows([0, 1, 2, 4], device="cpu"), rows16(4, 8), torch.zeros(4, 8)
    for score, what in ((M.KV4Score(slopes=torch.zeros(7)), "slopes"), (M.KV4Score(slopes=torch.zeros(0)), "slopes"),
                        (M.KV4Score(start=torch.zeros(2, dtype=torch.int32)), "start")):
        with pytest.raises(ValueError, match=what):
            c.attend(q, rows, score=score)
        with pytest.raises(ValueError, match=what):
            c.observe(q, lse, rows, score=score)

"""Refusals of the calls around the top-k that need no device."""
import pytest
import torch

from drafter_vocab_top_amd import topk_cols as T


@pytest.mark.parametrize("index", [False, True])
def test_adjust_refuses_a_mask_without_rows(index):
    """An empty tensor has no address: it must not turn into no mask at all."""
    with pytest.raises(ValueError, match="at least one row"):
        T.AdjustRules(100, 14, lanes=2, mask=torch.zeros((0, 4), dtype=torch.int32),
                      mask_index=torch.zeros(14, dtype=torch.int32) if index else None)

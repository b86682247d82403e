"""Refusals of the paged cache's entry points at the edges of what they can
address (no device is needed: nothing is launched)."""
import math

import pytest

from drafter_vocab_top_amd import topk_cols as T
from test_tree_abi import BAD, CACHE, FP8, LARGE, attend, lib, move, workspace, write  # noqa: F401


@pytest.mark.parametrize("base", [CACHE, FP8], ids=["bf16", "fp8"])
def test_the_last_row_ends_within_64_gib(lib, base):  # noqa: F811
    """Offsets are 32-bit numbers of 16 bytes: a row that starts below 2^32 of them and ends behind has a part that
    would be read from the layer's start."""
    each = 8 if base is CACHE else 16  # elements of 16 bytes
    row = base["dim"] // each
    for past in (1, row - 1):
        for kw in (dict(blocks=2, block_size=1, block_stride=((1 << 32) - row + past) * each),
                   dict(blocks=1, block_size=2, slot_stride=((1 << 32) - row + past) * each),
                   dict(blocks=2, block_size=2, block_stride=(1 << 31) * each, slot_stride=((1 << 31) - row + past) * each)):
            c = dict(base, **kw)
            assert write(lib, c) == attend(lib, c) == move(lib, c) == LARGE, kw
            assert workspace(lib, c) == (LARGE, 0), kw
    for kw in (dict(blocks=2, block_size=1, block_stride=((1 << 32) - row) * each),
               dict(blocks=1, block_size=2, slot_stride=((1 << 32) - row) * each)):
        assert workspace(lib, dict(base, **kw))[0] == T.TOPK_OK, kw


def test_scales_beyond_2_127_are_refused(lib):  # noqa: F811
    """Scores are multiplied by scale * log2(e) in binary32: where that overflows, a score of 0 would become NaN."""
    for scale in (2.0**127 * (1 + 2**-23), 3.4e38, -2.0**127 * (1 + 2**-23), math.inf, -math.inf):
        assert attend(lib, scale=scale) == BAD, scale
        assert workspace(lib, scale=scale) == (BAD, 0), scale
    for scale in (2.0**127, -2.0**127, 0.0, 1e-45):
        assert workspace(lib, scale=scale)[0] == T.TOPK_OK, scale

"""How the CTAs of the 8-bit decode share the keys, walked on the host by the kernels' own arithmetic (CPU
only): every block of keys once, no queries of a unit that is not there, and each unit's pieces where its
merge looks for them."""
import random

import pytest

import q8_line


@pytest.mark.parametrize("block", [64, 128])
def test_joined_splits(block):
    """Splits past the end of a short sequence have no blocks, and no unit after their own: the last unit of
    the last sequence has none behind it."""
    for spans in ([100], [0], [2000], [2000, 10], [5, 1999, 0], [1, 900, 128, 129]):
        for splits in range(1, 9):
            for chunk in (1, 2, 5):
                if chunk * splits * block < max(spans):
                    continue
                assert q8_line.joined(spans, 8, block, chunk, splits) == 0, (spans, splits, chunk)

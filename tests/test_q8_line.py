"""How the CTAs of the 8-bit decode share the keys, walked on the host by the kernels' own arithmetic (CPU
only): every block of keys once, no queries of a unit that is not there, and each unit's pieces where its
merge looks for them."""
import ctypes
import random

import pytest

import q8_line
from attention_forward_blackwell_gb300 import binding, build


@pytest.mark.parametrize("page", [1, 7, 16, 64, 4096 - 64])
def test_longest_tables(page):
    """Tables whose positions would leave 32 bits on the way are refused (the host's check, before any
    launch): a slice past the last key would wrap round to the first."""
    build.build()
    at = lambda x: ctypes.c_void_p(x)
    for keys in {2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 128, 2 ** 31 - 4095}:
        pages = keys // page
        if pages * page <= 2 ** 31 - 4096:
            pages += 1
        if pages * page >= 2 ** 31:
            continue
        st = binding.lib().fa_fwd_decode_paged_q8(
            at(1 << 12), at(1 << 12), at(1 << 12), at(1 << 12), at(1 << 12), at(1 << 12), at(1 << 12), 1, 4, 2, 1,
            at(1 << 12), at(1 << 12), pages, page, 9, page, 64, 0.1, 1, 0, 0, None, None)
        assert st == binding.FA_ERR_INVALID_ARG, (page, pages)
    for block in (64, 128):   # the last block of the longest table ends within 32 bits
        assert q8_line.lib().line_unit_blocks(2 ** 31 - 4096, block) * block + 2 * block < 2 ** 31


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


def kind_of(cut):
    if cut["aligned"] > 0:
        return "aligned"
    return "two sizes" if cut["small"] > 1 else "uneven"


@pytest.mark.parametrize("kind", ["aligned", "uneven", "two sizes"])
def test_lines(kind):
    """Pieces that end with their units, even pieces, and large ones with small ones behind them."""
    rng = random.Random(kind)
    seen = 0
    for _ in range(4000):
        block, units, slots = rng.choice((64, 128)), rng.choice((1, 2, 3, 8)), rng.randint(1, 40)
        B, most = rng.randint(1, 60), 10 ** rng.uniform(0, 5)
        spans = [int(rng.choice((0, 1, most * rng.random(), most))) for _ in range(B)]
        levels = rng.choice((0, 2))
        bad, cut = q8_line.line(spans, units, block, slots, levels)
        assert bad == 0, (bad, spans, units, block, slots, levels, cut)
        seen += kind_of(cut) == kind
        if seen == 50:
            return
    assert False, f"{seen} lines"

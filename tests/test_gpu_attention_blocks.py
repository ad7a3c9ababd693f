"""GPU: block sizes whose common part with a tile is a few keys, in every form
of the window attention, and rows of one call that differ in everything.
Oracle and bounds as for the window attention."""

import numpy as np
import pytest

from tests.attention_helpers import Case
from tests.test_gpu_window_attention import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block_size", [4, 8, 24, 40, 56])
@pytest.mark.parametrize("group,window", [(6, 7), (12, 8), (16, 8)])
def test_blocks_of_a_few_keys(dim, block_size, group, window):
    c = Case([window, 1, 3], [block_size * 7 - 2, 0, 511], group, 1, dim, block_size,
             seed=block_size + dim)
    _check(c, window)
    _check(c, window, left_window=70)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,window", [(1, 2), (5, 6), (4, 4), (8, 8), (16, 8)])
def test_ragged_rows_next_to_long_ones(dim, group, window):
    # a run may hold the end of one row, several whole short ones and the start
    # of a long one; every other table entry of one row is the null block
    rng = np.random.default_rng(dim + group)
    lens = [int(n) for n in rng.integers(0, window + 1, size=40)]
    computed = [int(n) for n in rng.integers(0, 90, size=40)]
    lens[3], computed[3], lens[20], computed[20] = window, 5000, 1, 3001
    c = Case(lens, computed, 2 * group, 2, dim, 24, seed=31)
    c.table[20, ::2] = 0
    _check(c, window)


@pytest.mark.parametrize("heads", [1, 3, 7])
def test_heads_and_rows_that_divide_nothing(heads):
    # fewer tiles than CTAs, as many, and a few more
    for rows in (1, 43, 101, 152 // heads + 1, 304 // heads + 1, 456 // heads + 1):
        c = Case([1] * rows, [(i * 37) % 63 for i in range(rows)], heads, heads, 64, 16,
                 seed=rows)
        _check(c, 1)

"""GPU: keys and values behind a sliding window, which no query of the row
sees but which lie in the first tile of 64 keys that the row reads.  Whatever
they hold (NaN, infinities, table entries that are not the row's any more), the
results keep the bits they have with ordinary numbers there, and those are
held to the oracle."""

import pytest
import torch

from tests.attention_helpers import Case
from tests.test_gpu_window_attention import _check, _run

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), float("-inf")]
# (channels, query heads a key head, window, block size): each kernel form
FORMS = [(64, 1, 1, 16), (128, 4, 4, 16), (128, 4, 8, 16), (64, 8, 8, 24), (128, 5, 8, 4),
         (64, 16, 8, 4), (128, 16, 8, 4),                      # mma.sync
         (128, 8, 8, 16), (128, 16, 8, 32), (64, 16, 8, 16), (128, 64, 1, 16), (64, 96, 1, 8)]


def _poison(c, row, first, end, bad):
    bs = c.block_size
    for p in range(first, end):
        block = int(c.table[row, p // bs])
        c.keys[block, p % bs] = bad
        c.values[block, p % bs] = bad


@pytest.mark.parametrize("dim,group,window,block_size", FORMS)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("left,computed", [(40, 90), (1, 64), (30, 157), (100, 226)])
def test_what_no_query_sees(dim, group, window, block_size, bad, left, computed):
    tokens = [window, 1, window]
    before = [computed, computed + 2, 20]     # the last row's window starts at 0
    c = Case(tokens, before, 2 * group, 2, dim, block_size, seed=left + group)
    clean, clean_lse = _check(c, window, left_window=left)
    for b in range(2):
        low = before[b] + 1 - left            # the first key that a query sees
        # all of the first tile before it, and one key of it alone
        _poison(c, b, low // 64 * 64, low, bad)
    out, lse = _run(c, window, left)
    assert int(c.err.item()) == 0
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dim,group,window,block_size", FORMS)
def test_one_bad_value_right_behind_the_window(dim, group, window, block_size):
    left, computed = 50, 100
    c = Case([window], [computed], 2 * group, 2, dim, block_size, seed=group)
    clean, clean_lse = _check(c, window, left_window=left)
    _poison(c, 0, computed - left, computed + 1 - left, float("nan"))
    out, lse = _run(c, window, left)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dim,group,window,block_size",
                         [f for f in FORMS if f[3] <= 32 and f[3] % 8 == 0] + [(128, 16, 8, 4)])
def test_table_entries_behind_the_window_are_not_looked_at(dim, group, window, block_size):
    # blocks that lie wholly behind the window may be anybody's by now
    left, computed = 33, 150
    c = Case([window, 1], [computed, computed + 1], 2 * group, 2, dim, block_size, seed=group + 1)
    clean, clean_lse = _check(c, window, left_window=left)
    for b, before in enumerate((computed, computed + 1)):
        c.table[b, :(before + 1 - left) // block_size] = c.keys.shape[0] + 5
    out, lse = _run(c, window, left)
    assert int(c.err.item()) == 0
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dim,group,window,block_size",
                         [(128, 4, 4, 16), (64, 8, 8, 24), (128, 8, 8, 16), (128, 16, 8, 32)])
def test_behind_a_long_window_that_many_share(dim, group, window, block_size):
    left, computed = 6001, 9000
    c = Case([window], [computed], group, 1, dim, block_size, seed=5)
    clean, clean_lse = _check(c, window, left_window=left)
    low = computed + 1 - left
    _poison(c, 0, low // 64 * 64, low, float("nan"))
    out, lse = _run(c, window, left)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)

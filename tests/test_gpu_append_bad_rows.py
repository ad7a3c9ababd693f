"""GPU: rows that the append has to report although no token leads to them:
a negative count between others, rows that start where the tokens end.  What
the rows that are right hold alone is written as if the others were not there."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import attention_oracle as A
from tests.attention_helpers import Case, f64, frequencies, half_step

pytestmark = pytest.mark.gpu


def _append(c, tokens, **kw):
    q_out = torch.full((tokens, c.q_heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    api.kda_kv_append(c.q[:tokens], c.k[:tokens], c.v[:tokens], c.keys, c.values, c.cu, c.table,
                      c.computed, q_out=q_out, error_word=c.err, **kw)
    torch.cuda.synchronize()
    return q_out


def test_a_negative_count_between_rows():
    c = Case([5, 3, 5], [0, 9, 30], 4, 2, 64, 8, seed=1)
    c.cu = torch.tensor([0, 5, 3, 8], dtype=torch.int32, device="cuda")
    freq = frequencies(64)
    before_k, before_v = c.keys.clone(), c.values.clone()
    q_out = _append(c, 8, inv_freq=freq)
    assert int(c.err.item()) == api.ROW_BAD_LENGTH
    table, computed = c.table.cpu().numpy(), [0, 9, 30]
    k = f64(c.k)
    own = [(0, t, t) for t in range(3)] + [(2, t, t - 3) for t in range(5, 8)]
    for row, token, at in own:      # tokens 3 and 4 lie in both rows
        p = computed[row] + at
        want = A.rotate(k[token][None], np.array([p]), f64(freq), False)[0]
        got = f64(c.keys[int(table[row, p // 8]), p % 8])
        size = np.abs(k[token]).max()
        assert np.all(np.abs(got - want) <= half_step(c.dtype) * np.abs(want) * 1.001 + 2e-6 * size)
        assert torch.equal(c.values[int(table[row, p // 8]), p % 8], c.v[token])
        q = A.rotate(f64(c.q[token])[None], np.array([p]), f64(freq), False)[0]
        assert np.all(np.abs(f64(q_out[token]) - q) <= half_step(c.dtype) * np.abs(q) * 1.001
                      + 2e-6 * np.abs(f64(c.q[token])).max())
    # nothing but the two rows' five places each can have been written
    touched = torch.zeros(c.keys.shape[:2], dtype=torch.bool)
    for row in (0, 2):
        for at in range(5):
            p = computed[row] + at
            touched[int(table[row, p // 8]), p % 8] = True
    keep = ~touched.cuda()
    assert torch.equal(c.keys[keep], before_k[keep])
    assert torch.equal(c.values[keep], before_v[keep])


def test_a_negative_count_at_the_end():
    c = Case([3, 2], [0, 0], 4, 2, 64, 8, seed=2)
    c.cu = torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda")
    q_out = _append(c, 5)
    assert int(c.err.item()) == api.ROW_BAD_LENGTH
    assert torch.equal(q_out[:2], c.q[:2])
    for t in range(2):
        assert torch.equal(c.keys[int(c.table[0, 0]), t], c.k[t])


@pytest.mark.parametrize("start", [3, 4])
def test_a_row_that_starts_where_the_tokens_end(start):
    c = Case([3, 2, 2], [0, 1, 2], 4, 2, 64, 8, seed=3)
    c.cu = torch.tensor([0, 3, start, 7], dtype=torch.int32, device="cuda")
    q_out = _append(c, 3)
    assert int(c.err.item()) == api.ROW_BAD_LENGTH
    assert torch.equal(q_out, c.q[:3])


@pytest.mark.parametrize("rows,bad", [(40, 39), (700, 0), (5000, 4321), (5000, 4999)])
def test_one_bad_row_of_many(rows, bad):
    # two tokens, all in row 7; another row claims tokens that are not there
    c = Case([2], [3], 4, 2, 64, 8, seed=4)
    cu = np.zeros(rows + 1, dtype=np.int32)
    cu[8:] = 2
    c.table = c.table.repeat(rows, 1)
    c.computed = torch.full((rows,), 3, dtype=torch.int32, device="cuda")
    c.cu = torch.from_numpy(cu).cuda()
    q_out = _append(c, 2)
    assert int(c.err.item()) == 0 and torch.equal(q_out, c.q)
    if bad > 7:
        cu[bad + 1:] = 5        # starts at the tokens' end
    else:
        cu[0] = -1
    c.cu = torch.from_numpy(cu).cuda()
    q_out = _append(c, 2)
    assert int(c.err.item()) == api.ROW_BAD_LENGTH and torch.equal(q_out, c.q)


def test_a_request_that_is_not_there_in_a_row_of_its_own():
    c = Case([2, 3, 1], [0, 4, 9], 4, 2, 64, 8, seed=5)
    req = torch.tensor([0, 9, 2], dtype=torch.int32, device="cuda")
    q_out = _append(c, 6, request_indices=req)
    assert int(c.err.item()) == api.ROW_BAD_BLOCK
    assert torch.equal(q_out[:2], c.q[:2]) and torch.equal(q_out[5:], c.q[5:])
    assert bool((q_out[2:5] == 7.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_frequency_that_is_no_number(bad, interleaved):
    # its pair's channels are no numbers either, the others are as they were
    c = Case([2, 1], [0, 9], 4, 2, 64, 8, "fp16", seed=6)
    freq = frequencies(32)
    want = _append(c, 3, inv_freq=freq, interleaved=interleaved)
    keys = c.keys.clone()
    freq[5] = bad
    q_out = _append(c, 3, inv_freq=freq, interleaved=interleaved)
    pair = [10, 11] if interleaved else [5, 21]
    rest = [i for i in range(64) if i not in pair]
    assert torch.isnan(q_out[..., pair]).all() and torch.equal(q_out[..., rest], want[..., rest])
    for row, p in ((0, 0), (0, 1), (1, 9)):
        at = int(c.table[row, p // 8]), p % 8
        assert torch.isnan(c.keys[at][..., pair]).all()
        assert torch.equal(c.keys[at][..., rest], keys[at][..., rest])

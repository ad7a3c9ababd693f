"""GPU: the cache append against the float64 oracle.

Bound: the phase is exact modulo a turn up to fp64's rounding of the
frequency (2^-53 of it per position, as in the oracle's own angle), its top
32 bits become an fp32 angle (2^-24 of at most pi), sine and cosine are
within 2^-22, and the two products and their sum within 3 * 2^-24: at most
1e-6 (|x0| + |x1|), then half a step of the storage type."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import attention_oracle as A
from tests.attention_helpers import Case, f64, frequencies, half_step, smallest_half

pytestmark = pytest.mark.gpu


def _check(c, rotary, interleaved, with_q=True, requests=None, inplace=False, want_err=0):
    freq = frequencies(rotary) if rotary else None
    cu, table, computed = c.meta()
    req = None if requests is None else torch.tensor(requests, dtype=torch.int32, device="cuda")
    keys, values = f64(c.keys), f64(c.values)
    q = f64(c.q) if with_q else None
    want_q, touched, issues = A.append(q, f64(c.k), f64(c.v), keys, values, cu, table, computed,
                                       [] if freq is None else f64(freq), interleaved, requests)
    before_k, before_v = c.keys.clone(), c.values.clone()
    if inplace:
        c.q = c.q.contiguous()
    q_out = None
    if with_q:
        q_out = c.q if inplace else torch.full(c.q.shape, 7.0, dtype=c.dtype, device="cuda")
    got = api.kda_kv_append(c.q if with_q else None, c.k, c.v, c.keys, c.values, c.cu, c.table,
                            c.computed, inv_freq=freq, interleaved=interleaved, q_out=q_out,
                            request_indices=req, error_word=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == want_err
    mark = torch.from_numpy(touched).cuda()[:, :, None, None]
    # what no row wrote has its old bits; values are copies
    assert torch.equal(torch.where(mark, before_k, c.keys), before_k)
    assert torch.equal(c.values, torch.from_numpy(values).to(c.dtype).cuda())
    step, least = half_step(c.dtype), smallest_half(c.dtype)

    def near(x, ref, source):
        size = np.abs(source).max(axis=-1, keepdims=True) * 2
        assert np.all(np.abs(x - ref) <= step * np.abs(ref) * 1.001 + 1e-6 * size + least)
    near(f64(c.keys), keys, keys)
    if with_q:
        written = ~np.isnan(want_q)
        ref = np.where(written, want_q, f64(q_out))
        near(f64(got), ref, np.where(written, want_q, 0.0))
        if not inplace:
            assert np.all(f64(got)[~written] == 7.0)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rotary", [(128, 128), (128, 64), (64, 64), (64, 16), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_and_layouts(dtype, dim, rotary, interleaved):
    layout = {128: "heads", 64: "pairs"}[dim] if rotary != 64 else "tokens"
    c = Case([1, 4, 0, 7, 2], [0, 15, 3, 30, 129], 6, 2, dim, 16, dtype, layout, seed=dim + rotary)
    _check(c, rotary, interleaved)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (5, 5), (16, 1), (28, 4), (64, 8)])
@pytest.mark.parametrize("block_size", [1, 5, 24, 128])
def test_heads_and_block_sizes(q_heads, kv_heads, block_size):
    c = Case([3, 1, 8], [0, 23, 50], q_heads, kv_heads, 64, block_size, seed=block_size)
    _check(c, 64, False)


def test_no_queries_and_in_place_queries():
    _check(Case([2, 5], [3, 0], 4, 4, 128, 16, seed=1), 128, False, with_q=False)
    _check(Case([2, 5], [3, 0], 4, 4, 128, 16, seed=1), 128, True, inplace=True)


def test_far_positions():
    # positions past a million: the table's columns before the row's are the
    # null block, so the cache stays small
    c = Case([4, 3], [0, 0], 4, 2, 128, 16, "fp16", seed=2)
    far = [(1 << 20) + 3, 2_000_000_011]
    real = c.table.clone()
    c.computed = torch.tensor(far, dtype=torch.int32, device="cuda")
    c.table = torch.zeros((2, far[1] // 16 + 2), dtype=torch.int32, device="cuda")
    for b, p in enumerate(far):
        c.table[b, p // 16] = real[b, 0]
        c.table[b, p // 16 + 1] = 1 + int(real.max()) + b
    _check(c, 128, False)


def test_prompts_and_many_empty_rows():
    lens = [0] * 70 + [301] + [0] * 40 + [1, 0, 130] + [0] * 33
    _check(Case(lens, [i % 7 for i in range(len(lens))], 8, 2, 128, 32, seed=3), 128, False)


def test_request_indices_and_bad_metadata():
    c = Case([2, 3, 1, 2, 2, 4], [5, 9, 0, 3, 1, 2], 4, 2, 64, 4, seed=4, extra_columns=0)
    req = [5, 0, 6, -1, 2, 1]              # rows 2 and 3: no such request
    c.computed[2] = -3                     # row 4: a negative position
    c.computed[5] = 4 * c.table.shape[1] - 1   # row 0: its second token is past the table
    _check(c, 64, False, requests=req, want_err=api.ROW_BAD_BLOCK)
    c = Case([2, 3], [0, 4], 4, 2, 64, 4, seed=5)
    c.table[1, 1] = c.keys.shape[0]        # one past the cache
    c.table[0, 0] = -4                     # a null entry: nothing stored
    _check(c, 64, False, want_err=api.ROW_BAD_SLOT)


def test_tokens_outside_every_row_are_left_alone():
    c = Case([3, 2], [0, 1], 4, 2, 64, 8, seed=6)
    c.cu = torch.tensor([1, 3, 4], dtype=torch.int32, device="cuda")   # tokens 0 and 4 in no row
    _check(c, 64, True)
    c.cu = torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda")   # a negative count
    c.computed[:] = 0
    q = torch.full(c.q.shape, 7.0, dtype=c.dtype, device="cuda")
    api.kda_kv_append(c.q, c.k, c.v, c.keys, c.values, c.cu, c.table, c.computed, q_out=q,
                      error_word=c.err)
    torch.cuda.synchronize()
    assert torch.equal(q[:2], c.q[:2])     # row 0's tokens that the search finds


def test_empty_calls():
    c = Case([2], [0], 4, 2, 64, 8, seed=7)
    before = c.keys.clone()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kda_kv_append(c.q[:0], c.k[:0], c.v[:0], c.keys, c.values, c.cu * 0, c.table, c.computed)
    api.kda_kv_append(c.q, c.k, c.v, c.keys, c.values, none, c.table, c.computed)
    torch.cuda.synchronize()
    assert torch.equal(before, c.keys)


def test_rows_that_reach_past_the_tokens():
    c = Case([3, 2, 4], [0, 1, 7], 4, 2, 64, 8, seed=8)
    c.q, c.k, c.v = c.q[:8], c.k[:8], c.v[:8]     # the last row's last token is not there
    _check(c, 64, True, want_err=api.ROW_BAD_LENGTH)

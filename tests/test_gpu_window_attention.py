"""GPU: the window attention against the float64 oracle.

Bound of an output, with u half a step of the storage type, A = sum_j p_j
|v_j| and S the largest scale sum_i |q_i k_i|: a score is off by at most
(D + 4) 2^-24 S (fp32 products summed in any order), so a weight by twice
that and 2^-22 of the exponential, and by u where it is rounded for the
product with v; sums of n weights add n 2^-24, the pieces' scaling 2^-20 at
most; the result is rounded by u:
    |out - ref| <= u |ref| + (u + 2 e) A,  e = (D + 4) 2^-24 S + n 2^-24 + 2^-20
    |lse - ref| <= e + 2^-22 (1 + |ref|)."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import attention_oracle as A
from tests.attention_helpers import Case, f64, half_step, smallest_half

pytestmark = pytest.mark.gpu


def _run(c, window=8, left_window=0, requests=None, scale=None, workspace=None):
    req = None if requests is None else torch.tensor(requests, dtype=torch.int32, device="cuda")
    if workspace is None:
        workspace = api.allocate_attention_workspace(c.cu.numel() - 1, c.q_heads, c.kv_heads,
                                                     c.dim, "cuda", window=window)
        workspace.fill_(255)   # NaN patterns: nothing may be read before it is written
    out = torch.full((c.q.shape[0], c.q_heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    lse = torch.full(out.shape[:2], 7.0, device="cuda")
    api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed, workspace,
                             window=window, left_window=left_window, scale=scale,
                             request_indices=req, out=out, lse=lse, error_word=c.err)
    torch.cuda.synchronize()
    return out, lse


def _check(c, window=8, left_window=0, requests=None, scale=None, want_err=0):
    cu, table, computed = c.meta()
    s = c.dim ** -0.5 if scale is None else scale
    out, lse = _run(c, window, left_window, requests, scale)
    want, want_lse, weight, spread, _ = A.attend(f64(c.q), f64(c.keys), f64(c.values), cu, table,
                                                 computed, np.float32(s), window, left_window,
                                                 requests)
    assert int(c.err.item()) == want_err
    skipped = np.isnan(want_lse)
    got, got_lse = f64(out), f64(lse)
    assert np.all(got[skipped] == 7.0) and np.all(got_lse[skipped] == 7.0)
    got, got_lse = got[~skipped], got_lse[~skipped]
    want, want_lse, weight, spread = (x[~skipped] for x in (want, want_lse, weight, spread))
    u = half_step(c.dtype)
    n = int(computed.max() + 8) if len(computed) else 0
    e = (c.dim + 4) * 2.0 ** -24 * spread + n * 2.0 ** -24 + 2.0 ** -20
    bound = u * np.abs(want) + (u + 2 * e[..., None]) * weight + smallest_half(c.dtype)
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())
    empty = want_lse == -np.inf
    assert np.all(got_lse[empty] == -np.inf) and np.all(got[empty] == 0.0)
    d = np.abs(got_lse[~empty] - want_lse[~empty])
    assert np.all(d <= e[~empty] + 2.0 ** -22 * (1 + np.abs(want_lse[~empty]))), float(d.max())
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,group", [(1, 1), (1, 7), (3, 5), (4, 4), (8, 3), (8, 8), (7, 9),
                                          (8, 16)])
def test_windows_and_head_groups(dtype, dim, window, group):
    lens = [window, 1, 0, max(1, window - 1)]
    layout = {1: "tokens", 3: "heads"}.get(window, "pairs")
    c = Case(lens, [0, 63, 5, 200], 2 * group, 2, dim, 16, dtype, layout, seed=window * group)
    _check(c, window)


@pytest.mark.parametrize("block_size", [1, 3, 16, 24, 128, 1000])
@pytest.mark.parametrize("context", [0, 1, 62, 63, 64, 65, 127, 128, 129])
def test_block_sizes_and_lengths(block_size, context):
    c = Case([2, 1, 3], [context, context + 1, 0], 6, 3, 64, block_size, seed=context)
    _check(c, 3)


@pytest.mark.parametrize("dim,group,window", [(128, 4, 4), (64, 8, 8), (128, 8, 8), (128, 16, 8),
                                              (128, 1, 1)])
def test_long_rows_are_cut_and_joined(dim, group, window):
    # one to three rows: every segment is shared by many CTAs
    c = Case([window], [9000], group, 1, dim, 32, seed=group)
    _check(c, window)
    c = Case([window, 1, window], [5003, 2, 4100], 2 * group, 2, dim, 32, "fp16", seed=group + 1)
    _check(c, window)


@pytest.mark.parametrize("left_window", [1, 2, 5, 64, 100, 1000])
@pytest.mark.parametrize("group,window", [(2, 4), (8, 8), (16, 8)])
def test_sliding_windows(left_window, group, window):
    c = Case([window, 1, window, 2], [0, 300, 129, 700], 2 * group, 2, 64, 24, seed=left_window)
    _check(c, window, left_window)


def test_many_short_rows():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 5, size=700).tolist()
    computed = rng.integers(0, 90, size=700).tolist()
    c = Case(lens, computed, 4, 2, 64, 16, seed=8)
    _check(c, 4)


@pytest.mark.parametrize("group,window", [(2, 2), (8, 8), (16, 8)])
def test_null_blocks_hide_their_keys(group, window):
    c = Case([window, 2, 1, window], [100, 40, 30, 257], group * 2, 2, 128, 16, seed=9)
    c.table[0, 1:5] = 0            # a hole, as a sliding cache leaves it
    c.table[1, :] = 0              # nothing left: zeros and -inf
    c.table[2, :2] = -1            # only the last keys
    c.table[3, 16:] = 0            # the window's own keys gone, older ones stay
    # what null blocks and places past a row's end hold does not matter
    c.keys[0], c.values[0] = float("nan"), float("inf")
    _check(c, window)


def test_garbage_past_the_rows_end():
    for group, window in ((2, 3), (8, 8), (16, 8)):
        c = Case([window, 1], [70, 33], 2 * group, 2, 128, 16, seed=10)
        for b, n in ((0, 70 + window), (1, 34)):
            block, at = int(c.table[b, (n - 1) // 16]), (n - 1) % 16
            c.keys[block, at + 1:] = float("nan")
            c.values[block, at + 1:] = float("nan")
        _check(c, window)


@pytest.mark.parametrize("dim,group,window", [(64, 1, 4), (128, 2, 8), (128, 8, 8), (64, 16, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_key_or_value_reaches_only_who_sees_it(dim, group, window, bad):
    # token 2 of the window carries it: tokens 0 and 1 must not notice; with a
    # sliding window, an old key that only token 0 sees
    c = Case([window], [90], 2 * group, 2, dim, 16, seed=11)
    pos = 92
    block, at = int(c.table[0, pos // 16]), pos % 16
    old = c.values[block, at, 0, 3].clone()
    for cache, channel in ((c.values, slice(3, 4)), (c.keys, slice(0, dim))):
        saved = cache.clone()
        clean, clean_lse = _run(c, window)
        cache[block, at, 0, channel] = bad
        out, lse = _run(c, window)
        assert torch.equal(out[:2], clean[:2]) and torch.equal(lse[:2], clean_lse[:2])
        assert torch.equal(out[:, group:], clean[:, group:])     # the other kv head
        if cache is c.values:
            seen = out[2:, :group, 3]
            assert torch.isnan(seen).all() if bad != bad else (seen == bad).all()
            keep = [x for x in range(dim) if x != 3]
            assert torch.allclose(out[2:, :group][..., keep].float(),
                                  clean[2:, :group][..., keep].float(), atol=0, rtol=2 ** -7)
        cache.copy_(saved)
    assert torch.equal(c.values[block, at, 0, 3], old)
    left = 40
    pos = 90 + 1 - left                       # only token 0 sees it
    block, at = int(c.table[0, pos // 16]), pos % 16
    clean, _ = _run(c, window, left)
    c.values[block, at, 0, 5] = bad
    out, _ = _run(c, window, left)
    assert torch.equal(out[1:], clean[1:])
    assert not torch.isfinite(out[0, :group, 5]).any()


def test_scores_of_minus_infinity_and_large_scores():
    c = Case([1], [5], 1, 1, 64, 16, seed=12)
    c.q[0, 0] = 1.0
    block = int(c.table[0, 0])
    c.keys[block, :6, 0] = float("-inf")
    out, lse = _run(c, 1)
    assert torch.equal(out, torch.zeros_like(out)) and (lse == float("-inf")).all()
    # maxima that keep growing, far past what a stale maximum may lag
    c = Case([1, 3], [500, 300], 2, 1, 64, 16, seed=13)
    for b in range(2):
        for p in range(int(c.computed[b]) + 1):
            c.keys[int(c.table[b, p // 16]), p % 16, 0] = 0.02 * p
    c.q[...] = 1.0
    _check(c, 3)
    c.q[...] = -1.0
    _check(c, 3)
    _check(c, 3, scale=-0.25)
    _check(c, 3, scale=0.0)


def test_request_indices_and_bad_metadata():
    c = Case([2, 3, 1, 2, 2, 4], [5, 9, 0, 3, 1, 2], 4, 2, 64, 4, seed=14, extra_columns=0)
    req = [5, 0, 6, -1, 2, 1]              # rows 2 and 3: no such request
    c.computed[2] = -3                     # row 4: a negative position
    c.computed[5] = 4 * c.table.shape[1] - 1   # row 0: its second token is past the table
    _check(c, 3, requests=req, want_err=api.ROW_BAD_BLOCK | api.ROW_BAD_LENGTH)
    c = Case([2, 3], [9, 4], 4, 2, 64, 4, seed=15)
    c.table[0, 1] = c.keys.shape[0]        # one past the cache: its keys are masked
    c.table[1, 0] = 0x7fffffff
    _check(c, 4, want_err=api.ROW_BAD_SLOT)


def test_empty_calls_and_rows():
    c = Case([0, 0, 0], [4, 5, 6], 4, 2, 64, 8, seed=16)
    out, lse = _run(c)
    assert out.numel() == 0 and int(c.err.item()) == 0
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = api.allocate_attention_workspace(0, 4, 2, 64, "cuda")
    api.kda_window_attention(c.q, c.keys, c.values, none, c.table, c.computed, work)
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    # the cache's last blocks start past 2^31 elements
    blocks, bs, hk, d = 2200, 512, 16, 128
    dev = "cuda"
    keys = torch.empty((blocks, bs, hk, d), dtype=torch.bfloat16, device=dev)
    values = torch.empty_like(keys)
    assert (blocks - 2) * bs * hk * d > 2 ** 31
    c = Case([2, 1], [700, 3], hk, hk, d, bs, seed=17)
    moved = {}
    table = c.table.clone()
    for i, old in enumerate(sorted(set(c.table.flatten().tolist()) - {0})):
        moved[old] = blocks - 1 - i
        keys[blocks - 1 - i].copy_(c.keys[old])
        values[blocks - 1 - i].copy_(c.values[old])
        table[c.table == old] = blocks - 1 - i
    near, near_lse = _run(c, 2)
    c.keys, c.values, c.table = keys, values, table
    far, far_lse = _run(c, 2)
    assert torch.equal(near, far) and torch.equal(near_lse, far_lse)
    # and the append writes there
    got = api.kda_kv_append(c.q, c.k, c.v, keys, values, c.cu, table, c.computed)
    torch.cuda.synchronize()
    assert torch.equal(got, c.q)
    assert torch.equal(keys[int(table[0, 1]), 700 - 512], c.k[0])
    assert torch.equal(values[int(table[1, 0]), 3], c.v[2])


def test_same_bits_every_time_and_on_other_streams():
    c = Case([8, 3, 8, 1], [6000, 800, 2500, 77], 16, 2, 128, 32, seed=18)
    work = api.allocate_attention_workspace(4, 16, 2, 128, "cuda")
    first, first_lse = _run(c, workspace=work)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(stream):
            out, lse = _run(c, workspace=work)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


def test_capture_and_replay_with_changed_lengths():
    c = Case([4, 2], [900, 40], 8, 2, 128, 16, seed=19, extra_columns=4)
    work = api.allocate_attention_workspace(2, 8, 2, 128, "cuda", window=4)
    out = torch.empty((6, 8, 128), dtype=c.dtype, device="cuda")
    lse = torch.empty((6, 8), device="cuda")

    def call():
        api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed, work, window=4,
                                 out=out, lse=lse)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    # the lengths are read on the device, so a replay follows them
    for computed in ([900, 40], [3, 41], [871, 0]):
        c.computed.copy_(torch.tensor(computed, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        replayed, replayed_lse = out.clone(), lse.clone()
        want, want_lse = _run(c, 4)
        assert torch.equal(replayed, want) and torch.equal(replayed_lse, want_lse)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,window", [(1, 3), (6, 4), (8, 8), (16, 8)])
def test_growing_maxima_and_scales(dim, group, window):
    # maxima that keep growing along the keys, then shrinking ones
    c = Case([window, 1], [1500, 300], group, 1, dim, 16, seed=20)
    for b in range(2):
        for p in range(int(c.computed[b]) + 1):
            c.keys[int(c.table[b, p // 16]), p % 16, 0] += 0.02 * p
    c.q[...] = c.q.abs()
    for scale in (None, -0.05, 0.0, 1.0):
        _check(c, window, scale=scale)


@pytest.mark.parametrize("group,window", [(1, 1), (4, 4), (8, 8), (16, 8)])
def test_many_segments_of_every_length(group, window):
    # a CTA's run spans several rows and heads, short and long in turn
    rng = np.random.default_rng(5)
    lens = rng.integers(0, window + 1, size=90).tolist()
    computed = [int(x) for x in np.exp(rng.uniform(0, np.log(700), size=90))]
    c = Case(lens, computed, 3 * group, 3, 64, 16, seed=21)
    _check(c, window)
    _check(c, window, left_window=37)


@pytest.mark.parametrize("group,window", [(1, 4), (12, 4)])
def test_rows_that_reach_past_the_tokens(group, window):
    c = Case([window, 2, 3], [20, 5, 70], 2 * group, 2, 128, 16, seed=22)
    total = c.q.shape[0]
    c.q = c.q[:total - 1]          # the last row's last token is not there
    _check(c, window, want_err=api.ROW_BAD_LENGTH)
    c = Case([window, 2, 3], [20, 5, 70], 2 * group, 2, 128, 16, seed=22)
    c.cu[0] = -1                   # a row that starts before the first token
    _check(c, window, want_err=api.ROW_BAD_LENGTH)


@pytest.mark.parametrize("group,window", [(1, 1), (16, 4)])
def test_thousands_of_rows(group, window):
    rng = np.random.default_rng(9)
    lens = rng.integers(0, window + 1, size=3000).tolist()
    computed = rng.integers(0, 20, size=3000).tolist()
    c = Case(lens, computed, group, 1, 64, 16, seed=23)
    _check(c, window)

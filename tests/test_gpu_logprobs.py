"""GPU: token log probabilities, entropy and alternatives against the float64
oracle.

Bound: a term 2^y is off by 2^-22 and by y's rounding, 2^-24 |y| (y is the
distance to the maximum in log2 units, so far terms weigh little: at most
2^-23 of the sum); a sum of n terms in at most n / 512 + 64 sequential steps
adds 2^-24 each; the logarithm and the conversions 2^-22 of |max| + |log s|.
So lse is off by at most e = 2^-21 (2 + |max| + log n) + (n / 512 + 64) 2^-23,
a log probability by that and its own rounding, and the entropy by e (2 + d)
with d the mean distance to the maximum."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import attention_oracle as A
from tests.attention_helpers import f64

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check(logits, tokens, top, want_err=0):
    dev = torch.device("cuda")
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    rows, vocab = logits.shape
    out = api.allocate_token_logprobs(rows, top, dev)
    for t in out:
        t.fill_(9)
    tok = torch.tensor(tokens, dtype=torch.int32, device=dev)
    api.kda_token_logprobs(logits, tok, num_top=top, out=out, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == want_err
    good = np.array([t < vocab for t in tokens])
    want = A.token_logprobs(f64(logits)[good], np.asarray(tokens)[good], top)
    lp, ent, lse, tv, ti = (f64(t) for t in out)
    for x in (lp, ent, lse, tv, ti):
        assert np.all(x[~good] == 9)
    lp, ent, lse, tv, ti = (x[good] for x in (lp, ent, lse, tv, ti))
    assert np.array_equal(ti.astype(np.int64), want[4])
    most = np.nan_to_num(np.where(np.isfinite(f64(logits)[good]), f64(logits)[good], 0)).max(1)
    e = 2.0 ** -21 * (2 + np.abs(most) + np.log(vocab)) + (vocab / 512 + 64) * 2.0 ** -23

    def near(x, ref, bound):
        assert np.array_equal(np.isnan(x), np.isnan(ref))
        assert np.array_equal(x[np.isinf(ref)], ref[np.isinf(ref)])
        ok = np.isfinite(ref)
        bound = np.broadcast_to(bound, ref.shape)
        assert np.all(np.abs(x[ok] - ref[ok]) <= bound[ok]), \
            float((np.abs(x[ok] - ref[ok]) / bound[ok]).max())
    near(lse, want[2], e)
    near(lp, want[0], e + 2.0 ** -23 * np.abs(np.nan_to_num(want[0], neginf=0.0)))
    near(ent, want[1], e * (2 + want[5]))
    near(tv, want[3], e[:, None] + 2.0 ** -23 * np.abs(np.nan_to_num(want[3], neginf=0.0)))
    return out


def _logits(rows, vocab, dtype, seed=0, pad=0, spread=2.5):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, vocab + pad), generator=gen) * spread).to(DTYPES[dtype]).cuda()
    return x[:, :vocab]


def _tokens(rows, vocab, seed=0):
    return np.random.default_rng(seed).integers(0, vocab, size=rows).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab,top", [(1, 1), (2, 0), (7, 7), (40, 32), (513, 5), (4096, 8),
                                       (5003, 1), (16384, 32), (40001, 20)])
def test_sizes_types_and_alternatives(dtype, vocab, top):
    # rows of an odd length start at every alignment
    _check(_logits(9, vocab, dtype, seed=vocab), _tokens(9, vocab), top)


@pytest.mark.parametrize("rows", [1, 2, 5, 20, 77, 160, 400])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_shared_by_clusters(rows, dtype):
    vocab = 70001
    _check(_logits(rows, vocab, dtype, seed=rows, pad=3), _tokens(rows, vocab), 8)
    _check(_logits(rows, vocab, dtype, seed=rows, pad=3), _tokens(rows, vocab), 0)


@pytest.mark.parametrize("vocab", [9, 1000, 66000])
def test_ties_masks_and_extremes(vocab):
    x = torch.zeros((13, vocab), dtype=torch.float32, device="cuda")
    at = torch.arange(vocab, device="cuda", dtype=torch.float32)
    x[0] = 0.0                                   # all equal
    x[1] = at                                    # ascending: every step has a new maximum
    x[2] = -at                                   # descending
    x[3] = float("-inf")                         # nothing left
    x[4] = float("-inf")
    x[4, vocab // 2] = 3.0                       # one left
    x[5] = float("-inf")
    x[5, vocab - 3:] = torch.tensor([1.0, 2.0, 2.0])
    x[6, vocab - 1] = float("nan")
    x[7, 0] = float("inf")
    x[8] = -3.4e38                               # the type's lowest value
    x[9] = at % 3                                # ties everywhere
    x[10] = -3.4e38
    x[10, 1] = 80.0
    x[11] = torch.where(at % 2 == 0, 0.0, -0.0)  # the two zeros are equal
    x[12] = float("-inf")
    x[12, 4] = float("nan")
    tokens = [vocab - 1, 0, 1, 2, vocab // 2, vocab - 1, 0, 0, 0, 1, 1, 3, 4]
    _check(x, tokens, min(8, vocab))
    if vocab < 2000:
        _check(x[:, :vocab].clamp(min=-60000).half(), tokens, min(8, vocab))


def test_no_token_and_bad_tokens():
    x = _logits(6, 300, "bf16", seed=3)
    out = _check(x, [-1, 5, 300, 299, -7, 0], 4, want_err=api.ROW_BAD_TOKEN)
    assert float(out.logprob[0]) == 0.0 and float(out.logprob[4]) == 0.0
    x = _logits(2, 70000, "bf16", seed=3)       # a cluster leaves a bad row together
    _check(x, [70000, 3], 4, want_err=api.ROW_BAD_TOKEN)


def test_strided_rows_shared_rows_and_no_rows():
    x = _logits(4, 1000, "fp16", seed=5, pad=24)
    _check(x, _tokens(4, 1000), 3)
    _check(x[:1].expand(4, 1000), _tokens(4, 1000), 3)   # a row stride of 0
    dev = torch.device("cuda")
    got = api.kda_token_logprobs(x[:0], torch.zeros(0, dtype=torch.int32, device=dev), num_top=3)
    torch.cuda.synchronize()
    assert got.top_index.shape == (0, 3)


def test_same_bits_every_time():
    x = _logits(33, 50021, "bf16", seed=6)
    tok = torch.tensor(_tokens(33, 50021), dtype=torch.int32, device="cuda")
    first = api.kda_token_logprobs(x, tok, num_top=20)
    for _ in range(5):
        again = api.kda_token_logprobs(x, tok, num_top=20)
        assert all(torch.equal(a, b) for a, b in zip(first, again))

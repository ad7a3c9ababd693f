"""GPU: rows of 16-bit logits that are masked by the type's lowest value, alone
and mixed with -inf.  A -inf weighs nothing next to them.

Oracle and bounds as for the token log probabilities, |max| being that of the
largest finite logit; the entropy has no part that grows with the size of the
logits (they enter as distances from the maximum), so it is held to the bound
for a maximum of 0."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import attention_oracle as A
from tests.attention_helpers import f64
from tests.test_gpu_logprobs import DTYPES

pytestmark = pytest.mark.gpu


def _rows(vocab, dtype):
    low = torch.finfo(DTYPES[dtype]).min
    gen = torch.Generator().manual_seed(vocab)
    x = torch.full((8, vocab), low, dtype=torch.float64)
    x[1, torch.rand(vocab, generator=gen) < 0.5] = -np.inf
    x[1, vocab // 2] = low
    x[2] = -np.inf
    x[2, vocab - 1] = low                         # one that is not -inf
    x[3, : vocab // 3] = -np.inf
    x[4, vocab // 2] = 3.0                        # one that is not masked
    x[5] = -np.inf
    x[5, ::2] = low
    x[5, 1] = 0.5
    # values next to the lowest one, where distances are small in fp16
    x[6, torch.rand(vocab, generator=gen) < 0.3] = -np.inf
    x[6, ::5] = low * (1 - 2.0 ** -9)
    x[7] = torch.where(torch.rand(vocab, generator=gen, dtype=torch.float64) < 0.5, low * 0.999,
                       -np.inf)
    x[7, 0] = low * 0.998
    return x.to(DTYPES[dtype])


def _check(x, tokens, top, vocab):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.kda_token_logprobs(x, torch.tensor(tokens, dtype=torch.int32, device="cuda"),
                                 num_top=top, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    logits = f64(x)
    lp, ent, lse, tv, ti, mean = A.token_logprobs(logits[:8], tokens[:8], top)
    e0 = 2.0 ** -21 * (2 + np.log(vocab)) + (vocab / 512 + 64) * 2.0 ** -23
    e = e0 + 2.0 ** -21 * np.abs(np.where(np.isfinite(logits), logits, -np.inf).max(1))
    copies = len(tokens) // 8
    lp, ent, lse, mean = (np.tile(a, copies) for a in (lp, ent, lse, mean))
    tv, ti = (np.tile(a, (copies, 1)) for a in (tv, ti))
    assert np.array_equal(f64(got.top_index), ti)
    assert np.all(np.abs(f64(got.entropy) - ent) <= e0 * (2 + mean))
    for a, want, bound in ((got.lse, lse, e), (got.logprob, lp, e), (got.top_logprob, tv, e[:, None])):
        a = f64(a)
        gone = want == -np.inf
        assert np.array_equal(a == -np.inf, gone)
        want = np.where(gone, 0.0, want)
        assert np.all(np.abs(np.where(gone, 0.0, a) - want) <= bound + 2.0 ** -23 * np.abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [8, 9, 1000, 1003, 8192, 40001, 131072])
@pytest.mark.parametrize("copies", [1, 9])
def test_lowest_values_and_minus_infinity(dtype, vocab, copies):
    # 8 rows are shared by clusters of wide CTAs, 72 by clusters of narrow ones
    x = _rows(vocab, dtype).repeat(copies, 1).cuda()
    tokens = ([vocab - 1, vocab // 2, vocab - 1, vocab - 1, vocab // 2, 0, 0, 0] * copies)
    for top in (0, min(5, vocab)):
        _check(x, tokens, top, vocab)

"""GPU: alternatives of rows that several CTAs share, where the lists of each
are joined, and of rows whose largest logits lie together.  Oracle and bounds as
for the token log probabilities."""

import pytest
import torch

from tests.test_gpu_logprobs import _check, _logits, _tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 6, 39, 75, 150])
@pytest.mark.parametrize("top", [1, 8, 9, 17, 32])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lists_of_several_ctas(rows, top, dtype):
    # (bf16 logits tie, within and across the CTAs)
    vocab = 150001
    _check(_logits(rows, vocab, dtype, seed=top, pad=1), _tokens(rows, vocab), top)


@pytest.mark.parametrize("vocab", [3000, 150001])
@pytest.mark.parametrize("top", [2, 32])
def test_where_the_largest_lie(vocab, top):
    x = torch.randn((7, vocab), generator=torch.Generator().manual_seed(1)).cuda()
    x[0, :64] += 20.0                 # at the start
    x[1, -64:] += 20.0                # at the end
    x[2, ::vocab // 40] += 20.0       # everywhere
    x[3, 1000:1000 + 2 * top] = 9.0   # more equal ones than asked for
    x[4] = float("-inf")              # fewer than asked for
    x[4, vocab // 3: vocab // 3 + top // 2] = 1.0
    x[5, 5:900] = float("nan")
    x[6] = -3.4e38                    # masked by the type's lowest value
    x[6, vocab // 2: vocab // 2 + top + 3] = -1.0
    _check(x, _tokens(7, vocab), top)

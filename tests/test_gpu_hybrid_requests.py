"""GPU: requests of the hybrid example from their prompts on.  The same tokens
by admission, by plain decoding or by speculative steps lead to the same
states, caches and logits, up to the roundings on the way.

Bounds.  The KDA layer's inputs are the same bits on every way, so its states
are held to 2e-5 of a tile's largest value (1e-5 each way).  Its outputs are
bf16 and may differ by a step (2^-8), as may what is made of them: caches and
logits agree within 2^-5 of their norm, four products in bf16 behind them."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

I32 = torch.int32


@pytest.fixture(scope="module")
def hybrid():
    from examples import hybrid_requests
    return hybrid_requests


def _prompts(model, lens, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(0, model.sizes.vocab, (n,), generator=gen) for n in lens]


def _near(x, y):
    x, y = x.float(), y.float()
    assert (x - y).norm() <= 2.0 ** -5 * y.norm()


def _same_states(a, b):
    top = b.pool[1:].abs().amax(dim=(-1, -2), keepdim=True)
    assert ((a.pool - b.pool)[1:].abs() <= 2e-5 * top).all()


def test_admission_is_decoding_token_by_token(hybrid):
    sizes = hybrid.Sizes(requests=3)
    one, other = (hybrid.NormedHybridModel(sizes, seed=5) for _ in range(2))
    prompts = _prompts(one, [41, 41, 41])
    logits = one.admit(prompts)
    for t in range(41):
        last = other.decode(torch.stack([p[t] for p in prompts]).to(I32).cuda())
    _same_states(one, other)
    assert torch.equal(one.num_computed, other.num_computed)
    _near(one.key_cache, other.key_cache)
    _near(one.value_cache, other.value_cache)
    _near(logits, last)
    assert int(one.error_word.item()) == 0 and int(other.error_word.item()) == 0


def test_admission_is_accepting_every_window(hybrid):
    sizes = hybrid.Sizes(requests=2, window=8)
    one, other = (hybrid.NormedHybridModel(sizes, seed=6) for _ in range(2))
    prompts = _prompts(one, [32, 32], seed=1)
    one.admit(prompts)
    full = torch.full((2,), 8, dtype=I32, device="cuda")
    for t in range(0, 32, 8):
        other.verify(torch.stack([p[t:t + 8] for p in prompts]).to(I32).cuda())
        other_api = hybrid.api
        other_api.kda_commit(other.A_log, other.g_bias, other.pool, other.cu_seqlens, other.slots,
                             full, other.records, window=8, record_slots=2)
        other.num_computed += 8
    _same_states(one, other)
    _near(one.key_cache, other.key_cache)


def test_a_life_of_requests(hybrid):
    """Ragged prompts, plain tokens, then speculative steps whose drafts are the
    target's own choice and are accepted."""
    sizes = hybrid.Sizes(max_len=400)
    model = hybrid.NormedHybridModel(sizes, seed=7)
    last = model.admit(_prompts(model, (7, 130, 33, 1, 64), seed=2)).argmax(1).to(I32)
    for _ in range(3):
        last = model.decode(last).argmax(1).to(I32)
    before = model.num_computed.clone()
    tokens = torch.zeros((sizes.requests, sizes.window), dtype=I32, device="cuda")
    tokens[:, 0] = last
    for t in range(sizes.window - 1):
        choice = model.verify(tokens).top_index.view(sizes.requests, sizes.window)
        tokens[:, t + 1] = choice[:, t]
    accepted, _, seen = model.step(tokens)
    assert accepted.tolist() == [sizes.window] * sizes.requests
    assert torch.equal(model.num_computed, before + sizes.window)
    assert torch.isfinite(seen.lse).all() and int(model.error_word.item()) == 0


def test_the_example_runs(hybrid, capsys):
    hybrid.main()
    assert "decoded to [11, 134, 37, 5, 68]" in capsys.readouterr().out

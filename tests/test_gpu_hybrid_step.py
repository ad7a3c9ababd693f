"""GPU: the hybrid example runs its layers together as a serving loop would.

What a step computes at a position depends on the tokens up to it alone, bit
for bit, so drafts taken from the target's own choices are accepted, and
whatever lay in the cache behind the accepted tokens does not show."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hybrid():
    import sys
    spec = importlib.util.spec_from_file_location(
        "hybrid_step", os.path.join(ROOT, "examples", "hybrid_step.py"))
    module = importlib.util.module_from_spec(spec)
    sys.modules["hybrid_step"] = module
    spec.loader.exec_module(module)
    return module


def _window(model, first, gen):
    s = model.sizes
    tokens = torch.randint(0, s.vocab, (s.requests, s.window), generator=gen, device="cuda",
                           dtype=torch.int32)
    tokens[:, 0] = first
    return tokens


@pytest.mark.parametrize("window", [2, 4, 8])
def test_drafts_of_the_targets_choice_are_accepted(hybrid, window):
    model = hybrid.HybridModel(hybrid.Sizes(window=window), seed=window)
    s = model.sizes
    gen = torch.Generator(device="cuda").manual_seed(3)
    last = torch.arange(s.requests, dtype=torch.int32, device="cuda")
    for right in (0, window - 1, 1, window - 1, 0):
        tokens = _window(model, last, gen)
        for t in range(right):  # the choice at t does not depend on tokens behind it
            choice = model.verify(tokens).top_index.view(s.requests, window)
            tokens[:, t + 1] = choice[:, t]
        if right < window - 1:  # and the one behind them is wrong
            choice = model.verify(tokens).top_index.view(s.requests, window)
            tokens[:, right + 1] = (choice[:, right] + 1) % s.vocab
        before = model.num_computed.clone()
        accepted, last, seen = model.step(tokens)
        assert accepted.tolist() == [right + 1] * s.requests
        assert torch.equal(model.num_computed, before + right + 1)
        logprob = seen.logprob.view(s.requests, window)
        assert torch.equal(logprob[:, :right],
                           seen.top_logprob.view(s.requests, window)[:, :right])
        assert (logprob[:, -1] == 0).all() and (seen.entropy > 0).all()
    assert int(model.error_word.item()) == 0


def test_rejected_tokens_leave_no_trace(hybrid):
    # two histories with the same accepted tokens, one of them with windows of
    # rejected drafts between: the same state and the same view
    sizes = hybrid.Sizes(window=4)
    a, b = hybrid.HybridModel(sizes), hybrid.HybridModel(sizes)
    gen = torch.Generator(device="cuda").manual_seed(4)
    last = torch.arange(sizes.requests, dtype=torch.int32, device="cuda")
    for _ in range(6):
        tokens = _window(a, last, gen)
        choice = a.verify(tokens).top_index.view(sizes.requests, 4)
        tokens[:, 1] = (choice[:, 0] + 1) % sizes.vocab     # rejected
        other = _window(b, last, gen)
        other[:, 1] = (choice[:, 0] + 7) % sizes.vocab      # another rejected draft
        n_a, last, _ = a.step(tokens)
        n_b, last_b, _ = b.step(other)
        assert n_a.tolist() == n_b.tolist() == [1] * sizes.requests
        assert torch.equal(last, last_b)
        assert torch.equal(a.pool, b.pool)


def test_the_example_runs(hybrid, capsys):
    hybrid.main()
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 8 and all("accepted" in x for x in lines)

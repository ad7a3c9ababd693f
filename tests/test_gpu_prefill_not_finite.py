"""GPU: what is not finite in kda_prefill's inputs reaches no token before it,
and of a value's no other channel; gates may be infinite."""

import pytest
import torch

from tests.delta_bounds import hold
from tests.delta_helpers import Case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("tokens,at", [(40, 37), (40, 3), (616, 589), (5, 2)])
def test_what_is_not_finite_stays_behind_its_token(tokens, at, what):
    lens = [tokens, 600] if tokens > 6 else [tokens, 3, 4]
    clean_case = Case(lens, 2, seed=12)
    clean = run(clean_case).clone()
    for name in ("q", "k", "v", "g", "beta"):
        if what == what and name in ("g", "beta"):
            continue    # these have a limit
        c = Case(lens, 2, seed=12)
        x = getattr(c, name).clone()
        x[at, 0] = what
        setattr(c, name, x)
        got = run(c)
        same = got == clean
        assert same[:at].all() and same[tokens:].all() and same[:, 1].all(), name
        assert not got[at, 0].isfinite().any(), name
        behind = ~got[at + 1:tokens, 0].isfinite()
        assert same[at + 1:tokens, 0].all() if name == "q" else behind.all(), name
        state, want = c.pool[c.slots.long()], clean_case.pool[c.slots.long()]
        assert torch.equal(state[1:], want[1:]) and torch.equal(state[0, 1], want[0, 1])
        if name == "q":
            assert torch.equal(state, want)
        else:
            assert not state[0, 0].isfinite().any(), name


@pytest.mark.parametrize("tokens", [40, 616])
def test_a_value_that_is_not_finite_stays_in_its_channel(tokens):
    lens = [tokens, 30]
    clean_case = Case(lens, 2, seed=13)
    clean = run(clean_case).clone()
    for what in (float("nan"), float("inf")):
        c = Case(lens, 2, seed=13)
        c.v = c.v.clone()
        c.v[21, 1, 77] = what
        got = run(c)
        others = torch.ones_like(got, dtype=torch.bool)
        others[21:tokens, 1, 77] = False
        assert torch.equal(got[others], clean[others])
        assert not got[~others].isfinite().any()
        state, want = c.pool[c.slots.long()], clean_case.pool[c.slots.long()]
        others = torch.ones_like(state, dtype=torch.bool)
        others[0, 1, 77] = False
        assert torch.equal(state[others], want[others])
        assert not state[~others].isfinite().any()


@pytest.mark.parametrize("tokens", [5, 40, 616])
def test_gates_without_a_limit(tokens):
    c = Case([tokens], 2, seed=14)
    c.g, c.beta = c.g.clone(), c.beta.clone()
    c.g[3, 0], c.g[4, 1, ::2] = float("inf"), float("-inf")
    c.beta[2, 0], c.beta[2, 1] = float("inf"), float("-inf")
    hold(c)

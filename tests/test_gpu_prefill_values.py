"""GPU: what kda_prefill writes to a state is as exact beside itself, however
weakly its tokens write and however large the values beside them are (bounds in
delta_bounds)."""

import pytest
import torch

from tests.delta_bounds import decays_of, hold
from tests.delta_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [40, 64, 600])
@pytest.mark.parametrize("raw", [-8.0, -12.0, -16.0, -24.0, -40.0])
def test_weakly_written_rows(raw, tokens):
    c = Case([tokens], 2, seed=5)
    c.beta = torch.full_like(c.beta, raw)
    hold(c, initial=torch.zeros_like(c.slots))
    c = Case([tokens], 2, seed=6, size=1e-3 * 2.0 ** raw)
    c.beta = torch.full_like(c.beta, raw)
    hold(c)


def test_tokens_written_weakly_and_strongly():
    c = Case([100, 17], 2, seed=7)
    c.beta = torch.full_like(c.beta, -20.0)
    c.beta[3::7] = 1.0
    hold(c, initial=torch.zeros_like(c.slots))


@pytest.mark.parametrize("lens", [[16], [16] * 100])
@pytest.mark.parametrize("size", [1e4, 1e8])
@pytest.mark.parametrize("at", [0, 3, 9])
def test_a_large_value_that_decays_away_within_a_few_tokens(lens, at, size):
    c = Case(lens, 2, seed=11)
    decays_of(c, 20.0)
    c.v = c.v.clone()
    c.v[at::16] *= size
    hold(c)

"""GPU: what kda_prefill leaves of a state is as exact where little is left
(bounds in delta_bounds)."""

import pytest
import torch

from tests.delta_bounds import decays_of, hold
from tests.delta_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("each", [0.02, 0.3, 0.5, 0.8, 1.5])
@pytest.mark.parametrize("tokens,heads", [(64, 2), (600, 2), (23, 200)])
def test_what_decays_and_is_not_written_to(tokens, heads, each):
    c = Case([tokens], heads, seed=1, size=1.0)
    each = min(each, 60 / tokens)
    decays_of(c, each)
    c.beta = torch.full_like(c.beta, -1e30)
    hold(c, outputs=False, total=each * tokens)


@pytest.mark.parametrize("each", [0.5, 0.7, 1.0])
def test_a_large_state_that_decays_while_it_is_written_to(each):
    c = Case([16, 70, 33], 2, seed=2, size=100.0)
    decays_of(c, each)
    c.beta = torch.zeros_like(c.beta)
    hold(c)

"""GPU: kda_prefill's outputs are rounded once, to bf16 (bounds in
delta_bounds)."""

import pytest
import torch

from tests.delta_bounds import hold
from tests.delta_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lower_bound", [None, -5.0])
@pytest.mark.parametrize("memory", ["long", "short"])
@pytest.mark.parametrize("lens,heads", [([1, 16, 17, 100], 2), ([600], 2), ([40] * 60, 3),
                                        ([40] * 60 + [300], 3)])
def test_outputs_are_rounded_once(lens, heads, memory, lower_bound):
    hold(Case(lens, heads, lower_bound, seed=3, memory=memory))


@pytest.mark.parametrize("tokens", [64, 600])
def test_outputs_of_keys_that_are_alike(tokens):
    c = Case([tokens], 2, seed=4)
    c.k = c.k[:1].expand_as(c.k).clone()
    c.beta = torch.full_like(c.beta, 4.0)
    hold(c)

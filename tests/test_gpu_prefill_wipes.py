"""GPU: states of kda_prefill behind decays that take most of them away are as
exact beside what is left (bounds in delta_bounds)."""

import pytest
import torch

from tests.delta_bounds import decays_of, hold
from tests.delta_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("each", [0.7, 2.0, 5.0, 20.0])
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8])
@pytest.mark.parametrize("lens,heads", [([18, 60, 130], 2), ([600], 2), ([40, 50] * 40, 2)])
def test_a_large_state_that_decays_away(lens, heads, size, each):
    c = Case(lens, heads, seed=8, size=size)
    decays_of(c, each)
    hold(c, outputs=False)


@pytest.mark.parametrize("size", [1e4, 1e6, 1e10])
def test_strong_gates_take_a_large_state_away(size):
    c = Case([60, 130], 2, seed=10, memory="short", size=size)
    c.bias += 6.0
    c.A_log += 3.0
    hold(c, outputs=False)


@pytest.mark.parametrize("at", [3, 18, 31])
@pytest.mark.parametrize("tokens", [35, 90, 530])
@pytest.mark.parametrize("size", [1e4, 1e8])
def test_a_large_value_that_decays_away(tokens, at, size):
    c = Case([tokens], 2, seed=11)
    c.v = c.v.clone()
    c.v[at] *= size
    decays_of(c, 20.0)
    hold(c, outputs=False)
    c = Case([tokens], 2, seed=12)     # taken by one token's gate
    c.v, c.g = c.v.clone(), c.g.clone()
    c.v[at] *= size
    c.bias[:], c.A_log[:] = -4.0, 0.0
    c.g[at + 2] = 32.0
    hold(c, outputs=False)


# The tokens' own products with a state that decays away, and their outputs.

@pytest.mark.parametrize("each", [0.3, 0.7, 2.0, 5.0, 20.0])
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8, 1e12])
@pytest.mark.parametrize("lens,heads", [([7], 2), ([18, 60, 130], 2), ([600], 2),
                                        ([10, 50] * 40, 2)])
def test_tokens_see_what_is_left_of_a_large_state(lens, heads, size, each):
    c = Case(lens, heads, seed=15, size=size)
    decays_of(c, each)
    hold(c)


@pytest.mark.parametrize("lens", [[9, 60], [530]])
def test_tokens_behind_strong_gates(lens):
    c = Case(lens, 2, seed=16, size=1e8)
    decays_of(c, 0.01)
    c.g = c.g.clone()
    c.g[3::11] = 30.0
    hold(c)


@pytest.mark.parametrize("size", [1e4, 1e6])
@pytest.mark.parametrize("lens", [[7, 90], [520]])
def test_a_large_state_that_decays_away_unevenly(lens, size):
    c = Case(lens, 2, seed=9, size=size)
    gen = torch.Generator().manual_seed(1)
    decays_of(c, 0.3 * 100.0 ** torch.rand(len(c.bias), generator=gen, dtype=torch.float64))
    hold(c)


@pytest.mark.parametrize("at", [3, 18, 31])
@pytest.mark.parametrize("tokens", [35, 90, 530])
@pytest.mark.parametrize("size", [1e4, 1e8])
def test_tokens_behind_a_large_value_that_decays_away(tokens, at, size):
    c = Case([tokens], 2, seed=11)
    c.v = c.v.clone()
    c.v[at] *= size
    decays_of(c, 20.0)
    hold(c)
    c = Case([tokens], 2, seed=12)
    c.v, c.g = c.v.clone(), c.g.clone()
    c.v[at] *= size
    c.bias[:], c.A_log[:] = -4.0, 0.0
    c.g[at + 2] = 32.0
    hold(c)


@pytest.mark.parametrize("each", [30.0, 41.0])
@pytest.mark.parametrize("at", [0, 1, 2, 6])
@pytest.mark.parametrize("lens", [[8, 16], [10] * 90, [520]])
def test_a_huge_value_that_one_token_takes_away(lens, at, each):
    """e^-30 is 2^-43 and e^-41 2^-59: below what is told apart from nothing."""
    c = Case(lens, 2, seed=17)
    c.v = c.v.clone()
    c.v[at::23] *= 1e12
    decays_of(c, each)
    hold(c, largest=float(c.v.float().abs().max()))


@pytest.mark.parametrize("size", [1e4, 1e8])
@pytest.mark.parametrize("lens", [[5, 12], [40] * 80, [300]])
def test_channels_that_decay_apart(lens, size):
    """Large channels that are gone at once, beside small ones that stay."""
    c = Case(lens, 2, seed=18, size=1.0)
    c.pool[..., :64] *= size
    each = torch.full((256,), 0.01, dtype=torch.float64)
    each.view(2, 128)[:, :64] = 40.0
    decays_of(c, each)
    hold(c, taken=float(c.pool.abs().max()))

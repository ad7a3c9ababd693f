"""GPU: kda_decode against the float64 oracle (bounds in delta_helpers)."""

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from tests.delta_helpers import Case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lower_bound", [None, -5.0])
@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 32), (7, 3), (65, 4)])
def test_single_tokens(rows, heads, lower_bound):
    check(Case([1] * rows, heads, lower_bound, seed=rows), decode=True)


def test_from_other_slots_and_from_nothing():
    c = Case([1] * 9, 2, seed=1)
    mixed = c.sources.clone()
    mixed[::3] = 0
    check(c, initial=mixed, decode=True)


def test_padding_and_bad_rows():
    c = Case([1] * 6, 2, seed=2)
    c.slots[1], c.slots[4] = 0, -1
    check(c, decode=True)
    c = Case([1] * 6, 2, seed=3)
    c.slots[2] = c.pool.shape[0]
    check(c, decode=True, want_err=api.ROW_BAD_SLOT)
    c = Case([1] * 6, 2, seed=3)
    sources = c.sources.clone()
    sources[5] = 2 ** 31 - 1
    check(c, initial=sources, decode=True, want_err=api.ROW_BAD_SLOT)


def test_a_chain_of_tokens_is_the_prompt():
    c = Case([60], 3, seed=4)
    d = Case([60], 3, seed=4)
    whole = run(c).float()
    outs = []
    for t in range(60):
        at = slice(t, t + 1)
        outs.append(api.kda_decode(d.q[at], d.k[at], d.v[at], d.g[at], d.beta[at], d.A_log, d.bias,
                                   d.pool, d.slots))
    slot = c.slots.long()
    top = c.pool[slot].abs().amax(dim=(-1, -2), keepdim=True)
    assert ((d.pool - c.pool)[slot].abs() <= 2e-5 * top).all()
    assert (torch.cat(outs).float() - whole).norm() <= 2.0 ** -7 * whole.norm()


def test_a_token_behind_a_verified_window():
    """Decoding goes on from the state that a commit left."""
    c = Case([4], 2, seed=5)
    records = api.allocate_records(2, 4, 1, c.q.device)
    d = Case([4], 2, seed=5)
    out = torch.empty_like(d.q, memory_format=torch.contiguous_format)
    api.kda_verify(*d.inputs(), d.pool, d.cu, d.slots, records, out, window=4, record_slots=1)
    api.kda_commit(d.A_log, d.bias, d.pool, d.cu, d.slots,
                   torch.tensor([4], dtype=torch.int32, device="cuda"), records, window=4,
                   record_slots=1)
    for t in range(4):
        at = slice(t, t + 1)
        one = api.kda_decode(c.q[at], c.k[at], c.v[at], c.g[at], c.beta[at], c.A_log, c.bias,
                             c.pool, c.slots)
        assert (one.float() - out[at].float()).norm() <= 2.0 ** -7 * out[at].float().norm()
    slot = c.slots.long()
    top = c.pool[slot].abs().amax(dim=(-1, -2), keepdim=True)
    assert ((d.pool - c.pool)[slot].abs() <= 2e-5 * top).all()


def test_runs_are_alike():
    c = Case([1] * 33, 4, -5.0, seed=6)
    first = run(c, initial=c.sources, decode=True).clone()
    after = c.pool.clone()
    assert torch.equal(run(c, initial=c.sources, decode=True), first)
    assert torch.equal(c.pool, after)


def test_empty_call():
    c = Case([1], 1, seed=7)
    out = api.kda_decode(*(x[:0] for x in c.inputs()[:5]), c.A_log, c.bias, c.pool, c.slots[:0])
    assert out.shape == (0, 1, 128)

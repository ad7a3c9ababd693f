"""Seeded cases of kda_prefill and kda_decode for the tests, and the check of
their results against the float64 oracle.

Bounds.  An output is one rounding to bf16 of a sum whose operands may be
rounded to 11 bits on the way: the state and the decayed query, or the deltas
and the tokens' products, 2^-11 of each, so 2^-10 of what the sum is made of
(the oracle's sizes, times the scale; the factors beside them are at most 1).
States: 1e-5 of the tile's largest value, the library's stated tolerance."""

from __future__ import annotations

import numpy as np
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import delta_oracle as D
from tests.attention_helpers import f64

BF = torch.bfloat16


class Case:
    """Rows of lens[b] tokens (None: one each), from their own slots; q, k and
    v are views of one buffer, as beta_raw is of a wider one."""

    def __init__(self, lens, heads, lower_bound=None, seed=0, device="cuda", memory="long",
                 extra_slots=3, scale=None, pad_tokens=0, size=0.05):
        gen = torch.Generator().manual_seed(seed)
        rows = len(lens)
        total = int(sum(lens)) + pad_tokens

        def normal(*shape):
            return torch.randn(shape, generator=gen)
        merged = normal(total, 3, heads, 128).to(BF).to(device)
        self.q, self.k, self.v = merged[:, 0], merged[:, 1], merged[:, 2]
        self.g = normal(total, heads, 128).to(BF).to(device)
        self.beta = normal(total, heads + 4).to(BF).to(device)[:, :heads]
        self.A_log = (2.7 * torch.rand(heads, generator=gen)).to(device)
        bias = 0.1 * normal(heads * 128)
        if memory == "long":     # steps of 0.001 to 0.1: memories of up to some thousand tokens
            step = torch.exp(np.log(1e-3) + np.log(100.0) * torch.rand(heads * 128, generator=gen))
            bias = torch.log(torch.expm1(step))
        self.bias = bias.to(device)
        self.pool = (size * normal(2 * rows + extra_slots, heads, 128, 128)).to(device)
        order = (torch.randperm(2 * rows + extra_slots - 1, generator=gen) + 1).to(torch.int32)
        self.slots, self.sources = order[:rows].to(device), order[rows:2 * rows].to(device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32,
                               device=device)
        self.lower_bound, self.scale = lower_bound, scale
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def inputs(self):
        return (self.q, self.k, self.v, self.g, self.beta, self.A_log, self.bias)


def run(c, initial=None, decode=False, out=None, err=True):
    more = dict(lower_bound=c.lower_bound, scale=c.scale, initial_indices=initial, out=out,
                error_word=c.err if err else None)
    if decode:
        return api.kda_decode(*c.inputs(), c.pool, c.slots, **more)
    return api.kda_prefill(*c.inputs(), c.pool, c.cu, c.slots, **more)


def check(c, initial=None, decode=False, want_err=0):
    """Runs the case and holds it to the oracle; returns the outputs."""
    before = c.pool.clone()
    want, after, sizes, issues = D.run(
        f64(c.pool), *(f64(x) for x in c.inputs()), None if decode else f64(c.cu).astype(int),
        c.slots.cpu().numpy(), None if initial is None else initial.cpu().numpy(), c.lower_bound,
        c.scale)
    out = torch.full(c.q.shape, 7.0, dtype=BF, device=c.q.device)
    got = run(c, initial, decode, out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    assert int(c.err.item()) == want_err
    written = ~np.isnan(want)
    x = f64(got)
    assert np.all(x[~written] == 7.0)
    scale = abs(128 ** -0.5 if c.scale is None else c.scale)
    bound = 2.0 ** -8 * np.abs(want) * 1.001 + 2.0 ** -10 * scale * sizes + 1e-30
    off = np.where(written, np.abs(x - np.where(written, want, 0.0)) - bound, 0.0)
    assert not np.isnan(off).any() and off.max() <= 0.0, off.max()
    state = f64(c.pool)
    touched = np.zeros(len(state), dtype=bool)
    cu = f64(c.cu).astype(int)
    bad = {b for b, _ in issues}
    for b, slot in enumerate(c.slots.cpu().tolist()):
        if slot > 0 and b not in bad and (decode or cu[b + 1] > cu[b]):
            touched[slot] = True
    left = torch.from_numpy(~touched).to(c.pool.device)
    assert torch.equal(c.pool[left], before[left])
    for slot in np.nonzero(touched)[0]:
        for h in range(state.shape[1]):
            most = np.abs(after[slot, h]).max()
            worst = np.abs(state[slot, h] - after[slot, h]).max()
            assert worst <= 1e-5 * most, (slot, h, worst / most)
    return got

"""Checks of kda_prefill and kda_decode beside what each token leaves, and gates
of known strength.

Bounds.  States: 1e-5 of the tile's largest value, the library's stated
tolerance.  An output is a product of such a state with a query of norm 1, so
1e-5 sqrt(128) of the largest value of the tile behind its token, times the
scale, and one rounding to bf16, 2^-8 of the value.
  Where a row's state is only what its decays leave of the first one, as the tile's
largest value is then too, their errors add up: a token's logarithm has 2 ulp
(tests/test_softplus_poly.py), 2^-22 of it, so what exp(-total) leaves is off by
2^-22 total of itself (total 60: 1.4e-5).
  What decays leave below 2^-40 between two tokens may count as anything up to that
(include/kda.h): beside a value that is larger than the others by more than some
1e7 it shows.  A token's delta is then off by that of each of the 15 values before
it at most, and so are an entry of the state, which is a delta times at most 1, and
an output, in which the deltas before it count for as much again: 32 times 2^-40 of
the largest value bounds both.
  Sixteen tokens see a state's entries to within 2^-23 of the largest of their row
(include/kda.h): their deltas are off by sqrt(128) 2^-23 < 2^-19 of it at most, and
so a state's entry and an output by 16 times that where the decays have taken the
largest away."""

from __future__ import annotations

import numpy as np
import torch

from oracle import delta_oracle as D
from tests.attention_helpers import f64
from tests.delta_helpers import run


def hold(c, initial=None, outputs=True, total=0.0, largest=0.0, taken=0.0):
    """Runs the case and holds the rows' states, and their outputs, to the
    oracle.  total: of the logarithms of the decays, where they are all there is;
    largest: the largest value, where it shows; taken: the largest entry of a
    state of which other channels than its own are left."""
    close, faint = 1e-5 + 2.0 ** -22 * total, 32 * 2.0 ** -40 * largest + 2.0 ** -15 * taken
    start, inputs = f64(c.pool), [f64(x) for x in c.inputs()]
    got = f64(run(c, initial))
    assert int(c.err.item()) == 0
    state, cu = f64(c.pool), c.cu.tolist()
    scale = 128 ** -0.5 if c.scale is None else c.scale
    sources = c.slots if initial is None else initial
    for slot, source, first, end in zip(c.slots.tolist(), sources.tolist(), cu, cu[1:]):
        if first == end:   # writes nothing
            continue
        s = start[source] if source > 0 else np.zeros(start.shape[1:])
        for t, (out, s, _) in enumerate(D.tokens(
                s, *(x[first:end] for x in inputs[:5]), *inputs[5:], c.lower_bound, scale), first):
            more = abs(scale) * (close * 128 ** 0.5 * np.abs(s).max((1, 2))[:, None] + faint)
            off = np.abs(got[t] - out) / (2.0 ** -8 * (np.abs(out) + more) + more + 1e-38)
            assert not outputs or off.max() <= 1.0, (t - first, end - first, off.max())
        off = np.abs(state[slot] - s).max((1, 2)) / (close * np.abs(s).max((1, 2)) + faint + 1e-38)
        assert off.max() <= 1.0, (end - first, off.max())


def decays_of(c, each):
    """Each token takes exp(-each) of the state, of all channels or of each."""
    c.g = torch.zeros_like(c.g)
    c.A_log = torch.zeros_like(c.A_log)
    each = torch.as_tensor(each, dtype=torch.float64).expand(len(c.bias))
    c.bias = (each + torch.log(-torch.expm1(-each))).float().to(c.bias.device)   # softplus^-1

"""GPU: many keys far below one that leads, as where attention has a sink.
The leading key's value is 0, so the output is what the others add up to.

Bound: as for the window attention (relative to sum p |v|, which is the
others'), and for fp16 the step of its smallest numbers: weights are taken
relative to the largest one, times 2^7, so one of them is off by half of
2^-24 in units of 2^-7, and n of them by n 2^-32 of the largest |v| in all."""

import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from tests.attention_helpers import Case, f64, half_step, smallest_half
from tests.test_gpu_window_attention import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,group,window", [(128, 1, 1), (64, 2, 4), (128, 4, 8), (64, 8, 8),
                                              (128, 8, 8), (128, 16, 8), (64, 12, 8)])
@pytest.mark.parametrize("lead", [11.0, 15.0, 17.0])
@pytest.mark.parametrize("keys", [130, 9000])
def test_the_others_of_a_leading_key(dtype, dim, group, window, lead, keys):
    c = Case([window], [keys], group, 1, dim, 16, dtype, seed=int(lead))
    c.q[...] = 0
    c.q[..., 0] = 1.0                       # a score is the key's first channel
    where = int(c.table[0, 0]), 3           # the fourth key leads
    c.keys *= 0.25
    c.keys[where[0], where[1], 0, 0] = lead
    c.values[...] = 1.0 + 0.25 * c.values.clamp(-2, 2)
    c.values[where[0], where[1]] = 0
    out, lse = _run(c, window, scale=1.0)
    cu, table, computed = c.meta()
    want, want_lse, weight, spread, _ = A.attend(f64(c.q), f64(c.keys), f64(c.values), cu, table,
                                                 computed, 1.0, window)
    assert int(c.err.item()) == 0
    n, u = keys + window, half_step(c.dtype)
    e = (dim + 4) * 2.0 ** -24 * spread + n * 2.0 ** -24 + 2.0 ** -20
    bound = u * np.abs(want) + (u + 2 * e[..., None]) * weight + smallest_half(c.dtype)
    if dtype == "fp16":
        bound = bound + n * 2.0 ** -32 * 1.5
    got = f64(out)
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())
    d = np.abs(f64(lse) - want_lse)
    assert np.all(d <= e + 2.0 ** -22 * (1 + np.abs(want_lse))), float(d.max())


@pytest.mark.parametrize("dim,group,window", [(128, 1, 1), (64, 8, 8), (128, 8, 8), (128, 16, 8)])
def test_a_leader_that_comes_late_or_grows(dim, group, window):
    # the maximum lags by up to 2^8 before the sums are scaled to it: weights
    # stay inside fp16 all the same
    c = Case([window], [3000], group, 1, dim, 16, "fp16", seed=3)
    c.q[...] = 0
    c.q[..., 0] = 1.0
    for p in range(3000):
        c.keys[int(c.table[0, p // 16]), p % 16, 0, 0] = 0.085 * (p // 64) + (5.5 if p == 2990 else 0)
    out, lse = _run(c, window, scale=1.0)
    cu, table, computed = c.meta()
    want, want_lse, weight, spread, _ = A.attend(f64(c.q), f64(c.keys), f64(c.values), cu, table,
                                                 computed, 1.0, window)
    u, n = half_step(c.dtype), 3000 + window
    e = (dim + 4) * 2.0 ** -24 * spread + n * 2.0 ** -24 + 2.0 ** -20
    bound = (u * np.abs(want) + (u + 2 * e[..., None]) * weight + smallest_half(c.dtype)
             + n * 2.0 ** -32 * np.abs(f64(c.values)).max())
    assert np.all(np.abs(f64(out) - want) <= bound)
    assert np.all(np.abs(f64(lse) - want_lse) <= e + 2.0 ** -22 * (1 + np.abs(want_lse)))

"""CPU pins of the oracle of kda_prefill, kda_decode and the head norms."""

import numpy as np
import pytest
import torch

from oracle import delta_oracle as D
from oracle import kda_oracle as O


@pytest.mark.parametrize("lower_bound", [None, -5.0])
def test_a_row_is_the_window_oracles_token_loop(lower_bound):
    rng = np.random.default_rng(0)
    n, d = 8, 128
    q, k, v, g = (rng.standard_normal((n, 1, d)) for _ in range(4))
    beta, a_log, bias = rng.standard_normal((n, 1)), np.array([1.3]), 0.1 * rng.standard_normal(d)
    state = rng.standard_normal((1, d, d))
    out, after, _ = D.row(state, q, k, v, g, beta, a_log, bias, lower_bound)
    want = O.window(state[0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], a_log[0], bias, q=q[:, 0],
                    scale=d ** -0.5, bounded=lower_bound is not None,
                    lower_bound=lower_bound or 0.0)
    assert np.allclose(after[0], want[2], rtol=0, atol=1e-11)
    assert np.allclose(out[:, 0], want[0], rtol=0, atol=1e-11)


def test_pieces_of_a_row_are_the_row():
    rng = np.random.default_rng(1)
    n, h, d = 21, 2, 16
    q, k, v, g = (rng.standard_normal((n, h, d)) for _ in range(4))
    beta, a_log, bias = rng.standard_normal((n, h)), rng.random(h), rng.standard_normal(h * d)
    pool = rng.standard_normal((4, h, d, d))
    whole, after, _, issues = D.run(pool, q, k, v, g, beta, a_log, bias, [0, n], [2], [0])
    first, half, _, _ = D.run(pool, q, k, v, g, beta, a_log, bias, [0, 9], [3], [0])
    rest, end, _, _ = D.run(half, q, k, v, g, beta, a_log, bias, [9, n], [2], [3])
    assert not issues
    assert np.allclose(after[2], end[2], atol=1e-12)
    assert np.allclose(whole, np.where(np.isnan(first), rest, first), atol=1e-12)
    assert np.array_equal(after[[0, 1, 3]], pool[[0, 1, 3]])


def test_rows_that_are_skipped():
    rng = np.random.default_rng(2)
    n, h, d = 6, 1, 8
    x = [rng.standard_normal((n, h, d)) for _ in range(4)]
    rest = (rng.standard_normal((n, h)), rng.random(h), rng.standard_normal(h * d))
    pool = rng.standard_normal((5, h, d, d))
    out, after, _, issues = D.run(pool, *x, *rest, [0, 2, 2, 4, 3, 6], [0, 1, 9, 2, 3])
    assert issues == [(2, "slot"), (3, "length")]
    assert np.isnan(out[:3]).all() and not np.isnan(out[3:]).any()
    assert np.array_equal(after[[0, 1, 2, 4]], pool[[0, 1, 2, 4]])


def test_head_norm_is_the_root_mean_square_norm():
    x = torch.randn(3, 5, 64, dtype=torch.float64)
    w = torch.randn(64, dtype=torch.float64)
    want = torch.nn.functional.rms_norm(x, (64,), w, 1e-5)
    assert np.allclose(D.head_norm(x.numpy(), w.numpy(), 1e-5), want.numpy(), atol=1e-13)

"""CPU pins of the attention oracle: closed forms and hand-worked cases."""

import numpy as np
import pytest

from oracle import attention_oracle as A


def test_rotation_keeps_pair_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    freq = [1.0, 0.1]
    for inter in (False, True):
        def turn(x, p):
            return A.rotate(x, np.array([p]), freq, inter)
        assert np.allclose((turn(q, 5) ** 2).sum(), (q ** 2).sum())
        assert np.array_equal(turn(q, 5)[..., 4:], q[..., 4:])   # past rotary_dim = 4
        a = (turn(q, 9) * turn(k, 4)).sum()
        b = (turn(q, 105) * turn(k, 100)).sum()
        assert a == pytest.approx(b, abs=1e-12)                  # only the distance counts
    x = np.zeros((1, 1, 4))
    x[..., 0] = 1.0
    quarter = A.rotate(x, np.array([1]), [np.pi / 2], True)
    assert np.allclose(quarter[0, 0], [0, 1, 0, 0])


def test_attention_closed_forms():
    # equal keys: the mean of the values seen; a null block hides its keys
    keys = np.zeros((4, 2, 1, 4))
    values = np.arange(4 * 2 * 4, dtype=np.float64).reshape(4, 2, 1, 4)
    table = np.array([[1, 3, 2]])
    q = np.ones((2, 1, 4))
    out, lse, *_ = A.attend(q, keys, values, [0, 2], table, [3], 0.5)
    rows = np.concatenate([values[1, :, 0], values[3, :, 0], values[2, :, 0]])
    assert np.allclose(out[0, 0], rows[:4].mean(0)) and np.allclose(out[1, 0], rows[:5].mean(0))
    assert np.allclose(lse[:, 0], np.log([4, 5]))
    out, lse, *_ = A.attend(q, keys, values, [0, 2], table, [3], 0.5, left_window=2)
    assert np.allclose(out[1, 0], rows[3:5].mean(0))
    out, lse, *_ = A.attend(q, keys, values, [0, 2], np.array([[0, 0, 2]]), [3], 0.5)
    assert np.array_equal(out[0, 0], np.zeros(4)) and lse[0, 0] == -np.inf
    assert np.allclose(out[1, 0], values[2, 0, 0]) and lse[1, 0] == 0.0


def test_append_then_attend_one_key():
    rng = np.random.default_rng(1)
    keys, values = np.zeros((2, 4, 1, 8)), np.zeros((2, 4, 1, 8))
    k, v = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    q_out, touched, issues = A.append(k, k, v, keys, values, [0, 1], np.array([[1]]), [0], [0.3])
    assert issues == [] and touched.sum() == 1 and touched[1, 0]
    assert np.allclose(q_out, k)                                  # position 0 turns nothing
    out, lse, *_ = A.attend(q_out, keys, values, [0, 1], np.array([[1]]), [0], 1.0)
    assert np.allclose(out, v) and np.allclose(lse, (k * k).sum())


def test_bad_rows_are_named():
    table = np.ones((2, 2), dtype=int)
    args = (table.shape[1], 4, 2)
    assert A.plan_row([0, 0, 9], 1, [0, 0], *args, window=8) == "length"
    assert A.plan_row([0, 0, 8], 1, [0, 1], *args, window=8) == "block"   # past column 1
    assert A.plan_row([0, 0, 8], 1, [0, 0], *args, window=8) == (0, 8, 0, 1)
    assert A.plan_row([0, 0, 8], 0, [0, 0], *args) == ""
    assert A.plan_row([0, 1], 0, [-1, 0], *args) == "block"
    assert A.plan_row([0, 1], 0, [0, 0], *args, requests=[2]) == "block"


def test_logprobs_closed_forms():
    n = 10
    x = np.zeros((4, n))
    x[1, 3:] = -np.inf
    x[2] = -np.inf
    x[3, 4] = np.nan
    x[3, 7] = 2.0
    lp, ent, lse, tv, ti, _ = A.token_logprobs(x, [2, -1, 0, 7], 4)
    assert lp[0] == pytest.approx(-np.log(n)) and ent[0] == pytest.approx(np.log(n))
    assert list(ti[0]) == [0, 1, 2, 3]
    assert lp[1] == 0.0 and ent[1] == pytest.approx(np.log(3)) and list(ti[1]) == [0, 1, 2, 3]
    assert tv[1, 3] == -np.inf
    assert lse[2] == -np.inf and lp[2] == -np.inf and ent[2] == 0.0
    assert np.isnan(lp[3]) and list(ti[3]) == [7, 0, 1, 2]

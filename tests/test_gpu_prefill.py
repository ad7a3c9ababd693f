"""GPU: kda_prefill against the float64 oracle (bounds in delta_helpers)."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from tests.delta_helpers import BF, Case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lower_bound", [None, -5.0])
@pytest.mark.parametrize("memory", ["long", "short"])
@pytest.mark.parametrize("lens", [[1], [16], [17], [64, 1, 0, 15], [33, 2, 48, 31, 130]])
def test_rows_of_any_length(lens, memory, lower_bound):
    check(Case(lens, 3, lower_bound, seed=len(lens), memory=memory))


@pytest.mark.parametrize("lens", [[1], [40, 3, 16], [100]])
def test_rows_from_nothing_and_from_other_slots(lens):
    c = Case(lens, 2, seed=5)
    check(c, initial=torch.zeros_like(c.slots))
    c = Case(lens, 2, seed=6)
    check(c, initial=c.sources)
    c = Case(lens, 2, seed=7)
    mixed = c.sources.clone()
    mixed[::2] = -1
    check(c, initial=mixed)


def test_rows_share_a_source_block():
    c = Case([20, 37, 5], 2, seed=8)
    check(c, initial=c.sources[:1].expand(3).contiguous())


def test_long_row():
    check(Case([1500, 700], 1, seed=9))


@pytest.mark.parametrize("lower_bound", [None, -5.0])
@pytest.mark.parametrize("memory", ["long", "short"])
@pytest.mark.parametrize("lens,heads", [([1500, 0, 17, 1, 1200], 3),   # two CTAs a row and head
                                        ([1025], 16), ([520, 500, 520], 16),
                                        ([520, 510], 26)])             # one, many of them
def test_long_rows(lens, heads, memory, lower_bound):
    c = Case(lens, heads, lower_bound, seed=24, memory=memory)
    check(c)
    mixed = c.sources.clone()
    mixed[1::2] = 0
    check(c, initial=mixed)
    c.slots[-1] = 0
    check(c)


def test_long_rows_are_the_short_ones_rows():
    """A row alone and among many short ones: the same states and outputs, to
    the order of the sums over the values' tokens."""
    c = Case([700] + [1] * 60, 2, seed=25)
    want = run(c)
    d = Case([700] + [1] * 60, 2, seed=25)
    got = api.kda_prefill(*(x[:700] for x in d.inputs()[:5]), d.A_log, d.bias, d.pool,
                          d.cu[:2], d.slots[:1])
    slot = int(c.slots[0])
    top = c.pool[slot].abs().amax(dim=(-1, -2), keepdim=True)
    assert ((d.pool[slot] - c.pool[slot]).abs() <= 2e-5 * top).all()
    assert (got.float() - want[:700].float()).norm() <= 2.0 ** -7 * got.float().norm()


def test_many_rows():
    rng = np.random.default_rng(0)
    check(Case(rng.integers(0, 40, 170).tolist(), 2, -5.0, seed=10))


def uneven(rows, most, long, seed):
    """Rows of 0 to most tokens, and long ones among them."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most + 1, rows)
    lens[rng.choice(rows, len(long), replace=False)] = long
    return lens.tolist()


@pytest.mark.parametrize("lens,heads", [
    (uneven(40, 60, [1500], 0), 5), (uneven(300, 12, [900, 700, 17], 1), 3),
    (uneven(512, 20, [1, 2000, 2900], 2), 1), (uneven(513, 20, [1, 2000, 2900], 2), 1),
    (uneven(13, 250, [], 3), 16), ([700] + [9] * 160, 7), ([9] * 160 + [700], 7), ([40] * 62, 5),
    (uneven(460, 12, [], 4), 3), ([8, 9, 10, 11, 12] * 92, 3)])
def test_uneven_rows(lens, heads):
    """More rows and heads than SMs, dealt out by their lengths."""
    c = Case(lens, heads, seed=26)
    c.slots[3::7] = 0
    check(c, initial=c.sources)
    c = Case(lens, heads, -5.0, seed=27, pad_tokens=5)
    c.slots[5] = c.pool.shape[0]
    check(c, want_err=api.ROW_BAD_SLOT)


def test_captured_and_replayed_with_other_lengths():
    lens = uneven(60, 60, [1400], 5)
    c = Case(lens, 4, seed=28)
    start, order = c.pool.clone(), np.random.default_rng(6).permutation(60)
    out = torch.zeros(c.q.shape, dtype=BF, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run(c, out=out)
        with torch.cuda.graph(graph, stream=stream):
            run(c, out=out)
    stream.synchronize()
    for some in (np.array(lens)[order], np.array(lens)):
        c.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(some)])))
        c.pool.copy_(start)
        want = run(c).clone()
        after = c.pool.clone()
        c.pool.copy_(start)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.pool, after)


@pytest.mark.parametrize("heads", [1, 5, 40])
def test_heads(heads):
    check(Case([50, 18], heads, seed=heads))


def test_scale():
    check(Case([50, 18], 2, seed=1, scale=3.0))
    check(Case([50, 18], 2, seed=1, scale=-0.01))


def test_pieces_are_the_whole():
    """A row in pieces passes through the same states, within their bound."""
    c = Case([300], 2, seed=11)
    whole = check(c).clone()
    d = Case([300], 2, seed=11)
    outs = []
    for a, b in ((0, 37), (37, 38), (38, 166), (166, 300)):
        at = slice(a, b)
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        outs.append(api.kda_prefill(d.q[at], d.k[at], d.v[at], d.g[at], d.beta[at], d.A_log,
                                    d.bias, d.pool, cu, d.slots))
    got = torch.cat(outs).float()
    top = c.pool[c.slots.long()].abs().amax(dim=(-1, -2), keepdim=True)
    assert ((d.pool - c.pool)[c.slots.long()].abs() <= 2e-5 * top).all()
    assert (got - whole.float()).norm() <= 2.0 ** -7 * whole.float().norm()


def test_large_and_small_values():
    """Values of any size: the states are as exact beside their own largest."""
    for size in (1e-20, 1e-3, 1e4, 1e18):
        c = Case([70, 20], 2, seed=12, size=0.05 * size)
        c.v = (c.v.float() * size).to(BF)
        check(c)
    # a state far larger than what comes, and the other way round
    for size in (1e3, 1e-6):
        check(Case([70, 20], 2, seed=13, size=size))


def test_strong_decay_wipes_the_state():
    c = Case([90], 2, seed=14, memory="short")
    c.bias += 6.0
    c.A_log += 3.0
    check(c)


def test_repeated_keys():
    """Keys that are all alike, or alternate: the products between tokens are
    as large as they get."""
    for sign in (1, -1):
        c = Case([64, 30], 2, seed=15)
        k = c.k[:1].clone().expand(94, 2, 128).clone()
        k[1::2] *= sign
        c.k = k
        c.beta = torch.full_like(c.beta, 6.0)
        check(c)


def test_zero_queries_keys_and_gates_of_infinite_strength():
    c = Case([40], 2, seed=16)
    c.q, c.k = c.q.clone(), c.k.clone()
    c.q[7], c.k[9], c.k[10] = 0, 0, 0
    c.g = c.g.clone()
    c.g[20, :, ::3] = 3e38        # decays to nothing
    c.g[21, :, 1::3] = -3e38      # does not decay
    c.beta = c.beta.clone()
    c.beta[5], c.beta[6] = 3e38, -3e38
    check(c)


def test_activations_on_eight_bytes():
    c = Case([33, 20], 3, seed=17)
    wide = torch.zeros((53, 3 * 128 * 4 + 4), dtype=BF, device="cuda")

    def moved(x, i):
        part = wide[:, 4 + i * 384:4 + (i + 1) * 384]
        part.copy_(x.reshape(53, 384))
        return part.view(53, 3, 128)
    c.q, c.k, c.v, c.g = (moved(x, i) for i, x in enumerate((c.q, c.k, c.v, c.g)))
    assert c.q.data_ptr() % 16 == 8
    check(c)


def test_rows_that_are_skipped():
    c = Case([20, 5, 7, 9], 2, seed=18, pad_tokens=6)
    c.slots[1], c.slots[2] = 0, -3
    check(c)
    c = Case([20, 5, 7, 9], 2, seed=19)
    c.slots[1] = c.pool.shape[0]
    check(c, want_err=api.ROW_BAD_SLOT)
    c = Case([20, 5, 7, 9], 2, seed=19)
    sources = c.sources.clone()
    sources[3] = c.pool.shape[0] + 5
    check(c, initial=sources, want_err=api.ROW_BAD_SLOT)
    c = Case([20, 5, 7, 9], 2, seed=20)
    c.cu[4] += 1                                   # past the tokens
    check(c, want_err=api.ROW_BAD_LENGTH)
    c = Case([20, 5, 7, 9], 2, seed=20)
    c.cu[0] = -1
    check(c, want_err=api.ROW_BAD_LENGTH)
    c = Case([20, 5, 7, 9], 2, seed=20)
    c.cu[2] = 3                                    # a negative count, and rows 0 and 2 overlap
    c.slots[0] = c.slots[2] = 0
    check(c, want_err=api.ROW_BAD_LENGTH)


@pytest.mark.parametrize("tokens", [40, 616])
def test_what_is_not_a_number_stays_in_its_row_and_behind_its_token(tokens):
    c = Case([tokens, 600], 2, seed=21)
    clean = run(c).clone()
    for name in ("q", "k", "v", "g", "beta"):
        d = Case([tokens, 600], 2, seed=21)
        x = getattr(d, name).clone()
        x[37, 0] = float("nan")
        setattr(d, name, x)
        got = run(d)
        # head 0 of the first row, from the piece of 16 tokens on that holds it
        assert torch.equal(got[:32], clean[:32]) and torch.equal(got[tokens:], clean[tokens:])
        assert torch.equal(got[:, 1], clean[:, 1])
        assert got[37, 0].isnan().any()


def test_empty_calls():
    c = Case([4], 1, seed=22)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.kda_prefill(*c.inputs(), c.pool, zero, none)
    assert out.shape == c.q.shape
    out = api.kda_prefill(*(x[:0] for x in c.inputs()[:5]), c.A_log, c.bias, c.pool,
                          torch.zeros(2, dtype=torch.int32, device="cuda"), c.slots)
    assert out.shape == (0, 1, 128)


@pytest.mark.parametrize("lens", [[70, 3, 33], [1200, 100, 530]])
def test_runs_are_alike_and_captured(lens):
    c = Case(lens, 4, -5.0, seed=23)
    first = run(c, initial=c.sources).clone()
    after = c.pool.clone()
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run(c, initial=c.sources, out=out)
        with torch.cuda.graph(graph, stream=stream):
            run(c, initial=c.sources, out=out)
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(c.pool, after)

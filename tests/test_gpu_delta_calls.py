"""GPU: kda_prefill, kda_decode and kda_kv_norm_append as programs call them:
through the compiled part of the binding and without it, on several streams,
from several threads, in graphs beside eager calls, with offsets past 32 bits."""

import threading

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from tests.attention_helpers import Case as CacheCase
from tests.attention_helpers import frequencies
from tests.delta_helpers import BF, Case, run

pytestmark = pytest.mark.gpu


def _calls(c, a):
    freq = frequencies(128)
    weight = torch.linspace(0.5, 1.5, 128, device="cuda").to(a.dtype)
    return {
        "prefill": lambda **k: run(c, initial=c.sources, **k),
        "decode": lambda **k: api.kda_decode(*(x[:3] for x in c.inputs()[:5]), c.A_log, c.bias,
                                             c.pool, c.slots, initial_indices=c.sources,
                                             lower_bound=c.lower_bound, **k),
        "append": lambda **k: api.kda_kv_norm_append(
            a.q, a.k, a.v, a.keys, a.values, a.cu, a.table, a.computed, q_weight=weight,
            k_weight=weight, inv_freq=freq, **k),
    }


def _state(c, a):
    return [c.pool.clone(), a.keys.clone(), a.values.clone()]


@pytest.mark.parametrize("name", ["prefill", "decode", "append"])
def test_the_compiled_part_and_the_other_are_alike(name, monkeypatch):
    c, a = Case([30, 4, 19], 2, -5.0, seed=1), CacheCase([5, 9], [3, 40], 4, 2, 128, 16)
    call = _calls(c, a)[name]
    api.load_library()
    if api._quick_more is None:
        pytest.skip("the compiled part of the binding was not built")
    quick = call().clone()
    state = _state(c, a)
    with monkeypatch.context() as m:
        m.setattr(api, "_quick_more", None)
        slow = call()
    assert torch.equal(quick, slow)
    assert all(torch.equal(x, y) for x, y in zip(state, _state(c, a)))


def test_keyword_values_that_are_not_plain_floats():
    """Whole numbers and the like go the other way through the binding."""
    c = Case([30, 4], 2, -5.0, seed=2)
    want = run(c, initial=c.sources).clone()
    c.lower_bound = -5
    assert torch.equal(run(c, initial=c.sources), want)
    a = CacheCase([5, 9], [3, 40], 4, 2, 128, 16)
    one = api.kda_kv_norm_append(a.q, a.k, a.v, a.keys, a.values, a.cu, a.table, a.computed, eps=1.0)
    two = api.kda_kv_norm_append(a.q, a.k, a.v, a.keys, a.values, a.cu, a.table, a.computed, eps=1)
    assert torch.equal(one, two)


def test_two_streams_at_once():
    cases = [Case([400, 90, 33], 8, seed=3 + i) for i in range(2)]
    wants = [(run(c, initial=c.sources).clone(), c.pool.clone()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w) for w, _ in wants]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, o in zip(cases, streams, outs):
            with torch.cuda.stream(s):
                run(c, initial=c.sources, out=o)
                run(c, initial=c.sources, out=o)
    torch.cuda.synchronize()
    for c, o, (want, after) in zip(cases, outs, wants):
        assert torch.equal(o, want) and torch.equal(c.pool, after)


def test_threads_on_their_own_streams():
    cases = [Case([70, 3], 2, seed=10 + i) for i in range(4)]
    wants = [run(c, initial=c.sources).clone() for c in cases]
    got, failed = [None] * len(cases), []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = run(cases[i], initial=cases[i].sources)
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert all(torch.equal(g, w) for g, w in zip(got, wants))


def test_graph_replays_beside_eager_calls():
    c, a = Case([50, 4, 19], 3, seed=5), CacheCase([5, 9], [3, 40], 4, 2, 128, 16)
    calls = _calls(c, a)
    wants = {n: f().clone() for n, f in calls.items()}
    outs = {n: torch.zeros_like(w) for n, w in wants.items()}
    keys = {"prefill": "out", "decode": "out", "append": "q_out"}
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        for n, f in calls.items():
            f(**{keys[n]: outs[n]})
        with torch.cuda.graph(graph, stream=stream):
            for n, f in calls.items():
                f(**{keys[n]: outs[n]})
    for _ in range(3):
        for o in outs.values():
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, f in calls.items():
            assert torch.equal(outs[n], wants[n]), n
            assert torch.equal(f(), wants[n]), n


def test_offsets_past_32_bits():
    """Token strides and slots whose element offsets pass 2^32."""
    c = Case([40, 5], 1, seed=6)
    want = run(c, initial=c.sources).clone()
    after = c.pool.clone()
    tokens, step = 45, 100_000_000                    # 45 tokens, 9 GB
    wide = torch.empty((tokens - 1) * step + 4 * 128, dtype=BF, device="cuda")

    def moved(x, i):
        y = wide.as_strided(x.shape, (step, 128, 1), i * 128)
        y.copy_(x)
        return y
    d = Case([40, 5], 1, seed=6)
    d.q, d.k, d.v, d.g = (moved(x, i) for i, x in enumerate((d.q, d.k, d.v, d.g)))
    assert torch.equal(run(d, initial=d.sources), want)
    del wide, d.q, d.k, d.v, d.g
    slots = 300_000                                   # x 64 KiB: 20 GB
    pool = torch.empty((slots, 1, 128, 128), device="cuda")
    far = slots - 1 - torch.arange(2, dtype=torch.int32, device="cuda")
    pool[far.long()] = Case([40, 5], 1, seed=6).pool[c.sources.long()]
    out = api.kda_prefill(*c.inputs(), pool, c.cu, far)
    assert torch.equal(out, want)
    assert torch.equal(pool[far.long()], after[c.slots.long()])


def test_rows_behind_each_other_and_many_empty_ones():
    """Empty and skipped rows between the others change nothing."""
    c = Case([33, 0, 0, 17, 0, 64, 0], 2, seed=7)
    got = run(c, initial=c.sources).clone()
    lens, keep = [33, 17, 64], [0, 3, 5]
    cu = torch.tensor([0, 33, 50, 114], dtype=torch.int32, device="cuda")
    assert lens == (cu[1:] - cu[:-1]).tolist()
    pool = c.pool.clone()
    again = api.kda_prefill(*c.inputs(), c.pool, cu, c.slots[keep].contiguous(),
                            initial_indices=c.sources[keep].contiguous())
    assert torch.equal(got, again) and torch.equal(pool, c.pool)


def test_one_row_of_each_kind_of_length():
    """Few tokens a row go token by token, others in chunks: both ways agree
    where a batch is taken apart."""
    c = Case([1, 2, 6, 7, 5, 3], 2, seed=8)            # mean below 6: both forms
    whole = run(c, initial=c.sources).clone()
    states = c.pool.clone()
    cu = c.cu.tolist()
    for b, (i, j) in enumerate(zip(cu, cu[1:])):
        one = torch.tensor([0, j - i], dtype=torch.int32, device="cuda")
        out = api.kda_prefill(*(x[i:j] for x in c.inputs()[:5]), c.A_log, c.bias, c.pool, one,
                              c.slots[b:b + 1], initial_indices=c.sources[b:b + 1])
        assert torch.equal(out, whole[i:j])
    assert torch.equal(c.pool, states)

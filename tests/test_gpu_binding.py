"""GPU: the compiled part of the binding and api.py's own marshalling give the
same calls: the same bits from the same inputs, and the same refusals."""

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from tests.attention_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def both():
    api.load_library()
    saved = api._quick
    if saved is None:
        pytest.skip("the compiled part was not built")
    yield saved
    api._quick = saved


def _both_ways(call):
    quick = call()
    saved, api._quick = api._quick, None
    plain = call()
    api._quick = saved
    torch.cuda.synchronize()
    return quick, plain


def _requests(rows):
    return torch.arange(rows, dtype=torch.int32, device="cuda").flip(0)


@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16")])
def test_append_and_attention(dim, dtype):
    tokens = [2, 1, 3]
    c = Case(tokens, [40, 0, 100], 6, 2, dim, 16, seed=3)
    kind = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q, keys, values = c.q.to(kind), c.keys.to(kind), c.values.to(kind)
    k, v = (torch.randn((sum(tokens), 2, dim), device="cuda").to(kind) for _ in range(2))
    freq = 10000.0 ** -(torch.arange(16, dtype=torch.float64, device="cuda") / 16)
    work = api.allocate_attention_workspace(3, 6, 2, dim, "cuda")
    given = torch.zeros_like(q.contiguous())
    sums = torch.zeros(q.shape[:2], device="cuda")

    def append(**kw):
        kc, vc = keys.clone(), values.clone()
        out = api.kda_kv_append(kw.pop("q", q), k, v, kc, vc, c.cu, c.table, c.computed,
                                error_word=c.err, **kw)
        return (kc, vc) if out is None else (kc, vc, out.clone())

    def attend(**kw):
        return [t.clone() for t in api.kda_window_attention(
            q, keys, values, c.cu, c.table, c.computed, work, error_word=c.err, **kw)]

    for kw in (dict(), dict(inv_freq=freq), dict(inv_freq=freq, interleaved=True),
               dict(q_out=given), dict(q=None), dict(request_indices=_requests(3))):
        for a, b in zip(*_both_ways(lambda: append(**dict(kw)))):
            assert torch.equal(a, b), kw
    for kw in (dict(), dict(window=3), dict(scale=0.3), dict(scale=1), dict(left_window=9),
               dict(out=given, lse=sums), dict(request_indices=_requests(3))):
        for a, b in zip(*_both_ways(lambda: attend(**dict(kw)))):
            assert torch.equal(a, b), kw
    out, lse = api.kda_window_attention(q, keys, values, c.cu, c.table, c.computed, work,
                                        out=given, lse=sums)
    assert out is given and lse is sums
    assert api.kda_kv_append(q, k, v, keys, values, c.cu, c.table, c.computed,
                             q_out=given) is given


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_token_logprobs(dtype):
    x = torch.randn((5, 700), device="cuda").to(dtype)[:, 3:680]
    tokens = torch.tensor([1, 2, -1, 600, 676], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for top in (0, 1, 7):
        quick, plain = _both_ways(
            lambda: api.kda_token_logprobs(x, tokens, num_top=top, error_word=err))
        assert isinstance(quick, api.TokenLogprobs)
        for a, b in zip(quick, plain):
            assert torch.equal(a, b) and a.shape == b.shape and a.dtype == b.dtype


def test_refusals_are_the_same():
    c = Case([2, 1], [40, 3], 4, 2, 64, 16, seed=4)
    work = api.allocate_attention_workspace(2, 4, 2, 64, "cuda")
    base = dict(q=c.q, key_cache=c.keys, value_cache=c.values, cu_seqlens=c.cu,
                block_table=c.table, num_computed=c.computed, workspace=work)
    x, tokens = torch.zeros((3, 50), device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    calls = [lambda kw=kw: api.kda_window_attention(**dict(base, **kw)) for kw in (
        dict(q=c.q.float()), dict(q=c.q.cpu()), dict(q=c.q[:, :3]), dict(q=c.q[..., :32]),
        dict(value_cache=c.values[:1]), dict(cu_seqlens=c.cu.long()), dict(window=9),
        dict(window=0), dict(workspace=work[:64]), dict(workspace=work[1:]),
        dict(left_window=-1), dict(scale=float("nan")), dict(block_table=c.table[:1]),
        dict(lse=torch.zeros(3, device="cuda")), dict(error_word=torch.zeros(1, device="cuda")),
        dict(window=2 ** 40))]
    calls += [lambda: api.kda_token_logprobs(x, tokens, num_top=51),
              lambda: api.kda_token_logprobs(x, tokens, num_top=33),
              lambda: api.kda_token_logprobs(x, tokens.long()),
              lambda: api.kda_token_logprobs(x.t(), tokens),
              lambda: api.kda_token_logprobs(x.int(), tokens),
              lambda: api.kda_token_logprobs(x.cpu(), tokens.cpu()),
              lambda: api.kda_kv_append(c.q, c.q, c.q, c.keys, c.values, c.cu, c.table,
                                        c.computed),
              lambda: api.kda_kv_append(None, c.q[:, :2], c.q[:, :2], c.keys, c.values, c.cu,
                                        c.table, c.computed, q_out=c.q)]

    def kind(call):
        with pytest.raises(Exception) as e:
            call()
        return e.type, str(e.value)

    for i, call in enumerate(calls):
        quick, plain = _both_ways(lambda: kind(call))
        assert quick == plain, (i, quick, plain)


def test_threads_on_their_own_streams():
    # the calls let other threads run while they allocate and launch
    from concurrent.futures import ThreadPoolExecutor
    x = torch.randn((4, 6, 30000), device="cuda").bfloat16()
    tokens = torch.arange(6, dtype=torch.int32, device="cuda")
    want = [api.kda_token_logprobs(x[i], tokens, num_top=5) for i in range(4)]
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [api.kda_token_logprobs(x[i], tokens, num_top=5) for _ in range(50)]
        stream.synchronize()
        return got

    with ThreadPoolExecutor(4) as pool:
        for i, got in enumerate(pool.map(work, range(4))):
            for g in got:
                assert all(torch.equal(a, b) for a, b in zip(g, want[i]))

"""GPU: arguments of the attention layers' calls that both parts of the binding
have to take alike: a window that is left to the call, a truth value that
raises, strides of dimensions of one element, which mean nothing."""

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from tests.attention_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["compiled", "python"], autouse=True)
def part(request):
    api.load_library()
    saved = api._quick
    if request.param == "python":
        api._quick = None
    elif saved is None:
        pytest.skip("the compiled part was not built")
    yield request.param
    api._quick = saved


@pytest.mark.parametrize("group,most", [(2, 8), (16, 8), (20, 6), (64, 2), (128, 1)])
def test_the_window_that_the_head_counts_allow(group, most):
    c = Case([most, 1], [30, 5], group, 1, 64, 16, seed=group)
    work = api.allocate_attention_workspace(2, group, 1, 64, "cuda")
    out, lse = api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed, work,
                                        error_word=c.err)
    given, given_lse = api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed,
                                                work, window=most, error_word=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert torch.equal(out, given) and torch.equal(lse, given_lse)
    if most < 8:
        with pytest.raises(api.KDAError, match="UNSUPPORTED"):
            api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed, work,
                                     window=most + 1)


def test_too_many_heads_are_unsupported():
    c = Case([1], [5], 129, 1, 64, 16, seed=1)
    work = api.allocate_attention_workspace(1, 128, 1, 64, "cuda")
    with pytest.raises(api.KDAError, match="UNSUPPORTED"):
        api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed, work)


def test_a_truth_value_that_raises_launches_nothing():
    class Undecided:
        def __bool__(self):
            raise RuntimeError("undecided")
    c = Case([2], [3], 4, 2, 64, 16, seed=2)
    before = c.keys.clone()
    with pytest.raises(RuntimeError, match="undecided"):
        api.kda_kv_append(c.q, c.k, c.v, c.keys, c.values, c.cu, c.table, c.computed,
                          interleaved=Undecided())
    torch.cuda.synchronize()
    assert torch.equal(c.keys, before)


def _restrided(t, **strides):
    """t with other strides at dimensions of one element."""
    new = list(t.stride())
    for dim, stride in strides.items():
        assert t.shape[int(dim[1:])] == 1
        new[int(dim[1:])] = stride
    return t.as_strided(t.shape, new, t.storage_offset())


@pytest.mark.parametrize("stride", [0, 1, 4, 1 << 50])
def test_strides_of_one_head_and_one_token_blocks(stride):
    # as they come from another library's tensors, or from expand
    for block_size, dims in ((16, ("d2",)), (1, ("d1", "d2"))):
        c = Case([3, 1], [20, 9], 4, 1, 64, block_size, seed=3)
        work = api.allocate_attention_workspace(2, 4, 1, 64, "cuda")
        keys, values = c.keys.clone(), c.values.clone()
        q = api.kda_kv_append(c.q, c.k, c.v, keys, values, c.cu, c.table, c.computed)
        out, lse = api.kda_window_attention(q, keys, values, c.cu, c.table, c.computed, work)
        odd = [_restrided(c.keys, **{d: stride for d in dims}), c.values]
        api.kda_kv_append(c.q, c.k, c.v, *odd, c.cu, c.table, c.computed, error_word=c.err)
        got, got_lse = api.kda_window_attention(q, *odd, c.cu, c.table, c.computed, work,
                                                error_word=c.err)
        torch.cuda.synchronize()
        assert int(c.err.item()) == 0
        assert torch.equal(c.keys, keys) and torch.equal(c.values, values)
        assert torch.equal(got, out) and torch.equal(got_lse, lse)


def test_strides_of_a_cache_of_one_block():
    # (the null block alone: nothing is stored, nothing is seen)
    keys = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    odd = _restrided(keys, d0=3)
    c = Case([2], [0], 4, 2, 64, 16, seed=4)
    c.table.zero_()
    work = api.allocate_attention_workspace(1, 4, 2, 64, "cuda")
    out, lse = api.kda_window_attention(c.q, odd, keys, c.cu, c.table, c.computed, work)
    torch.cuda.synchronize()
    assert not out.any() and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("stride", [0, 1, 3])
def test_token_strides_of_one_token(stride):
    c = Case([1], [4], 4, 2, 64, 16, seed=5)
    q, k, v = c.q.contiguous(), c.k.contiguous(), c.v.contiguous()
    keys, values = c.keys.clone(), c.values.clone()
    want = api.kda_kv_append(q, k, v, keys, values, c.cu, c.table, c.computed)
    got = api.kda_kv_append(*(_restrided(t, d0=stride) for t in (q, k, v)), c.keys, c.values,
                            c.cu, c.table, c.computed)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(c.keys, keys) and torch.equal(c.values, values)

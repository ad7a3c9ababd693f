"""GPU: arguments of the attention layers' calls that both parts of the binding
have to take alike: a truth value that raises."""

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

"""The bounded waits of the attention's tensor-core form, on the GPU.

No input of the C ABI can leave one of its waits unsatisfied, so this test
uses a test build of the library (build.build_variant, compiled with a wait
budget of about 10 ms; never the product library) in which the first CTA's
queries are never handed to the tensor cores.  Every role of that CTA gives
up, with all its copies landed and its tensor memory freed; the launch
returns, the error word carries KDA_ERR_WAIT_TIMEOUT, the rows of the other
CTAs are right, and the product library then runs in the same process.
"""

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from linear_attention_speculative_kda_gb300 import build as kbuild
from tests.attention_helpers import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def starved_lib():
    path = kbuild.build_variant("attention_starved",
                                ["KDA_TEST_ATTENTION_WAIT_BUDGET=20000000LL"])
    return api.bind_library(path)


def _run(c, lib=None):
    work = api.allocate_attention_workspace(c.cu.numel() - 1, c.q_heads, c.kv_heads, c.dim, "cuda",
                                            window=8)
    work.zero_()
    c.err.zero_()
    saved = api._lib_handle
    api._lib_handle = saved if lib is None else lib
    try:
        out, lse = api.kda_window_attention(c.q, c.keys, c.values, c.cu, c.table, c.computed, work,
                                            error_word=c.err)
    finally:
        api._lib_handle = saved
    torch.cuda.synchronize()
    return out, lse, int(c.err.item())


@pytest.mark.parametrize("computed", [[60, 50, 40], [5000, 90, 7000]])
@pytest.mark.parametrize("group", [8, 16])
def test_a_starved_cta_gives_up_and_the_context_stays_usable(starved_lib, computed, group):
    c = Case([8, 3, 8], computed, 2 * group, 2, 128, 16, seed=31)
    api.load_library()
    want, want_lse, err = _run(c)
    assert err == 0
    for _ in range(2):
        out, lse, err = _run(c, starved_lib)
        assert err == api.ERR_WAIT_TIMEOUT
        # the first CTA has the first row's first head only
        assert torch.equal(out[8:], want[8:]) and torch.equal(lse[8:], want_lse[8:])
    again, again_lse, err = _run(c)
    assert err == 0 and torch.equal(again, want) and torch.equal(again_lse, want_lse)

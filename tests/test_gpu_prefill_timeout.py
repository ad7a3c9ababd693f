"""The bounded waits of kda_prefill, on the GPU.

No input of the C ABI can leave one of its waits unsatisfied, so this test
uses a test build of the library (build.build_variant, compiled with a wait
budget of about 10 ms; never the product library) in which the first CTA's
operands are never handed to its consumers.  Every warp of that CTA gives up,
with its copies landed and its tensor memory freed; the launch returns, the
error word carries KDA_ERR_WAIT_TIMEOUT, the rows of the other CTAs are right,
and the product library then runs in the same process.
"""

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from linear_attention_speculative_kda_gb300 import build as kbuild
from tests.delta_helpers import Case, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def starved_lib():
    path = kbuild.build_variant("prefill_starved", ["KDA_TEST_PREFILL_WAIT_BUDGET=20000000LL"])
    return api.bind_library(path)


@pytest.mark.parametrize("lens,heads", [([600, 700], 1), ([1300, 230, 333], 2),  # two CTAs
                                        ([20, 100], 1), ([40, 100], 76)])         # a head; one
def test_a_starved_cta_gives_up_and_the_context_stays_usable(starved_lib, monkeypatch, lens, heads):
    if len(lens) * heads > torch.cuda.get_device_properties(0).multi_processor_count:
        pytest.skip("a CTA would have more than one row and head")
    c = Case(lens, heads, seed=3)
    out = torch.zeros_like(c.q, memory_format=torch.contiguous_format)
    start = c.pool.clone()
    want = run(c, initial=c.sources).clone()
    after = c.pool.clone()
    assert int(c.err.item()) == 0
    # the first CTA has the first row's first head, of which nothing is written
    want_out, want_pool = want.clone(), after.clone()
    want_out[:lens[0], 0] = 7.0
    slot = int(c.slots[0])
    want_pool[slot, 0] = start[slot, 0]
    for _ in range(2):
        c.pool.copy_(start)
        out.fill_(7.0)
        with monkeypatch.context() as m:
            m.setattr(api, "_lib_handle", starved_lib)
            run(c, initial=c.sources, out=out)
        torch.cuda.synchronize()
        assert int(c.err.item()) == api.ERR_WAIT_TIMEOUT
        assert torch.equal(out, want_out) and torch.equal(c.pool, want_pool)
        c.err.zero_()
    c.pool.copy_(start)
    assert torch.equal(run(c, initial=c.sources), want) and torch.equal(c.pool, after)
    assert int(c.err.item()) == 0

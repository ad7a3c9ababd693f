"""The bounded waits of kda_prefill where CTAs have several rows and heads, with
a plan and in turn, on the GPU: as test_gpu_prefill_timeout.py, whose test build
this uses.  The first CTA gives up at its first row and head and writes none of
its others; what the other CTAs have is right."""

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


@pytest.mark.parametrize("lens,heads", [([700] + [30] * 59, 4),       # planned
                                        ([40] + [9] * 99, 2)])        # in turn
def test_a_starved_cta_leaves_the_others_theirs(starved_lib, monkeypatch, lens, heads):
    c = Case(lens, heads, seed=4)
    out = torch.zeros_like(c.q, memory_format=torch.contiguous_format)
    start = c.pool.clone()
    want = run(c, initial=c.sources).clone()
    after = c.pool.clone()
    assert int(c.err.item()) == 0
    c.pool.copy_(start)
    out.fill_(7.0)
    with monkeypatch.context() as m:
        m.setattr(api, "_lib_handle", starved_lib)
        run(c, initial=c.sources, out=out)
    torch.cuda.synchronize()
    assert int(c.err.item()) == api.ERR_WAIT_TIMEOUT
    c.err.zero_()
    lost = []
    cu = c.cu.tolist()
    for b, slot in enumerate(c.slots.tolist()):
        for h in range(heads):
            at = slice(cu[b], cu[b + 1])
            if torch.equal(c.pool[slot, h], after[slot, h]):
                assert torch.equal(out[at, h], want[at, h])
            else:   # all of it is as it was
                assert torch.equal(c.pool[slot, h], start[slot, h])
                assert (out[at, h] == 7.0).all()
                lost.append((b, h))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (0, 0) in lost and len(lost) <= -(-len(lens) * heads // sms) + 1
    c.pool.copy_(start)
    assert torch.equal(run(c, initial=c.sources), want) and torch.equal(c.pool, after)
    assert int(c.err.item()) == 0

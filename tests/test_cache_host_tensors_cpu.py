"""CPU checks of the binding: tensors in host memory, consistent in everything
else, are refused before their addresses reach a kernel."""

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api


@pytest.fixture(scope="module", autouse=True)
def library():
    from linear_attention_speculative_kda_gb300 import build as kbuild
    kbuild.build()


def _plan():
    return dict(cu_seqlens=torch.tensor([0, 2, 4], dtype=torch.int32),
                block_table=torch.ones((2, 4), dtype=torch.int32),
                num_computed=torch.zeros(2, dtype=torch.int32))


def _caches():
    return tuple(torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16) for _ in range(2))


def test_append_refuses_host_tensors():
    keys, values = _caches()
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        api.kda_kv_append(torch.zeros((4, 8, 64), dtype=torch.bfloat16), k, k, keys, values,
                          **_plan())


def test_attention_refuses_host_tensors():
    keys, values = _caches()
    with pytest.raises(ValueError, match="GPU"):
        api.kda_window_attention(torch.zeros((4, 8, 64), dtype=torch.bfloat16), keys, values,
                                 workspace=torch.zeros(1 << 20, dtype=torch.uint8), window=2,
                                 **_plan())


def test_token_logprobs_refuses_host_tensors():
    with pytest.raises(ValueError, match="GPU"):
        api.kda_token_logprobs(torch.zeros((3, 50)), torch.zeros(3, dtype=torch.int32), num_top=2)

"""CPU check of the binding: every call of the library is made with its
tensors' device as the current one (the library launches on the current device,
and a stream handle may not say which device it belongs to).  Host tensors that
say they are on a second GPU, and a library and a device switch that only keep
record, stand in."""

import contextlib

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
WHERE = torch.device("cuda", 1)


class Elsewhere(torch.Tensor):
    @property
    def device(self):
        return WHERE

    def get_device(self):
        return WHERE.index


def _there(*shape, dtype=F32):
    return torch.Tensor._make_subclass(Elsewhere, torch.zeros(shape, dtype=dtype))


@pytest.fixture()
def calls(monkeypatch):
    current, made = [0], []

    @contextlib.contextmanager
    def device(which):
        before, current[0] = current[0], which
        yield
        current[0] = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("records_bytes"):
                    return 64
                made.append((name, current[0]))
                return api.KDA_OK
            return call
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "load_library", lambda: Library())
    monkeypatch.setattr(api, "_quick", None)
    monkeypatch.setattr(api, "_stream_ptr", lambda device: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda device: 0)
    api.records_bytes.cache_clear()
    yield made
    api.records_bytes.cache_clear()
    assert current[0] == 0          # and the current device is what it was


def _rows():
    return dict(cu_seqlens=_there(3, dtype=I32), state_indices=_there(2, dtype=I32))


def _kda():
    return dict(A_log=_there(1), g_bias=_there(128), state_pool=_there(3, 1, 128, 128),
                records=_there(64, dtype=BF), window=4, record_slots=2)


def _table():
    return dict(block_table=_there(2, 4, dtype=I32), num_computed=_there(2, dtype=I32))


def _cache():
    return dict(key_cache=_there(3, 16, 2, 64, dtype=BF), value_cache=_there(3, 16, 2, 64, dtype=BF),
                cu_seqlens=_there(3, dtype=I32), **_table())


CALLS = {
    "kda_verify": lambda: api.kda_verify(
        *(_there(4, 1, 128, dtype=BF) for _ in range(4)), _there(4, 1, dtype=BF),
        out=_there(4, 1, 128, dtype=BF), **_rows(), **_kda()),
    "kda_commit": lambda: api.kda_commit(num_accepted=_there(2, dtype=I32), **_rows(), **_kda()),
    "kda_flush": lambda: api.kda_flush(pending=_there(2, dtype=I32),
                                       state_indices=_there(2, dtype=I32), **_kda()),
    "kda_conv_compact": lambda: api.kda_conv_compact(
        _there(3, 16, 8, dtype=BF), num_accepted=_there(2, dtype=I32), window=4, **_rows()),
    "kda_commit_align": lambda: api.kda_commit_align(
        num_accepted=_there(2, dtype=I32), block_size=16, **_rows(), **_kda(), **_table()),
    "kda_conv_compact_align": lambda: api.kda_conv_compact_align(
        _there(3, 16, 8, dtype=BF), num_accepted=_there(2, dtype=I32), block_size=16, window=4,
        **_rows(), **_table()),
    "kda_record_state_blocks": lambda: api.kda_record_state_blocks(
        *(_there(2, dtype=I32) for _ in range(5)), block_size=16, block_table_width=4),
    "kda_kv_append_packed": lambda: api.kda_kv_append(
        None, _there(4, 2, 64, dtype=BF), _there(4, 2, 64, dtype=BF), **_cache()),
    "kda_window_attention_packed": lambda: api.kda_window_attention(
        _there(4, 8, 64, dtype=BF), workspace=_there(64, dtype=torch.uint8),
        out=_there(4, 8, 64, dtype=BF), lse=_there(4, 8), **_cache()),
    "kda_token_logprobs_packed": lambda: api.kda_token_logprobs(
        _there(3, 50), _there(3, dtype=I32), num_top=1,
        out=api.TokenLogprobs(_there(3), _there(3), _there(3), _there(3, 1),
                              _there(3, 1, dtype=I32))),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_are_made_on_the_tensors_device(calls, name, monkeypatch):
    CALLS[name]()
    assert calls == [(name, 1)]
    # and where it is the current one already, nothing is switched
    monkeypatch.setattr(torch.cuda, "device", None)
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        CALLS[name]()
    assert [n for n, _ in calls] == [name, name]

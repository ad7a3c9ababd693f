"""CPU checks of the append, window attention and log probability entry
points: every refusal returns its status before anything is launched, and the
binding refuses mismatched tensors before it calls the library."""

import ctypes

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from linear_attention_speculative_kda_gb300 import build as kbuild

FAKE = 0x100000  # an aligned address that is never dereferenced
BAD, UNSUPPORTED, OK = api.KDA_ERR_INVALID_ARG, api.KDA_ERR_UNSUPPORTED, api.KDA_OK


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return api.load_library()


def _cfg(**kw):
    base = dict(q_heads=8, kv_heads=2, head_dim=128, dtype=0, num_blocks=9, window=4,
                left_window=0, rotary_dim=64, interleaved=0, scale=0.1, stride_block=16 * 256,
                stride_token=256, stride_head=128, stride_q_t=1536, stride_k_t=1536,
                stride_v_t=1536)
    base.update(kw)
    return api.KdaCacheConfig(**base)


def _align(**kw):
    base = dict(block_table=FAKE, block_table_stride=8, block_table_width=8, block_size=16,
                num_requests=4, reserved=0, num_computed=FAKE, request_indices=None)
    base.update(kw)
    return api.KdaAlign(**base)


def _append(lib, cfg=None, al=None, B=3, T=5, **ptrs):
    p = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, keys=FAKE, values=FAKE, freq=FAKE, cu=FAKE,
             err=None)
    p.update(ptrs)
    cfg = _cfg() if cfg is None else cfg
    alp = ctypes.byref(_align() if al is None else al) if al is not False else None
    return lib.kda_kv_append(ctypes.byref(cfg) if cfg is not False else None, p["q"], p["k"],
                             p["v"], p["q_out"], p["keys"], p["values"], p["freq"], p["cu"], B, T,
                             alp, p["err"], None)


def _attend(lib, cfg=None, al=None, B=3, T=5, size=None, **ptrs):
    p = dict(q=FAKE, keys=FAKE, values=FAKE, cu=FAKE, work=FAKE, out=FAKE, lse=None, err=None)
    p.update(ptrs)
    cfg = _cfg() if cfg is None else cfg
    cfgp = ctypes.byref(cfg) if cfg is not False else None
    alp = ctypes.byref(_align() if al is None else al) if al is not False else None
    if size is None:
        size = 1 << 40
    return lib.kda_window_attention(cfgp, p["q"], p["keys"], p["values"], p["cu"], B, T, alp,
                                    p["work"], size, p["out"], p["lse"], p["err"], None)


COMMON = [
    (dict(q_heads=0), BAD), (dict(kv_heads=0), BAD), (dict(q_heads=7), BAD),
    (dict(num_blocks=0), BAD), (dict(dtype=2), BAD), (dict(dtype=-1), BAD),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(q_heads=65536, kv_heads=65536), UNSUPPORTED),
    (dict(stride_block=4), BAD), (dict(stride_token=0), BAD), (dict(stride_head=129), BAD),
    (dict(stride_q_t=1540), BAD),
]


@pytest.mark.parametrize("change,status", COMMON)
def test_config_refusals(lib, change, status):
    assert _append(lib, _cfg(**change)) == status
    assert _attend(lib, _cfg(**change)) == status


@pytest.mark.parametrize("change", [
    dict(block_table=None), dict(num_computed=None), dict(block_table_width=0),
    dict(block_table_stride=4), dict(block_size=0), dict(num_requests=0), dict(num_requests=2),
    dict(reserved=1), dict(block_table=FAKE + 2), dict(num_computed=FAKE + 1),
    dict(request_indices=FAKE + 2)])
def test_plan_refusals(lib, change):
    assert _append(lib, al=_align(**change)) == BAD
    assert _attend(lib, al=_align(**change)) == BAD


def test_append_refusals(lib):
    assert _append(lib, False) == BAD and _append(lib, al=False) == BAD
    for ptr in ("k", "v", "q_out", "keys", "values", "freq", "cu"):
        assert _append(lib, **{ptr: None}) == BAD, ptr
    for ptr in ("q", "k", "v", "q_out", "keys", "values"):
        assert _append(lib, **{ptr: FAKE + 8}) == BAD, ptr
    assert _append(lib, freq=FAKE + 4) == BAD
    assert _append(lib, err=FAKE + 2) == BAD
    for change in (dict(rotary_dim=136), dict(rotary_dim=24), dict(rotary_dim=-16),
                   dict(interleaved=2), dict(stride_k_t=0), dict(stride_v_t=12)):
        assert _append(lib, _cfg(**change)) == BAD, change
    assert _append(lib, B=-1) == BAD and _append(lib, T=-1) == BAD
    # nothing to do: no pointer is looked at
    assert _append(lib, B=0, al=False, k=None, cu=None) == OK
    assert _append(lib, T=0, al=False, k=None, cu=None) == OK


def test_attention_refusals(lib):
    assert _attend(lib, False) == BAD and _attend(lib, al=False) == BAD
    for ptr in ("q", "keys", "values", "cu", "work", "out"):
        assert _attend(lib, **{ptr: None}) == BAD, ptr
        assert _attend(lib, **{ptr: FAKE + 2}) == BAD, ptr
    assert _attend(lib, lse=FAKE + 2) == BAD and _attend(lib, err=FAKE + 1) == BAD
    assert _attend(lib, _cfg(window=0)) == BAD
    assert _attend(lib, _cfg(left_window=-1)) == BAD
    assert _attend(lib, _cfg(scale=float("nan"))) == BAD
    assert _attend(lib, _cfg(scale=float("inf"))) == BAD
    assert _attend(lib, _cfg(window=9)) == UNSUPPORTED
    assert _attend(lib, _cfg(window=8, q_heads=34)) == UNSUPPORTED     # 8 * 17 query rows
    need = lib.kda_attention_workspace_bytes(ctypes.byref(_cfg()), 3)
    assert need > 0 and _attend(lib, size=need - 1) == BAD
    assert _attend(lib, B=-1) == BAD and _attend(lib, T=-1) == BAD
    assert _attend(lib, T=0, al=False, q=None, work=None, size=0) == OK
    assert _attend(lib, B=0, al=False, q=None, work=None, size=0) == OK
    assert lib.kda_attention_workspace_bytes(ctypes.byref(_cfg(window=9)), 3) == 0
    assert lib.kda_attention_workspace_bytes(None, 3) == 0
    assert lib.kda_attention_workspace_bytes(ctypes.byref(_cfg()), -1) == 0


def test_logprobs_refusals(lib):
    def call(logits=FAKE, dtype=0, stride=100, rows=3, vocab=100, tokens=FAKE, top=4, lp=FAKE,
             ent=None, lse=None, tv=FAKE, ti=FAKE, err=None):
        return lib.kda_token_logprobs(logits, dtype, stride, rows, vocab, tokens, top, lp, ent,
                                      lse, tv, ti, err, None)
    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(stride=-1),
               dict(top=-1), dict(top=9, vocab=8), dict(logits=None), dict(tokens=None),
               dict(lp=None), dict(tv=None), dict(ti=None), dict(logits=FAKE + 1),
               dict(dtype=2, logits=FAKE + 2), dict(tokens=FAKE + 2), dict(lp=FAKE + 1),
               dict(ent=FAKE + 2), dict(lse=FAKE + 2), dict(tv=FAKE + 2), dict(ti=FAKE + 2),
               dict(err=FAKE + 2)):
        assert call(**kw) == BAD, kw
    assert call(top=33) == UNSUPPORTED
    assert call(rows=0, logits=None, tokens=None, lp=None) == OK


def _tensors(T=5, hq=8, hk=2, d=64, bs=16, blocks=6, B=2, dtype=torch.bfloat16):
    i32 = torch.int32
    return dict(q=torch.zeros((T, hq, d), dtype=dtype), k=torch.zeros((T, hk, d), dtype=dtype),
                v=torch.zeros((T, hk, d), dtype=dtype),
                key_cache=torch.zeros((blocks, bs, hk, d), dtype=dtype),
                value_cache=torch.zeros((blocks, bs, hk, d), dtype=dtype),
                cu_seqlens=torch.tensor([0, 2, T], dtype=i32),
                block_table=torch.ones((B, 4), dtype=i32),
                num_computed=torch.zeros(B, dtype=i32))


def test_binding_refuses_bad_append_arguments(lib):
    def call(**kw):
        a = _tensors()
        extra = {}
        for name, val in kw.items():
            (a if name in a else extra)[name] = val
        api.kda_kv_append(**a, **extra)
    bf, f16, i32 = torch.bfloat16, torch.float16, torch.int32
    for kw in (dict(k=torch.zeros((5, 2, 64), dtype=f16)),
               dict(key_cache=torch.zeros((6, 16, 2, 64))),
               dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)),
               dict(inv_freq=torch.zeros(16)),
               dict(error_word=torch.zeros(1))):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(k=torch.zeros((4, 2, 64), dtype=bf)), dict(v=torch.zeros((5, 2, 32), dtype=bf)),
               dict(q=torch.zeros((5, 7, 64), dtype=bf)), dict(q=torch.zeros((4, 8, 64), dtype=bf)),
               dict(q=torch.zeros((5, 8, 128), dtype=bf)[..., ::2]),
               dict(value_cache=torch.zeros((6, 16, 1, 64), dtype=bf)),
               dict(value_cache=torch.zeros((6, 2, 16, 64), dtype=bf).transpose(1, 2)),
               dict(key_cache=torch.zeros((6, 32, 64), dtype=bf)),
               dict(q_out=torch.zeros((5, 4, 64), dtype=bf)),
               dict(q=None, q_out=torch.zeros((5, 8, 64), dtype=bf)),
               dict(num_computed=torch.zeros(1, dtype=i32)),
               dict(block_table=torch.ones((1, 4), dtype=i32)),
               dict(request_indices=torch.zeros(1, dtype=i32)),
               dict(error_word=torch.zeros(0, dtype=i32)),
               dict(inv_freq=torch.zeros((2, 8), dtype=torch.float64))):
        with pytest.raises(ValueError):
            call(**kw)


def test_binding_refuses_bad_attention_arguments(lib):
    work = api.allocate_attention_workspace(2, 8, 2, 64, "cpu")

    def call(**kw):
        a = _tensors()
        del a["k"], a["v"]
        extra = dict(workspace=work)
        for name, val in kw.items():
            (a if name in a else extra)[name] = val
        api.kda_window_attention(**a, **extra)
    bf = torch.bfloat16
    for kw in (dict(q=torch.zeros((5, 8, 64))), dict(workspace=work.view(torch.int32)),
               dict(out=torch.zeros((5, 8, 64))), dict(lse=torch.zeros((5, 8), dtype=bf))):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=torch.zeros((5, 3, 64), dtype=bf)),
               dict(out=torch.zeros((4, 8, 64), dtype=bf)), dict(lse=torch.zeros((5, 4)))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        api.allocate_attention_workspace(2, 8, 2, 96, "cpu")


def test_binding_refuses_bad_logprob_arguments(lib):
    x = torch.zeros((3, 50))
    tokens = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        api.kda_token_logprobs(x.double(), tokens)
    with pytest.raises(TypeError):
        api.kda_token_logprobs(x, tokens.long())
    with pytest.raises(ValueError):
        api.kda_token_logprobs(x, tokens[:2])
    with pytest.raises(ValueError):
        api.kda_token_logprobs(x.t(), torch.zeros(50, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.kda_token_logprobs(x, tokens, num_top=2, out=api.allocate_token_logprobs(3, 1, "cpu"))


def test_packed_calls_read_their_fields(lib):
    # each field where it belongs: breaking one gives the status that the call
    # with separate arguments gives, and only then
    def append(**change):
        f = dict(q_heads=8, kv_heads=2, head_dim=128, dtype=0, num_blocks=9, window=1,
                 left_window=0, rotary_dim=64, interleaved=0, scale=1.0, stride_block=4096,
                 stride_token=256, stride_head=128, stride_q=1536, stride_k=1536, stride_v=1536,
                 table=FAKE, table_stride=8, width=8, block_size=16, requests=4, reserved=0,
                 computed=FAKE, request_indices=0, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, keys=FAKE,
                 values=FAKE, freq=FAKE, cu=FAKE, B=3, T=5, err=0, stream=0)
        f.update(change)
        return lib.kda_kv_append_packed(api._APPEND_ARGS(*f.values()))

    def attend(**change):
        f = dict(q_heads=8, kv_heads=2, head_dim=128, dtype=0, num_blocks=9, window=4,
                 left_window=0, rotary_dim=0, interleaved=0, scale=0.1, stride_block=4096,
                 stride_token=256, stride_head=128, stride_q=1536, stride_k=8, stride_v=8,
                 table=FAKE, table_stride=8, width=8, block_size=16, requests=4, reserved=0,
                 computed=FAKE, request_indices=0, q=FAKE, keys=FAKE, values=FAKE, cu=FAKE, B=3,
                 T=5, work=FAKE, size=1 << 40, out=FAKE, lse=0, err=0, stream=0)
        f.update(change)
        return lib.kda_window_attention_packed(api._ATTENTION_ARGS(*f.values()))

    def logprobs(**change):
        f = dict(logits=FAKE, stride=100, dtype=0, rows=3, vocab=100, top=4, tokens=FAKE, lp=FAKE,
                 ent=FAKE, lse=FAKE, tv=FAKE, ti=FAKE, err=0, stream=0)
        f.update(change)
        return lib.kda_token_logprobs_packed(api._LOGPROBS_ARGS(*f.values()))

    assert append(B=0) == OK and append(T=0) == OK
    assert attend(B=0) == OK and attend(T=0) == OK and logprobs(rows=0) == OK
    common = [dict(q_heads=7), dict(kv_heads=0), dict(dtype=3), dict(num_blocks=0),
              dict(stride_block=4), dict(stride_token=0), dict(stride_head=129), dict(stride_q=4),
              dict(table=0), dict(table_stride=7), dict(width=0), dict(block_size=0),
              dict(requests=0), dict(reserved=1), dict(computed=FAKE + 1),
              dict(request_indices=FAKE + 2), dict(q=FAKE + 8), dict(keys=0), dict(values=FAKE + 8),
              dict(cu=FAKE + 2), dict(B=-1), dict(err=FAKE + 1)]
    for change in common:
        assert append(**change) == BAD, change
        assert attend(**change) == BAD, change
    assert append(head_dim=96) == UNSUPPORTED and attend(head_dim=96) == UNSUPPORTED
    for change in (dict(rotary_dim=24), dict(interleaved=2), dict(stride_k=0), dict(stride_v=4),
                   dict(k=0), dict(v=FAKE + 8), dict(q_out=0), dict(freq=FAKE + 4), dict(T=-1)):
        assert append(**change) == BAD, change
    for change in (dict(window=0), dict(left_window=-1), dict(scale=float("nan")), dict(work=0),
                   dict(size=64), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(T=-1)):
        assert attend(**change) == BAD, change
    assert attend(window=9) == UNSUPPORTED
    for change in (dict(logits=0), dict(stride=-1), dict(dtype=3), dict(rows=-1), dict(vocab=0),
                   dict(top=101), dict(tokens=FAKE + 1), dict(lp=0), dict(ent=FAKE + 1),
                   dict(lse=FAKE + 1), dict(tv=0), dict(ti=FAKE + 2), dict(err=FAKE + 2)):
        assert logprobs(**change) == BAD, change
    assert logprobs(top=33) == UNSUPPORTED
    assert lib.kda_kv_append_packed(None) == BAD
    assert lib.kda_window_attention_packed(None) == BAD
    assert lib.kda_token_logprobs_packed(None) == BAD

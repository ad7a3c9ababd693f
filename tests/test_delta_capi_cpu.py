"""CPU: refusals of kda_prefill, kda_decode and kda_kv_norm_append, in the C
ABI (made-up addresses, nothing is launched) and in the binding."""

import ctypes

import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from linear_attention_speculative_kda_gb300 import build as kbuild

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FAKE = 1 << 20
BAD, NOT_BUILT = api.KDA_ERR_INVALID_ARG, api.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return api.load_library()


def _config(**changes):
    c = api.make_config(2, 1, 5, 0, strides=(256,) * 4 + (2,))
    for name, value in changes.items():
        setattr(c, name, value)
    return c


def _call(lib, prefill, cfg=None, B=3, tokens=9, **changes):
    p = dict.fromkeys(("q", "k", "v", "g", "beta", "A_log", "bias", "pool", "cu", "slots",
                       "initial", "out", "err"), FAKE)
    p.update(changes)
    head = [ctypes.byref(cfg or _config())] + [p[n] for n in ("q", "k", "v", "g", "beta", "A_log",
                                                              "bias", "pool")]
    if prefill:
        return lib.kda_prefill(*head, p["cu"], p["slots"], p["initial"], B, tokens, p["out"],
                               p["err"], None)
    return lib.kda_decode(*head, p["slots"], p["initial"], B, p["out"], p["err"], None)


@pytest.mark.parametrize("prefill", [True, False])
def test_delta_refusals(lib, prefill):
    def call(*a, **k):
        return _call(lib, prefill, *a, **k)
    for name in ("q", "k", "v", "g", "beta", "A_log", "bias", "pool", "slots", "out"):
        assert call(**{name: None}) == BAD, name
    for name, off in (("q", 4), ("k", 4), ("v", 4), ("g", 4), ("beta", 1), ("A_log", 2),
                      ("bias", 8), ("pool", 8), ("slots", 2), ("initial", 2), ("out", 8),
                      ("err", 2)):
        assert call(**{name: FAKE + off}) == BAD, name
    for field in ("stride_q_t", "stride_k_t", "stride_v_t", "stride_g_t"):
        for value in (0, -4, 258):
            assert call(_config(**{field: value})) == BAD
    assert call(_config(stride_beta_t=0)) == BAD
    assert call(B=-1) == BAD
    for field, value, want in (("num_heads", 0, BAD), ("num_heads", 32768, NOT_BUILT),
                               ("num_slots", 0, BAD), ("head_dim", 64, NOT_BUILT),
                               ("use_lower_bound", 2, BAD), ("reserved", 1, BAD),
                               ("scale", float("inf"), BAD), ("scale", float("nan"), BAD)):
        assert call(_config(**{field: value})) == want, field
    for bound in (0.0, 1.0, float("nan"), float("-inf")):
        assert call(_config(use_lower_bound=1, lower_bound=bound)) == BAD
    # nothing to do: no pointer is looked at
    assert call(B=0, q=None, pool=None, slots=None) == api.KDA_OK


def test_prefill_refusals(lib):
    assert _call(lib, True, cu=None) == BAD
    assert _call(lib, True, cu=FAKE + 2) == BAD
    assert _call(lib, True, tokens=-1) == BAD
    assert _call(lib, True, tokens=0, q=None) == api.KDA_OK
    assert lib.kda_prefill_packed(None) == BAD and lib.kda_decode_packed(None) == BAD
    assert lib.kda_kv_norm_append_packed(None) == BAD


def _norm(lib, weight_dtype=0, eps=1e-6, q_weight=FAKE, k_weight=FAKE, B=2, **config):
    c = api.KdaCacheConfig(4, 2, 64, 0, 9, 1, 0, 64, 0, 1.0, 2048, 128, 64, 256, 128, 128)
    for name, value in config.items():
        setattr(c, name, value)
    al = api.KdaAlign(FAKE, 8, 8, 16, 2, 0, FAKE, None)
    return lib.kda_kv_norm_append(ctypes.byref(c), FAKE, FAKE, FAKE, q_weight, k_weight,
                                  weight_dtype, eps, FAKE, FAKE, FAKE, FAKE, FAKE, B, 5,
                                  ctypes.byref(al), None, None)


def test_norm_append_refusals(lib):
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == BAD
    for dtype in (1, 3, -1):
        assert _norm(lib, weight_dtype=dtype) == BAD
    assert _norm(lib, q_weight=FAKE + 1) == BAD and _norm(lib, k_weight=FAKE + 1) == BAD
    assert _norm(lib, weight_dtype=2, k_weight=FAKE + 2) == BAD
    assert _norm(lib, rotary_dim=8) == BAD       # and all that the append refuses
    assert _norm(lib, head_dim=96) == NOT_BUILT
    assert _norm(lib, B=0) == api.KDA_OK


def _tensors(tokens=4, rows=2, heads=2, slots=5, dim=128):
    def zeros(*shape, dtype=BF):
        return torch.zeros(shape, dtype=dtype)
    return dict(q=zeros(tokens, heads, dim), k=zeros(tokens, heads, dim),
                v=zeros(tokens, heads, dim), g_raw=zeros(tokens, heads, dim),
                beta_raw=zeros(tokens, heads), A_log=zeros(heads, dtype=F32),
                g_bias=zeros(heads * dim, dtype=F32),
                state_pool=zeros(slots, heads, dim, dim, dtype=F32),
                cu_seqlens=zeros(rows + 1, dtype=I32), state_indices=zeros(rows, dtype=I32))


@pytest.mark.parametrize("name,bad,error", [
    ("q", torch.zeros(4, 2, 128), TypeError),
    ("q", torch.zeros(4, 3, 128, dtype=BF), ValueError),
    ("k", torch.zeros(5, 2, 128, dtype=BF), ValueError),
    ("v", torch.zeros(4, 2, 256, dtype=BF)[:, :, ::2], ValueError),
    ("g_raw", torch.zeros(4, 256, dtype=BF), ValueError),
    ("beta_raw", torch.zeros(4, 3, dtype=BF), ValueError),
    ("beta_raw", torch.zeros(4, 4, dtype=BF)[:, ::2], ValueError),
    ("A_log", torch.zeros(1), ValueError),
    ("A_log", torch.zeros(2, dtype=BF), TypeError),
    ("g_bias", torch.zeros(255), ValueError),
    ("state_pool", torch.zeros(5, 2, 128, 64), ValueError),
    ("state_pool", torch.zeros(5, 2, 128, 128).transpose(2, 3), ValueError),
    ("cu_seqlens", torch.zeros(2, dtype=I32), ValueError),
    ("cu_seqlens", torch.zeros(3, dtype=torch.int64), TypeError),
    ("cu_seqlens", None, ValueError),
    ("state_indices", torch.zeros(4, dtype=I32)[::2], ValueError),
    ("initial_indices", torch.zeros(1, dtype=I32), ValueError),
    ("initial_indices", torch.zeros(2, dtype=torch.int64), TypeError),
    ("out", torch.zeros(4, 2, 128), TypeError),
    ("out", torch.zeros(4, 2, 64, dtype=BF), ValueError),
    ("error_word", torch.zeros(0, dtype=I32), ValueError),
])
def test_binding_refuses(lib, name, bad, error):
    t = _tensors()
    t[name] = bad
    with pytest.raises(error):
        api.kda_prefill(**t)


def test_binding_refuses_host_tensors_and_counts(lib):
    with pytest.raises(ValueError, match="GPU"):
        api.kda_prefill(**_tensors())
    t = _tensors()
    t.pop("cu_seqlens")
    with pytest.raises(ValueError, match="one token per row"):
        api.kda_decode(**t)
    with pytest.raises(ValueError, match="GPU"):
        t = _tensors(tokens=2)
        t.pop("cu_seqlens")
        api.kda_decode(**t)


def _append_tensors(dtype=BF):
    return dict(q=torch.zeros(4, 4, 64, dtype=dtype), k=torch.zeros(4, 2, 64, dtype=dtype),
                v=torch.zeros(4, 2, 64, dtype=dtype),
                key_cache=torch.zeros(3, 16, 2, 64, dtype=dtype),
                value_cache=torch.zeros(3, 16, 2, 64, dtype=dtype),
                cu_seqlens=torch.zeros(3, dtype=I32), block_table=torch.zeros(2, 4, dtype=I32),
                num_computed=torch.zeros(2, dtype=I32))


@pytest.mark.parametrize("weights,error", [
    (dict(q_weight=torch.ones(64, dtype=torch.float16)), TypeError),
    (dict(q_weight=torch.ones(64, dtype=torch.float64)), TypeError),
    (dict(q_weight=torch.ones(64, dtype=BF), k_weight=torch.ones(64)), TypeError),
    (dict(k_weight=torch.ones(128)), ValueError),
    (dict(k_weight=torch.ones(1, 64)), ValueError),
    (dict(q_weight=torch.ones(128)[::2]), ValueError),
    (dict(q_weight=torch.ones(64)), ValueError),          # host tensors
])
def test_norm_append_binding_refuses(lib, weights, error):
    with pytest.raises(error):
        api.kda_kv_norm_append(**_append_tensors(), **weights)


def test_calls_are_made_on_the_tensors_device(monkeypatch):
    """As test_call_device_cpu does for the other calls."""
    from tests import test_call_device_cpu as other
    made = []

    class Library:
        prefill_address = decode_address = norm_append_address = 0

        def __getattr__(self, name):
            def call(*args):
                made.append((name, current[0]))
                return api.KDA_OK
            return call
    import contextlib
    current = [0]

    @contextlib.contextmanager
    def device(which):
        before, current[0] = current[0], which
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "load_library", lambda: Library())
    monkeypatch.setattr(api, "_quick_more", None)
    monkeypatch.setattr(api, "_raw_stream", lambda device: 0)
    there = {n: torch.Tensor._make_subclass(other.Elsewhere, t) for n, t in _tensors().items()}
    out = torch.Tensor._make_subclass(other.Elsewhere, torch.zeros(4, 2, 128, dtype=BF))
    api.kda_prefill(**there, out=out)
    for name in ("q", "k", "v", "g_raw", "beta_raw"):
        there[name] = there[name][:2]
    there.pop("cu_seqlens")
    api.kda_decode(**there, out=out[:2])
    cache = {n: torch.Tensor._make_subclass(other.Elsewhere, t)
             for n, t in _append_tensors().items()}
    api.kda_kv_norm_append(**dict(cache, q=None))
    assert made == [("kda_prefill_packed", 1), ("kda_decode_packed", 1),
                    ("kda_kv_norm_append_packed", 1)]

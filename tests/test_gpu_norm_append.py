"""GPU: the cache append with head norms against the float64 oracle.

Bound: the sum of D squares is within (D / 2 + 8) 2^-24 of it in fp32 and its
root within half of that and 2^-22; the products with the root and the weight
add 2 * 2^-24; the rotation adds 1e-6 of the pair (test_gpu_append).  So 6e-6
of the head's largest normed value, then half a step of the storage type."""

import numpy as np
import pytest
import torch

from linear_attention_speculative_kda_gb300 import api
from oracle import attention_oracle as A
from oracle import delta_oracle as D
from tests.attention_helpers import Case, f64, frequencies, half_step, smallest_half

pytestmark = pytest.mark.gpu


def _check(c, rotary, interleaved=False, weights="own", eps=1e-6, with_q=True, inplace=False,
           requests=None, want_err=0, seed=0):
    gen = torch.Generator().manual_seed(seed + 100)
    freq = frequencies(rotary) if rotary else None
    cu, table, computed = c.meta()
    req = None if requests is None else torch.tensor(requests, dtype=torch.int32, device="cuda")
    dtype = {"own": c.dtype, "fp32": torch.float32}.get(weights)
    wq, wk = (None if dtype is None else
              (1 + 0.5 * torch.randn(c.dim, generator=gen)).to(dtype).cuda() for _ in range(2))
    keys, values = f64(c.keys), f64(c.values)
    q = D.head_norm(f64(c.q), None if wq is None else f64(wq), eps) if with_q else None
    k = D.head_norm(f64(c.k), None if wk is None else f64(wk), eps)
    want_q, touched, _ = A.append(q, k, f64(c.v), keys, values, cu, table, computed,
                                  [] if freq is None else f64(freq), interleaved, requests)
    before_k = c.keys.clone()
    if inplace:
        c.q = c.q.contiguous()
    q_out = None
    if with_q:
        q_out = c.q if inplace else torch.full(c.q.shape, 7.0, dtype=c.dtype, device="cuda")
    got = api.kda_kv_norm_append(c.q if with_q else None, c.k, c.v, c.keys, c.values, c.cu, c.table,
                                 c.computed, q_weight=wq, k_weight=wk, eps=eps, inv_freq=freq,
                                 interleaved=interleaved, q_out=q_out, request_indices=req,
                                 error_word=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == want_err
    mark = torch.from_numpy(touched).cuda()[:, :, None, None]
    assert torch.equal(torch.where(mark, before_k, c.keys), before_k)
    assert torch.equal(c.values, torch.from_numpy(values).to(c.dtype).cuda())
    step, least = half_step(c.dtype), smallest_half(c.dtype)

    def near(x, ref):
        size = np.abs(ref).max(axis=-1, keepdims=True)
        assert np.all(np.abs(x - ref) <= step * np.abs(ref) * 1.001 + 6e-6 * size + least)
    near(f64(c.keys), keys)
    if with_q:
        written = ~np.isnan(want_q)
        near(f64(got), np.where(written, want_q, f64(q_out)))
        if not inplace:
            assert np.all(f64(got)[~written] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rotary", [(128, 128), (128, 64), (64, 64), (64, 16), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_types_and_rotations(dtype, dim, rotary, interleaved):
    c = Case([1, 4, 0, 7], [0, 15, 3, 1000], 8, 2, dim, 16, dtype, seed=dim + rotary)
    _check(c, rotary, interleaved, weights="fp32" if interleaved else "own")


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (7, 1), (12, 4), (64, 8), (33, 11)])
def test_head_counts(q_heads, kv_heads):
    _check(Case([3, 5], [9, 40], q_heads, kv_heads, 64, 24, seed=q_heads), 32)


@pytest.mark.parametrize("layout", ["tokens", "heads", "pairs"])
def test_cache_layouts(layout):
    _check(Case([5, 70], [100, 3], 4, 2, 128, 32, layout=layout), 128, weights=None)


def test_prompts():
    _check(Case([900, 1, 333], [0, 5000, 77], 16, 4, 128, 64, "fp16"), 64, True)
    _check(Case([2000], [0], 8, 8, 64, 16), 64)


def test_keys_alone_in_place_and_other_requests():
    _check(Case([3, 9], [4, 100], 8, 2, 128, 16), 128, with_q=False)
    _check(Case([3, 9], [4, 100], 8, 2, 128, 16), 128, inplace=True)
    _check(Case([3, 9, 2], [4, 100, 6], 8, 2, 64, 16), 64, requests=[2, 0, 1])


def test_sizes_of_values_and_eps():
    for size, eps in ((1e-4, 1e-6), (1e-4, 0.0), (300.0, 1e-6), (1.0, 0.5)):
        c = Case([6, 2], [5, 30], 4, 2, 128, 16)
        c.q, c.k = (c.q.float() * size).to(c.dtype), (c.k.float() * size).to(c.dtype)
        _check(c, 128, eps=eps)
    c = Case([6, 2], [5, 30], 4, 2, 128, 16)
    c.k = c.k.clone()
    c.k[2] = 0.0                    # a head of zeros stays one
    _check(c, 128)


def test_null_blocks_and_bad_rows():
    c = Case([5, 6, 7], [10, 20, 30], 4, 2, 128, 16)
    c.table[1] = 0
    _check(c, 128)
    c = Case([5, 6, 7], [10, 20, 30], 4, 2, 128, 16)
    c.computed[1] = -1
    _check(c, 128, want_err=api.ROW_BAD_BLOCK)


def test_a_norm_of_ones_is_scaled_alone():
    """Without weights and with heads whose mean square is 1 it is the append."""
    c = Case([9], [12], 4, 2, 128, 16)
    signs = torch.where(c.q > 0, 1.0, -1.0).to(c.dtype)
    keys = torch.where(c.k > 0, 1.0, -1.0).to(c.dtype)
    freq = frequencies(128)
    a = api.kda_kv_norm_append(signs, keys, c.v, c.keys, c.values, c.cu, c.table, c.computed,
                               eps=0.0, inv_freq=freq)
    first = c.keys.clone()
    b = api.kda_kv_append(signs, keys, c.v, c.keys, c.values, c.cu, c.table, c.computed,
                          inv_freq=freq)
    # the root of a mean of 1 is within 2^-22 of 1: at most one step apart
    for x, y in ((a, b), (first, c.keys)):
        assert ((x.float() - y.float()).abs() <= 2.0 ** -7 * y.float().abs() + 1e-6).all()

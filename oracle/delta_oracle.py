"""Oracle of the delta rule's prompts and single tokens, and of the norms in
front of the cache append, in float64 on the CPU from their definitions
(include/kda.h).  Test infrastructure only; shares no code with the library.
"""

from __future__ import annotations

import numpy as np


def _sigmoid(x):
    z = np.exp(-np.abs(x))   # (as exact beside itself far below 0)
    return np.where(x < 0.0, z, 1.0) / (1.0 + z)


def log_decay(x, a_log, lower_bound=None):
    """x: [..., H, D] gate inputs with their bias; a_log: [H]."""
    a = np.exp(a_log)[:, None]
    if lower_bound is not None:
        return lower_bound * _sigmoid(a * x)
    return -a * (np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x))))


def tokens(state, q, k, v, g_raw, beta_raw, a_log, g_bias, lower_bound=None, scale=None):
    """One row from state [H, V, K], token by token: (output [H, V], the state
    behind the token, its delta [H, V])."""
    s = np.array(state, dtype=np.float64)
    n, h, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    for t in range(n):
        s = s * np.exp(log_decay(g_raw[t] + g_bias.reshape(h, d), a_log, lower_bound))[:, None, :]
        unit_k = k[t] / np.sqrt((k[t] ** 2).sum(-1, keepdims=True) + 1e-6)
        unit_q = q[t] / np.sqrt((q[t] ** 2).sum(-1, keepdims=True) + 1e-6)
        delta = _sigmoid(beta_raw[t])[:, None] * (v[t] - np.einsum("hvk,hk->hv", s, unit_k))
        s = s + delta[:, :, None] * unit_k[:, None, :]
        yield scale * np.einsum("hvk,hk->hv", s, unit_q), s, delta


def row(state, q, *args):
    """One row, with the arguments of tokens(): (outputs [T, H, V], the state
    behind it, sizes [T, H, V]).  A size bounds what an output's sums are made
    of: the largest norm of its row of the state and the deltas that were added
    to it, over the 16 tokens up to it."""
    s = np.array(state, dtype=np.float64)
    out, sizes = np.zeros(q.shape), np.zeros(q.shape)
    norms, deltas = [np.sqrt((s * s).sum(-1))], []
    for t, (out[t], s, delta) in enumerate(tokens(state, q, *args)):
        norms.append(np.sqrt((s * s).sum(-1)))
        deltas.append(np.abs(delta))
        first = max(0, t - 15)
        sizes[t] = np.max(norms[first:t + 2], axis=0) + np.sum(deltas[first:t + 1], axis=0)
    return out, s, sizes


def run(pool, q, k, v, g_raw, beta_raw, a_log, g_bias, cu, slots, initial=None, lower_bound=None,
        scale=None):
    """All rows: (outputs, NaN where no row wrote; the pool; sizes; issues).
    cu None: one token a row."""
    total, h, d = q.shape
    out, sizes = np.full((total, h, d), np.nan), np.zeros((total, h, d))
    after, issues = np.array(pool, dtype=np.float64), []
    for b, slot in enumerate(int(x) for x in slots):
        source = slot if initial is None else int(initial[b])
        first, end = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
        if slot <= 0 or end == first:
            continue
        if end < first or first < 0 or end > total:
            issues.append((b, "length"))
            continue
        if max(slot, source) >= len(pool):
            issues.append((b, "slot"))
            continue
        state = pool[source] if source > 0 else np.zeros(pool.shape[1:])
        at = slice(first, end)
        out[at], after[slot], sizes[at] = row(state, q[at], k[at], v[at], g_raw[at], beta_raw[at],
                                              a_log, g_bias, lower_bound, scale)
    return out, after, sizes, issues


def head_norm(x, weight=None, eps=1e-6):
    """x: [..., D]."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * weight

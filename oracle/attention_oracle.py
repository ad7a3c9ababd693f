"""Oracle of the full-attention layers' part of a speculative step: the cache
append, the window attention and the token log probabilities, in float64 on
the CPU, row by row from their definitions (include/kda.h).  Test
infrastructure only; shares no code with the library.
"""

from __future__ import annotations

import numpy as np


def plan_row(cu, b, computed, width, block_size, num_requests, requests=None, window=None,
             num_tokens=None):
    """(first token, token count, position of the first, request) of row b, or
    the name of what is wrong with it ("" for an empty row)."""
    first, n = int(cu[b]), int(cu[b + 1]) - int(cu[b])
    if n == 0:
        return ""
    if (n < 0 or first < 0 or (window is not None and n > window)
            or (num_tokens is not None and first + n > num_tokens)):
        return "length"
    q = b if requests is None else int(requests[b])
    if not 0 <= q < num_requests:
        return "block"
    c = int(computed[q])
    if c < 0 or (c + n - 1) // block_size >= width:
        return "block"
    return first, n, c, q


def rotate(x, positions, inv_freq, interleaved):
    """x: [n, heads, D]; the first 2 * len(inv_freq) channels turned."""
    out = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = positions.astype(np.float64)[:, None] * float(f)
        c, s = np.cos(angle), np.sin(angle)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def append(q, k, v, keys, values, cu, table, computed, inv_freq=(), interleaved=False,
           requests=None):
    """Returns (q_out, touched, issues): q_out is NaN where no row wrote it,
    keys and values ([blocks, block_size, heads, D] float64) are updated in
    place; touched marks the written (block, token) places."""
    blocks, bs = keys.shape[:2]
    q_out = None if q is None else np.full(q.shape, np.nan)
    touched = np.zeros((blocks, bs), dtype=bool)
    issues = []
    for b in range(len(cu) - 1):
        row = plan_row(cu, b, computed, table.shape[1], bs, table.shape[0], requests,
                       num_tokens=len(k))
        if isinstance(row, str):
            if row:
                issues.append((b, row))
            continue
        first, n, c, r = row
        pos = c + np.arange(n)
        at = slice(first, first + n)
        if q is not None:
            q_out[at] = rotate(q[at], pos, inv_freq, interleaved)
        turned = rotate(k[at], pos, inv_freq, interleaved)
        for t in range(n):
            block = int(table[r, pos[t] // bs])
            if block >= blocks:
                issues.append((b, "slot"))
            elif block > 0:
                keys[block, pos[t] % bs] = turned[t]
                values[block, pos[t] % bs] = v[first + t]
                touched[block, pos[t] % bs] = True
    return q_out, touched, issues


def attend(q, keys, values, cu, table, computed, scale, window=8, left_window=0, requests=None):
    """Returns (out, lse, weight, spread, issues).  weight is sum_j p_j |v_j|
    and spread the largest scale * sum_i |q_i k_i| of a query's keys: what an
    error bound needs.  Rows that are skipped are NaN."""
    blocks, bs = keys.shape[:2]
    heads, dim = q.shape[1:]
    group = heads // keys.shape[2]
    out = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    weight = np.full(q.shape, np.nan)
    spread = np.zeros(q.shape[:2])
    issues = []
    for b in range(len(cu) - 1):
        row = plan_row(cu, b, computed, table.shape[1], bs, table.shape[0], requests, window,
                       len(q))
        if isinstance(row, str):
            if row:
                issues.append((b, row))
            continue
        first, n, c, r = row
        for t in range(n):
            p = c + t
            low = 0 if left_window == 0 else max(0, p - left_window + 1)
            pos = np.arange(low, p + 1)
            block = table[r, pos // bs].astype(np.int64)
            if (block >= blocks).any():
                issues.append((b, "slot"))
            ok = (block > 0) & (block < blocks)
            pos, block = pos[ok], block[ok]
            for h in range(heads):
                kk = keys[block, pos % bs, h // group]
                vv = values[block, pos % bs, h // group]
                score = kk @ q[first + t, h] * scale
                m = score.max() if score.size else -np.inf
                if m == -np.inf:
                    out[first + t, h], lse[first + t, h] = 0.0, -np.inf
                    weight[first + t, h] = 0.0
                    continue
                e = np.exp(score - m)
                total = e.sum()
                out[first + t, h] = e @ vv / total
                weight[first + t, h] = e @ np.abs(vv) / total
                lse[first + t, h] = m + np.log(total)
                spread[first + t, h] = (np.abs(kk) @ np.abs(q[first + t, h])).max() * abs(scale)
    return out, lse, weight, spread, issues


def token_logprobs(logits, tokens, num_top):
    """Returns (logprob, entropy, lse, top_logprob, top_index, mean) from
    float64 logits [rows, vocab]; mean is sum_j p_j |x_j - max|."""
    rows, vocab = logits.shape
    logprob, entropy, lse, mean = (np.zeros(rows) for _ in range(4))
    top_v = np.zeros((rows, num_top))
    top_i = np.zeros((rows, num_top), dtype=np.int64)
    for i in range(rows):
        x = logits[i]
        ranked = np.where(np.isnan(x), -np.inf, x)
        order = np.lexsort((np.arange(vocab), -ranked))[:num_top]
        top_i[i] = order
        if np.isnan(x).any() or (x == np.inf).any():
            logprob[i] = 0.0 if tokens[i] < 0 else np.nan
            entropy[i] = lse[i] = np.nan
            top_v[i] = np.nan
            continue
        m = x.max()
        if m == -np.inf:
            lse[i] = -np.inf
            logprob[i] = 0.0 if tokens[i] < 0 else -np.inf
            top_v[i] = -np.inf
            continue
        e = np.exp(x - m)
        total = e.sum()
        d = np.where(e > 0, x - m, 0.0)
        lse[i] = m + np.log(total)
        mean[i] = -(e * d).sum() / total
        entropy[i] = np.log(total) + mean[i]
        logprob[i] = 0.0 if tokens[i] < 0 else x[tokens[i]] - lse[i]
        top_v[i] = x[order] - lse[i]
    return logprob, entropy, lse, top_v, top_i, mean

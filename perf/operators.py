"""Cases of the operators around the KDA layers of a speculative step.

Three operators, each over the range that serving a hybrid model meets:

- ``append``: rotate the new tokens' queries and keys by position and write
  keys and values to the paged cache (``api.kda_kv_append``);
- ``attend``: attention of a window of 1..8 new tokens per request over the
  paged cache (``api.kda_window_attention``);
- ``logprobs``: log probability of a given token, entropy and the top
  alternatives of each row of logits (``api.kda_token_logprobs``).

``run`` computes them as elementary torch operations, or, with ``own`` set,
through the library.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FAR_BASE = 10000.0   # rotary base of every case


def listed():
    return [
        # one request decodes one token: latency is all there is
        dict(name="append_one", op="append", rows=1, tokens=1, ragged=False, q_heads=8, kv_heads=2,
             head_dim=128, rotary_dim=128, interleaved=False, block_size=16, context=777,
             dtype="bf16"),
        # a decode step of the three-draft workload: 64 requests, 4 tokens each, far positions
        dict(name="append_mtp3", op="append", rows=64, tokens=4, ragged=False, q_heads=32,
             kv_heads=8, head_dim=128, rotary_dim=128, interleaved=False, block_size=16,
             context=131000, dtype="bf16"),
        # prompts of uneven length, half of the channels rotated, pairs side by side
        dict(name="append_prompts", op="append", rows=13, tokens=2501, ragged=True, q_heads=32,
             kv_heads=4, head_dim=128, rotary_dim=64, interleaved=True, block_size=64,
             context=5000, dtype="fp16"),
        # one request, one token, a short context: latency
        dict(name="attend_one", op="attend", rows=1, tokens=1, ragged=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, context=1001, spread=False, left_window=0, dtype="bf16"),
        # the three-draft workload over contexts of very different length
        dict(name="attend_mtp3", op="attend", rows=64, tokens=4, ragged=False, q_heads=32,
             kv_heads=8, head_dim=128, block_size=16, context=8191, spread=True, left_window=0,
             dtype="bf16"),
        # two requests with a very long context: few rows, all parallelism from the length
        dict(name="attend_long", op="attend", rows=2, tokens=8, ragged=False, q_heads=32,
             kv_heads=4, head_dim=128, block_size=64, context=131059, spread=False, left_window=0,
             dtype="fp16"),
        # many requests with ragged windows, a sliding window and small heads
        dict(name="attend_sliding", op="attend", rows=513, tokens=8, ragged=True, q_heads=32,
             kv_heads=4, head_dim=64, block_size=24, context=4099, spread=True, left_window=1000,
             dtype="bf16"),
        # a full batch at eight tokens and eight query heads per key head: the most to compute
        dict(name="attend_wide", op="attend", rows=128, tokens=8, ragged=False, q_heads=64,
             kv_heads=8, head_dim=128, block_size=32, context=12000, spread=True, left_window=0,
             dtype="bf16"),
        # four draft positions of one request
        dict(name="logprobs_few", op="logprobs", rows=4, vocab=32000, top=1, dtype="bf16"),
        # 64 requests of four tokens
        dict(name="logprobs_mtp3", op="logprobs", rows=256, vocab=131072, top=8, dtype="bf16"),
        # an odd vocabulary in fp32: no row but the first starts on 16 bytes
        dict(name="logprobs_odd", op="logprobs", rows=517, vocab=100003, top=20, dtype="fp32"),
        # 1024 requests of four tokens
        dict(name="logprobs_deferred", op="logprobs", rows=4096, vocab=131072, top=0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n < 1000 else min(n | 1, hi)   # large sizes are odd: nothing lines up by chance


def draw(rng):
    """One more case, costing no more than the largest listed one."""
    op = rng.choice(["append", "attend", "attend", "logprobs"])
    if op == "logprobs":
        vocab = _log_int(rng, 4000, 200000)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = min(4096, int(4096 * 131072 / vocab) // (2 if dtype == "fp32" else 1))
        return dict(op=op, rows=_log_int(rng, 1, most), vocab=vocab,
                    top=rng.choice([0, 1, 5, 8, 20, 32]), dtype=dtype)
    head_dim = rng.choice([128, 128, 64])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8, 16] if head_dim == 128 else [1, 3, 4, 8])
    q_heads = group * kv_heads
    block_size = rng.choice([16, 24, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        width = (q_heads + 2 * kv_heads) * head_dim
        rows = _log_int(rng, 1, 256)
        most = max(1, min(4096, 16_000 * 40 * 128 // (rows * max(width, 1024))))
        return dict(op=op, rows=rows, tokens=_log_int(rng, 1, most), ragged=rng.random() < 0.5,
                    q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                    rotary_dim=rng.choice([head_dim, head_dim // 2, 32]),
                    interleaved=rng.random() < 0.5, block_size=block_size,
                    context=_log_int(rng, 1, 500_000), dtype=dtype)
    tokens = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    rows = _log_int(rng, 1, 600)
    # keys x kv heads, and the plain form's scores, stay inside the largest listed case's
    spread = rng.random() < 0.7
    most = 128 * 12000 if spread else 128 * 6500
    keys = min(most * 8 * 128 // (rows * kv_heads * head_dim),
               most * 64 * 8 // (rows * q_heads * tokens))
    return dict(op=op, rows=rows, tokens=tokens, ragged=rng.random() < 0.5, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
                context=_log_int(rng, 1, max(2, min(200_000, keys))), spread=spread,
                left_window=rng.choice([0, 0, 0, 128, 1024]), dtype=dtype)


def _spread(n, lo, hi):
    """n whole numbers over lo..hi, evenly mixed; they belong to the case, not to the seed."""
    return [lo + int(((i + 0.5) * 0.6180339887498949) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lens(case):
    return _spread(case["rows"], 1, case["tokens"]) if case["ragged"] else [case["tokens"]] * case["rows"]


def _contexts(case):
    """Tokens computed before this step, for each row."""
    if case["op"] == "append" or case["spread"]:
        return _spread(case["rows"], case["context"] // 8, case["context"])
    return [case["context"]] * case["rows"]


def _first_key(case, c):
    return max(0, c + 1 - case["left_window"]) if case.get("left_window") else 0


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * DTYPES[case["dtype"]].itemsize + case["rows"] * (16 + 8 * case["top"]),
                    flops=6 * n)
    lens, d = _lens(case), case["head_dim"]
    tokens = sum(lens)
    if case["op"] == "append":
        return dict(bytes=4 * tokens * (case["q_heads"] + 2 * case["kv_heads"]) * d,
                    flops=3 * tokens * (case["q_heads"] + case["kv_heads"]) * case["rotary_dim"])
    keys = [c + t - _first_key(case, c) for c, t in zip(_contexts(case), lens)]
    return dict(bytes=4 * sum(keys) * case["kv_heads"] * d + tokens * case["q_heads"] * (4 * d + 4),
                flops=4 * d * case["q_heads"] * sum(n * t for n, t in zip(keys, lens)))


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "logprobs":
        n, v = case["rows"], case["vocab"]
        logits = torch.empty((n, v), dtype=dtype, device=dev)
        for at in range(0, n, 512):
            part = torch.randn((min(512, n - at), v), generator=gen, device=dev)
            # a few tokens stand out, as they do where a model is sure of itself
            logits[at:at + 512] = (part * 2.5 + 4.0 * (part > 3.5)).to(dtype)
        tokens = torch.randint(0, v, (n,), generator=gen, device=dev, dtype=torch.int32)
        sure = torch.rand(n, generator=gen, device=dev) < 0.7
        tokens = torch.where(sure, logits.argmax(1).to(torch.int32), tokens)
        return dict(case=case, logits=logits, tokens=tokens)
    rows, hq, hk, d, bs = (case[x] for x in ("rows", "q_heads", "kv_heads", "head_dim", "block_size"))
    lens, before = _lens(case), _contexts(case)
    total = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    computed = torch.tensor(before, dtype=torch.int32, device=dev)
    width = max((c + t + bs - 1) // bs for c, t in zip(before, lens))
    # the blocks that this step reads or writes are real, all others are the null block 0
    table = np.zeros((rows, width), dtype=np.int32)
    spans = []
    for c, t in zip(before, lens):
        first = (c if case["op"] == "append" else _first_key(case, c)) // bs
        spans.append((first, (c + t + bs - 1) // bs))
    blocks = 1 + sum(e - s for s, e in spans)
    order = torch.randperm(blocks - 1, generator=gen, device=dev).cpu().numpy().astype(np.int32) + 1
    at = 0
    for i, (s, e) in enumerate(spans):
        table[i, s:e] = order[at:at + e - s]
        at += e - s
    key_cache = torch.empty((blocks, bs, hk, d), dtype=dtype, device=dev)
    value_cache = torch.empty((blocks, bs, hk, d), dtype=dtype, device=dev)
    step = max(1, (1 << 28) // (bs * hk * d))
    for cache in (key_cache, value_cache):
        for i in range(0, blocks, step):
            cache[i:i + step].normal_(generator=gen)
    # q, k and v are views of one merged projection, which has a slice of another use behind them
    merged = torch.randn((total, hq + 2 * hk + 1, d), generator=gen, device=dev).to(dtype)
    state = dict(case=case, q=merged[:, :hq], k=merged[:, hq:hq + hk], v=merged[:, hq + hk:hq + 2 * hk],
                 key_cache=key_cache, value_cache=value_cache, cu_seqlens=cu,
                 block_table=torch.from_numpy(table).to(dev), num_computed=computed)
    if case["op"] == "append":
        r = case["rotary_dim"]
        state["inv_freq"] = torch.tensor([FAR_BASE ** (-2.0 * i / r) for i in range(r // 2)],
                                         dtype=torch.float64, device=dev)
    return state


# ------------------------------------------------------------------ passes --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "attend": _attend_own, "logprobs": _logprobs_own}[op](state)
    return {"append": _append_plain, "attend": _attend_plain, "logprobs": _logprobs_plain}[op](state)


def _append_own(s):
    from linear_attention_speculative_kda_gb300 import api
    q = api.kda_kv_append(s["q"], s["k"], s["v"], s["key_cache"], s["value_cache"],
                          s["cu_seqlens"], s["block_table"], s["num_computed"],
                          inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
    return q, s["key_cache"], s["value_cache"]


def _attend_own(s):
    from linear_attention_speculative_kda_gb300 import api
    if "workspace" not in s:   # kept from call to call, as a serving loop does
        s["workspace"] = api.allocate_attention_workspace(
            s["case"]["rows"], s["case"]["q_heads"], s["case"]["kv_heads"], s["case"]["head_dim"],
            s["q"].device)
    return api.kda_window_attention(s["q"], s["key_cache"], s["value_cache"], s["cu_seqlens"],
                                    s["block_table"], s["num_computed"], s["workspace"],
                                    window=s["case"]["tokens"],
                                    left_window=s["case"]["left_window"])


def _logprobs_own(s):
    from linear_attention_speculative_kda_gb300 import api
    return tuple(api.kda_token_logprobs(s["logits"], s["tokens"], num_top=s["case"]["top"]))


def _rows_of_tokens(s):
    """Each token's row and its index in the row."""
    total = s["q"].shape[0]
    lens = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens,
                                  output_size=total)
    return row, torch.arange(total, device=lens.device) - s["cu_seqlens"][row]


def _rotate(x, cos, sin, interleaved):
    """x: [T, H, D] in fp32; cos, sin: [T, 1, R/2]."""
    r = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, x[..., r:]], dim=-1)


def _append_plain(s):
    case, dtype = s["case"], s["q"].dtype
    row, t = _rows_of_tokens(s)
    position = s["num_computed"][row].long() + t
    angle = position.double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, case["interleaved"]).to(dtype)
    k = _rotate(s["k"].float(), cos, sin, case["interleaved"]).to(dtype)
    bs = case["block_size"]
    block = s["block_table"][row, position // bs].long()
    s["key_cache"][block, position % bs] = k
    s["value_cache"][block, position % bs] = s["v"]
    return q, s["key_cache"], s["value_cache"]


def _attend_plain(s):
    case = s["case"]
    hq, hk, d, bs, w = (case[x] for x in ("q_heads", "kv_heads", "head_dim", "block_size", "tokens"))
    rows, g = case["rows"], hq // hk
    dev = s["q"].device
    row, t = _rows_of_tokens(s)
    longest = s["block_table"].shape[1] * bs
    pos = torch.arange(longest, device=dev)
    block = s["block_table"][:, pos // bs].long()                       # [B, L]
    c = s["num_computed"].long()[:, None, None]
    at = c + torch.arange(w, device=dev)[:, None]                       # [B, W, 1]
    seen = (block > 0)[:, None] & (pos <= at)                           # [B, W, L]
    if case["left_window"]:
        seen = seen & (pos > at - case["left_window"])
    q = torch.zeros((rows, w, hk, g, d), device=dev)
    q[row, t] = s["q"].float().view(-1, hk, g, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(rows, hk, w * g, d)
    k = s["key_cache"][block, pos % bs].permute(0, 2, 3, 1).float()     # [B, Hk, D, L]
    score = torch.matmul(q, k).mul_(d ** -0.5)
    del k
    score = score.view(rows, hk, w, g, longest).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["value_cache"][block, pos % bs].permute(0, 2, 1, 3).float()   # [B, Hk, L, D]
    o = torch.matmul(p.view(rows, hk, w * g, longest), v).view(rows, hk, w, g, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)                               # [B, Hk, W, G]
    o = o.permute(0, 2, 1, 3, 4)[row, t].reshape(-1, hq, d).to(s["q"].dtype)
    return o, lse.permute(0, 2, 1, 3)[row, t].reshape(-1, hq).contiguous()


def _logprobs_plain(s):
    x = s["logits"].float()
    n, v = x.shape
    top = x.amax(1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    lse = (top + total.log()).squeeze(1)
    # log total - mean of (x - top); a masked logit (-inf) weighs nothing
    mean = torch.where(e > 0, e * (x - top), torch.zeros_like(x)).sum(1) / total.squeeze(1)
    entropy = total.log().squeeze(1) - mean
    logprob = x.gather(1, s["tokens"].long()[:, None]).squeeze(1) - lse
    k = s["case"]["top"]
    del e
    index = torch.empty((n, 0), dtype=torch.int64, device=x.device)
    if k:
        # one whole number per logit that orders by value, then by the lower index: no ties
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
        order += torch.arange(v - 1, -1, -1, device=x.device)
        index = order.topk(k, dim=1).indices
    return (logprob, entropy, lse, x.gather(1, index) - lse[:, None], index.to(torch.int32))


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _logprobs_exact(s)
    if case["op"] == "append":
        return _append_exact(s)
    return _attend_exact(s)


def _logprobs_exact(s):
    found = []
    k = s["case"]["top"]
    for x, token in zip(s["logits"].split(64), s["tokens"].long().split(64)):
        x = x.double()
        logp = torch.log_softmax(x, dim=1)
        entropy = -(logp.exp() * logp).sum(1)
        at = torch.arange(x.shape[0], device=x.device)
        # a stable sort keeps the lower index first among equals
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k] if k else x[:, :0].long()
        found.append((logp[at, token], entropy, torch.logsumexp(x, dim=1), logp.gather(1, order),
                      order.to(torch.int32)))
    return tuple(torch.cat(part) for part in zip(*found))


def _append_exact(s):
    case = s["case"]
    cu, before = s["cu_seqlens"].cpu().tolist(), s["num_computed"].cpu().tolist()
    q = s["q"].double()
    keys, values = s["key_cache"].double(), s["value_cache"].double()
    r, bs = case["rotary_dim"], case["block_size"]
    i = torch.arange(r // 2, device=q.device)
    one, other = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    for b in range(case["rows"]):
        at = slice(cu[b], cu[b + 1])
        pos = before[b] + torch.arange(cu[b + 1] - cu[b], device=q.device)
        # rotation as a product of complex numbers
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=q.device),
                           pos.double()[:, None] * s["inv_freq"])[:, None]
        k = s["k"][at].double()
        for x in (q[at], k):
            z = torch.complex(x[..., one], x[..., other]) * turn
            x[..., one], x[..., other] = z.real, z.imag
        block = s["block_table"][b].long()[pos // bs]
        keys[block, pos % bs] = k
        values[block, pos % bs] = s["v"][at].double()
    return q, keys, values


def _attend_exact(s):
    case = s["case"]
    hq, hk, d, bs = (case[x] for x in ("q_heads", "kv_heads", "head_dim", "block_size"))
    cu, before = s["cu_seqlens"].cpu().tolist(), s["num_computed"].cpu().tolist()
    outs, lses = [], []
    for b in range(case["rows"]):
        n = cu[b + 1] - cu[b]
        first = _first_key(case, before[b]) // bs
        blocks = s["block_table"][b, first:(before[b] + n + bs - 1) // bs].long()
        k = s["key_cache"][blocks].reshape(-1, hk, d).double()
        v = s["value_cache"][blocks].reshape(-1, hk, d).double()
        q = s["q"][cu[b]:cu[b + 1]].double().view(n, hk, hq // hk, d)
        key = torch.arange(first * bs, first * bs + k.shape[0], device=k.device)
        behind = before[b] + torch.arange(n, device=k.device)[:, None] - key
        hidden = behind < 0
        if case["left_window"]:
            hidden = hidden | (behind >= case["left_window"])
        score = torch.einsum("nhgd,lhd->hgnl", q, k) / math.sqrt(d)
        score = score.masked_fill(hidden, -math.inf)
        lse = torch.logsumexp(score, dim=-1)
        o = torch.einsum("hgnl,lhd->nhgd", (score - lse[..., None]).exp(), v)
        outs.append(o.reshape(n, hq, d))
        lses.append(lse.permute(2, 0, 1).reshape(n, hq))
    return torch.cat(outs), torch.cat(lses)

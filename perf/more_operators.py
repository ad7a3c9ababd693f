"""Cases of the operators that admit prompts and decode single tokens.

Three operators, each over the range that serving a hybrid model meets:

- ``prefill``: the gated delta rule over rows of any length, chunked, from a
  state of the pool or from none (``api.kda_prefill``);
- ``decode``: the same for one token a row (``api.kda_decode``);
- ``norm_append``: norms of each head's queries and keys, their rotation by
  position and the append to the paged cache (``api.kda_kv_norm_append``).

``run`` computes them as elementary torch operations, or, with ``own`` set,
through the library.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DIM = 128            # channels of a head of the delta rule
PIECE = 16           # tokens that the plain form takes at once
NORM_EPS = 1e-6
ROTARY_BASE = 10000.0


def listed():
    return [
        # one short prompt: latency is all there is
        dict(name="prefill_one", op="prefill", rows=1, tokens=37, mix="even", heads=16, resumed=False,
             lower_bound=0.0),
        # one long prompt: the only parallel work is its heads
        dict(name="prefill_long", op="prefill", rows=1, tokens=16001, mix="even", heads=32,
             resumed=False, lower_bound=0.0),
        # prompts of uneven length with the bounded gate; some go on from a cached prefix
        dict(name="prefill_ragged", op="prefill", rows=13, tokens=2501, mix="ragged", heads=16,
             resumed=True, lower_bound=-5.0),
        # pieces of a few prompts in one batch with many rows of a few tokens
        dict(name="prefill_mixed", op="prefill", rows=200, tokens=1501, mix="few", heads=16,
             resumed=True, lower_bound=0.0),
        # short turns of many conversations: the states are most of the bytes
        dict(name="prefill_turns", op="prefill", rows=256, tokens=45, mix="ragged", heads=32,
             resumed=True, lower_bound=-5.0),
        # a full batch of prompts: the most to compute
        dict(name="prefill_batch", op="prefill", rows=64, tokens=1024, mix="even", heads=32,
             resumed=False, lower_bound=0.0),
        # one request decodes one token
        dict(name="decode_one", op="decode", rows=1, heads=32, lower_bound=0.0),
        # the three-draft workload's batch without drafts
        dict(name="decode_mtp3", op="decode", rows=64, heads=32, lower_bound=-5.0),
        # the deferred workload's batch without drafts
        dict(name="decode_deferred", op="decode", rows=1024, heads=16, lower_bound=0.0),
        # one request decodes one token
        dict(name="norm_append_one", op="norm_append", rows=1, tokens=1, ragged=False, q_heads=8,
             kv_heads=2, head_dim=128, rotary_dim=128, interleaved=False, block_size=16,
             context=777, dtype="bf16", weights="bf16"),
        # a decode step of the three-draft workload, far positions
        dict(name="norm_append_mtp3", op="norm_append", rows=64, tokens=4, ragged=False, q_heads=32,
             kv_heads=8, head_dim=128, rotary_dim=128, interleaved=False, block_size=16,
             context=131000, dtype="bf16", weights="fp32"),
        # prompts of uneven length, half of the channels rotated, pairs side by side
        dict(name="norm_append_prompts", op="norm_append", rows=13, tokens=2501, ragged=True,
             q_heads=32, kv_heads=4, head_dim=128, rotary_dim=64, interleaved=True, block_size=64,
             context=5000, dtype="fp16", weights="fp16"),
    ]


def _log_int(rng, lo, hi):
    hi = max(lo, hi)
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n if n < 1000 else min(n | 1, hi)   # large sizes are odd: nothing lines up by chance


def draw(rng):
    """One more case, costing no more than the largest listed one."""
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "norm_append"])
    if op == "norm_append":
        head_dim = rng.choice([128, 128, 64])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 4, 7, 8, 16] if head_dim == 128 else [1, 3, 4, 8])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        rows = _log_int(rng, 1, 256)
        width = (q_heads + 2 * kv_heads) * head_dim
        most = max(1, min(4096, 16_000 * 40 * 128 // (rows * max(width, 1024))))
        return dict(op=op, rows=rows, tokens=_log_int(rng, 1, most), ragged=rng.random() < 0.5,
                    q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                    rotary_dim=rng.choice([head_dim, head_dim // 2, 32]),
                    interleaved=rng.random() < 0.5, block_size=rng.choice([16, 24, 32, 64, 128]),
                    context=_log_int(rng, 1, 500_000), dtype=dtype,
                    weights=rng.choice([dtype, "fp32"]))
    heads = rng.choice([1, 2, 3, 4, 7, 8, 12, 16, 32])
    bound = rng.choice([0.0, -5.0])
    if op == "decode":
        return dict(op=op, rows=_log_int(rng, 1, 1024 * 16 // heads if heads > 16 else 1024),
                    heads=heads, lower_bound=bound)
    rows = _log_int(rng, 1, min(256, 8192 // heads))
    # tokens x heads stay inside the largest listed case's, rows padded to the longest; a row's
    # states weigh as much as 103 of its tokens
    most = min(16_000, 64 * 1024 * 32 // (rows * heads) - 103)
    return dict(op=op, rows=rows, tokens=_log_int(rng, 1, most),
                mix=rng.choice(["even", "ragged", "ragged", "few"]), heads=heads,
                resumed=rng.random() < 0.5, lower_bound=bound)


def _spread(n, lo, hi):
    """n whole numbers over lo..hi, evenly mixed; they belong to the case, not to the seed."""
    return [lo + int(((i + 0.5) * 0.6180339887498949) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lens(case):
    rows = case["rows"]
    if case["op"] == "norm_append":
        return _spread(rows, 1, case["tokens"]) if case["ragged"] else [case["tokens"]] * rows
    if case["mix"] == "even":
        return [case["tokens"]] * rows
    if case["mix"] == "ragged":
        return _spread(rows, 1, case["tokens"])
    # one row in forty is long, the others have 1 to 8 tokens
    short = _spread(rows, 1, min(8, case["tokens"]))
    return [case["tokens"] if i % 40 == 7 else n for i, n in enumerate(short)]


def _starts(case):
    """Which rows go on from a state."""
    if case["op"] == "decode":
        return [True] * case["rows"]
    return [case["resumed"] and i % 3 != 1 for i in range(case["rows"])]


def _contexts(case):
    return _spread(case["rows"], case["context"] // 8, case["context"])


def work(case):
    if case["op"] == "norm_append":
        lens, d = _lens(case), case["head_dim"]
        heads = case["q_heads"] + case["kv_heads"]
        return dict(bytes=4 * sum(lens) * (heads + case["kv_heads"]) * d,
                    flops=sum(lens) * heads * (4 * d + 3 * case["rotary_dim"]))
    tokens = case["rows"] if case["op"] == "decode" else sum(_lens(case))
    h, tile = case["heads"], DIM * DIM
    return dict(bytes=tokens * h * (5 * 2 * DIM + 2) + 4 * tile * h * (sum(_starts(case)) + case["rows"]),
                flops=7 * tile * tokens * h)


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "norm_append":
        return _prepare_append(case, gen, dev)
    rows, h = case["rows"], case["heads"]
    lens = [1] * rows if case["op"] == "decode" else _lens(case)
    total = sum(lens)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev)

    # q, k and v are views of one merged projection, as the layer makes them
    merged = torch.empty((total, 3, h, DIM), dtype=torch.bfloat16, device=dev)
    gate = torch.empty((total, h, DIM), dtype=torch.bfloat16, device=dev)
    for at in range(0, total, 8192):
        end = min(total, at + 8192)
        merged[at:end] = normal(end - at, 3, h, DIM).to(torch.bfloat16)
        gate[at:end] = normal(end - at, h, DIM).to(torch.bfloat16)
    # steps of 0.001 to 0.1 where the gate's input is 0: memories of a few to some thousand tokens
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), h * DIM))
    slots = 2 * rows + 1
    order = torch.randperm(slots - 1, generator=gen, device=dev).to(torch.int32) + 1
    starts = torch.tensor(_starts(case), device=dev)
    pool = torch.empty((slots, h, DIM, DIM), device=dev)
    for at in range(0, slots, 64):
        pool[at:at + 64].normal_(0.0, 0.05, generator=gen)
    return dict(
        case=case, q=merged[:, 0], k=merged[:, 1], v=merged[:, 2], g_raw=gate,
        beta_raw=normal(total, h + 8).to(torch.bfloat16)[:, :h],
        A_log=uniform(0.0, 2.7, h), g_bias=torch.log(torch.expm1(step)), pool=pool,
        cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev),
        # a row's state comes from one block of the pool and goes to another, as with cached prefixes
        initial=torch.where(starts, order[:rows], torch.zeros_like(order[:rows])),
        slots=order[rows:].contiguous(), longest=max(lens),
        lower_bound=case["lower_bound"] if case["lower_bound"] < 0 else None)


def _prepare_append(case, gen, dev):
    dtype = DTYPES[case["dtype"]]
    rows, hq, hk, d, bs = (case[x] for x in ("rows", "q_heads", "kv_heads", "head_dim", "block_size"))
    lens, before = _lens(case), _contexts(case)
    total = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    width = max((c + t + bs - 1) // bs for c, t in zip(before, lens))
    table = np.zeros((rows, width), dtype=np.int32)     # blocks that the step does not write: null
    spans = [(c // bs, (c + t + bs - 1) // bs) for c, t in zip(before, lens)]
    blocks = 1 + sum(e - s for s, e in spans)
    order = torch.randperm(blocks - 1, generator=gen, device=dev).cpu().numpy().astype(np.int32) + 1
    at = 0
    for i, (s, e) in enumerate(spans):
        table[i, s:e] = order[at:at + e - s]
        at += e - s
    caches = [torch.randn((blocks, bs, hk, d), generator=gen, device=dev).to(dtype) for _ in range(2)]
    # some heads are far larger than others, as they are before a norm
    size = torch.exp(1.5 * torch.randn((1, hq + 2 * hk + 1, 1), generator=gen, device=dev))
    merged = (size * torch.randn((total, hq + 2 * hk + 1, d), generator=gen, device=dev)).to(dtype)
    weights = [(1.0 + 0.3 * torch.randn(d, generator=gen, device=dev)).to(DTYPES[case["weights"]])
               for _ in range(2)]
    r = case["rotary_dim"]
    freq = torch.tensor([ROTARY_BASE ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64,
                        device=dev)
    return dict(case=case, q=merged[:, :hq], k=merged[:, hq:hq + hk], v=merged[:, hq + hk:hq + 2 * hk],
                key_cache=caches[0], value_cache=caches[1], cu_seqlens=cu,
                block_table=torch.from_numpy(table).to(dev),
                num_computed=torch.tensor(before, dtype=torch.int32, device=dev),
                q_weight=weights[0], k_weight=weights[1], inv_freq=freq)


# ------------------------------------------------------------------ passes --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"prefill": _prefill_own, "decode": _decode_own, "norm_append": _append_own}[op](state)
    return {"prefill": _prefill_plain, "decode": _decode_plain, "norm_append": _append_plain}[op](state)


def _prefill_own(s):
    from linear_attention_speculative_kda_gb300 import api
    out = api.kda_prefill(s["q"], s["k"], s["v"], s["g_raw"], s["beta_raw"], s["A_log"], s["g_bias"],
                          s["pool"], s["cu_seqlens"], s["slots"], initial_indices=s["initial"],
                          lower_bound=s["lower_bound"])
    return out, s["pool"]


def _decode_own(s):
    from linear_attention_speculative_kda_gb300 import api
    out = api.kda_decode(s["q"], s["k"], s["v"], s["g_raw"], s["beta_raw"], s["A_log"], s["g_bias"],
                         s["pool"], s["slots"], initial_indices=s["initial"],
                         lower_bound=s["lower_bound"])
    return out, s["pool"]


def _append_own(s):
    from linear_attention_speculative_kda_gb300 import api
    q = api.kda_kv_norm_append(s["q"], s["k"], s["v"], s["key_cache"], s["value_cache"],
                               s["cu_seqlens"], s["block_table"], s["num_computed"],
                               q_weight=s["q_weight"], k_weight=s["k_weight"], eps=NORM_EPS,
                               inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
    return q, s["key_cache"], s["value_cache"]


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _inputs(s):
    """Unit queries and keys, values, log decays and betas of every token in fp32."""
    x = s["g_raw"].float() + s["g_bias"].view(-1, DIM)
    a = s["A_log"].exp()[:, None]
    if s["lower_bound"] is not None:
        g = s["lower_bound"] / (1.0 + (-a * x).exp())
    else:
        z = (-x.abs()).exp()
        g = -a * (x.clamp_min(0.0) + torch.log1p(z))
    beta = 1.0 / (1.0 + (-s["beta_raw"].float()).exp())
    return _unit(s["q"].float()), _unit(s["k"].float()), s["v"].float(), g, beta


def _rows_of_tokens(cu, total):
    """Each token's row and its index in the row."""
    lens = (cu[1:] - cu[:-1]).long()
    row = torch.repeat_interleave(torch.arange(lens.numel(), device=cu.device), lens, output_size=total)
    return row, torch.arange(total, device=cu.device) - cu[row]


def _first_states(s):
    initial = s["initial"].long()
    return s["pool"][initial] * (initial > 0)[:, None, None, None]


def _decode_plain(s):
    q, k, v, g, beta = _inputs(s)
    state = _first_states(s) * g.exp()[:, :, None, :]                       # [B, H, V, K]
    delta = beta[..., None] * (v - torch.matmul(state, k[..., None]).squeeze(-1))
    state = state + delta[..., None] * k[:, :, None, :]
    s["pool"][s["slots"].long()] = state
    out = torch.matmul(state, q[..., None]).squeeze(-1) * DIM ** -0.5
    return out.to(torch.bfloat16), s["pool"]


def _prefill_plain(s):
    """Pieces of 16 tokens of all rows and heads: what a piece adds to itself comes from the decays
    between its tokens, what came before it from the state."""
    rows, h, total = s["case"]["rows"], s["case"]["heads"], s["q"].shape[0]
    c = min(PIECE, s["longest"])
    pieces = (s["longest"] + c - 1) // c
    row, t = _rows_of_tokens(s["cu_seqlens"], total)
    dev = s["q"].device

    def padded(x):   # [B, pieces, H, C, ...], zeros behind a row's end: no decay, nothing written
        full = torch.zeros((rows, pieces * c) + x.shape[1:], device=dev)
        full[row, t] = x
        return full.view((rows, pieces, c) + x.shape[1:]).transpose(2, 3)

    q, k, v, g, beta = (padded(x) for x in _inputs(s))
    at = torch.arange(c, device=dev)
    # sums of log decays over the tokens behind s up to t, and of all up to t or behind s
    between = ((at > at[None, :, None]) & (at <= at[:, None, None])).float()     # [t, s, i]
    upto, behind = between.new_ones(c, c).tril(), between.new_ones(c, c).triu(1)
    below = upto - torch.eye(c, device=dev)
    state = _first_states(s)
    out = torch.empty((rows, pieces, h, c, DIM), device=dev)
    for i in range(pieces):
        qi, ki, vi, gi, bi = q[:, i], k[:, i], v[:, i], g[:, i], beta[:, i, :, :, None]
        decay = torch.matmul(between.view(c * c, c), gi).exp_().view(rows, h, c, c, DIM)
        keys = decay * ki[:, :, None]                                            # [B, H, t, s, K]
        inner = torch.matmul(keys, ki[..., None]).squeeze(-1) * below * bi
        cross = torch.matmul(keys, qi[..., None]).squeeze(-1) * upto
        reach = torch.matmul(upto, gi).exp_()
        old = torch.matmul(torch.cat([ki * reach, qi * reach], dim=2), state.mT)  # [B, H, 2 C, V]
        delta = bi * (vi - old[:, :, :c])
        # (1 + N)^-1 = (1 - N)(1 + N^2)(1 + N^4)..., N strictly below the diagonal
        power, step = inner, 1
        delta = delta - torch.matmul(inner, delta)
        while 2 * step < c:
            power, step = torch.matmul(power, power), 2 * step
            delta = delta + torch.matmul(power, delta)
        out[:, i] = old[:, :, c:] + torch.matmul(cross, delta)
        left = torch.matmul(behind, gi).exp_()
        state = state * reach[:, :, -1:] + torch.matmul(delta.mT, ki * left)
    s["pool"][s["slots"].long()] = state
    out = out.transpose(2, 3).reshape(rows, pieces * c, h, DIM)[row, t] * DIM ** -0.5
    return out.to(torch.bfloat16), s["pool"]


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
    row, t = _rows_of_tokens(s["cu_seqlens"], s["q"].shape[0])
    position = s["num_computed"][row].long() + t
    angle = position.double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()

    def normed(x, weight):
        x = x.float()
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * weight.float()

    q = _rotate(normed(s["q"], s["q_weight"]), cos, sin, case["interleaved"]).to(dtype)
    k = _rotate(normed(s["k"], s["k_weight"]), cos, sin, case["interleaved"]).to(dtype)
    bs = case["block_size"]
    block = s["block_table"][row, position // bs].long()
    s["key_cache"][block, position % bs] = k
    s["value_cache"][block, position % bs] = s["v"]
    return q, s["key_cache"], s["value_cache"]


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    return _append_exact(s) if case["op"] == "norm_append" else _delta_exact(s)


def _delta_exact(s):
    """Token by token, all rows that have one at a time."""
    cu = s["cu_seqlens"].cpu().tolist()
    lens = [e - b for b, e in zip(cu, cu[1:])]
    dev = s["q"].device
    a, bias = torch.exp(s["A_log"].double())[:, None], s["g_bias"].double().view(-1, DIM)
    # longest rows first, so that those with a token t are always the first ones
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    first = torch.tensor([cu[b] for b in order], device=dev)
    source = s["initial"].long()[order]
    state = s["pool"].double()[source]
    state[source <= 0] = 0.0
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    alive = len(order)
    for t in range(s["longest"]):
        while lens[order[alive - 1]] <= t:
            alive -= 1
        at = first[:alive] + t
        x = s["g_raw"][at].double() + bias
        if s["lower_bound"] is None:
            g = -a * torch.nn.functional.softplus(x, threshold=40.0)
        else:
            g = s["lower_bound"] * torch.sigmoid(a * x)
        q, k = s["q"][at].double(), s["k"][at].double()
        q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + 1e-6) / math.sqrt(DIM)
        k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + 1e-6)
        now = state[:alive]
        now.mul_(torch.exp(g)[:, :, None, :])
        guess = torch.einsum("bhvk,bhk->bhv", now, k)
        now.add_(torch.einsum("bhv,bhk->bhvk", torch.sigmoid(s["beta_raw"][at].double())[..., None]
                              * (s["v"][at].double() - guess), k))
        out[at] = torch.einsum("bhvk,bhk->bhv", now, q)
    pool = s["pool"].double()
    pool[s["slots"].long()[order]] = state
    return out, pool


def _append_exact(s):
    case = s["case"]
    cu, before = s["cu_seqlens"].cpu().tolist(), s["num_computed"].cpu().tolist()

    def normed(x, weight):
        return x * torch.rsqrt(x.square().sum(-1, keepdim=True) / case["head_dim"] + NORM_EPS) * weight

    q = normed(s["q"].double(), s["q_weight"].double())
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
        k = normed(s["k"][at].double(), s["k_weight"].double())
        for x in (q[at], k):
            z = torch.complex(x[..., one], x[..., other]) * turn
            x[..., one], x[..., other] = z.real, z.imag
        block = s["block_table"][b].long()[pos // bs]
        keys[block, pos % bs] = k
        values[block, pos % bs] = s["v"][at].double()
    return q, keys, values

"""Speculative steps of a small hybrid model: a KDA layer, a full-attention
layer and the acceptance of the drafts, all through the library.

Each step runs a window of 1 + num_spec tokens per request (the last accepted
token and the drafts behind it):

    kda_verify            the KDA layer from each request's checkpoint state
    kda_kv_append         rotated keys and values of the window to the paged cache
    kda_window_attention  the window over its request's keys and values
    kda_token_logprobs    the target's choice at every position
    kda_commit            the accepted tokens into the checkpoint state

A draft is accepted while it is what the target would have chosen.  Rejected
tokens need no rollback: their keys and values lie past the new num_computed
and the next step's append overwrites them, and the checkpoint only ever takes
accepted tokens.  Weights are random, projections and the output head plain
torch products; the drafts are random too, but for the first of each request,
so that some are accepted.

    python examples/hybrid_step.py
"""

from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_speculative_kda_gb300 import api  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


@dataclass(frozen=True)
class Sizes:
    requests: int = 5
    window: int = 4          # 1 + num_spec
    vocab: int = 1000
    width: int = 256         # of the residual stream
    kda_heads: int = 2
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    block_size: int = 16
    max_len: int = 200       # tokens a request may reach


class HybridModel:
    """One KDA layer and one full-attention layer with random weights, and
    the serving state of ``sizes.requests`` requests."""

    def __init__(self, sizes: Sizes, device="cuda", seed: int = 0):
        s, d = sizes, torch.device(device)
        gen = torch.Generator().manual_seed(seed)
        self.sizes, self.device = sizes, d

        def weight(*shape):
            return (torch.randn(shape, generator=gen) * shape[0] ** -0.5).to(BF16).to(d)
        kda = s.kda_heads * 128
        self.embed = (torch.randn((s.vocab, s.width), generator=gen)).to(BF16).to(d)
        self.w_qkv, self.w_gate = weight(s.width, 3 * kda), weight(s.width, kda)
        self.w_beta, self.w_kda_out = weight(s.width, s.kda_heads), weight(kda, s.width)
        self.w_merged = weight(s.width, (s.q_heads + 2 * s.kv_heads) * s.head_dim)
        self.w_out = weight(s.q_heads * s.head_dim, s.width)
        self.w_head = weight(s.width, s.vocab)
        self.A_log = torch.rand(s.kda_heads, generator=gen).to(d)
        self.g_bias = (torch.randn(kda, generator=gen) * 0.1).to(d)
        # serving state: a KDA checkpoint per request (slot 0 is the null
        # block) and its records, and the attention layer's paged cache
        self.pool = torch.zeros((s.requests + 1, s.kda_heads, 128, 128), device=d)
        self.slots = torch.arange(1, s.requests + 1, dtype=I32, device=d)
        self.records = api.allocate_records(s.kda_heads, s.window, s.requests, d)
        per_request = (s.max_len + s.block_size - 1) // s.block_size
        blocks = torch.randperm(s.requests * per_request, generator=gen) + 1
        self.block_table = blocks.view(s.requests, per_request).to(I32).to(d)
        cache = (s.requests * per_request + 1, s.block_size, s.kv_heads, s.head_dim)
        self.key_cache = torch.zeros(cache, dtype=BF16, device=d)
        self.value_cache = torch.zeros(cache, dtype=BF16, device=d)
        self.num_computed = torch.zeros(s.requests, dtype=I32, device=d)
        self.inv_freq = 10000.0 ** (-torch.arange(0, s.head_dim, 2, dtype=torch.float64, device=d)
                                    / s.head_dim)
        self.workspace = api.allocate_attention_workspace(s.requests, s.q_heads, s.kv_heads,
                                                          s.head_dim, d, window=s.window)
        self.cu_seqlens = torch.arange(0, (s.requests + 1) * s.window, s.window, dtype=I32,
                                       device=d)
        self.error_word = torch.zeros(1, dtype=I32, device=d)

    def verify(self, tokens: torch.Tensor) -> api.TokenLogprobs:
        """The target's view of a window of tokens int32 [requests, window]:
        at every position the log probability of the token that follows in
        the window (0 at the last), the entropy and the target's own choice."""
        s = self.sizes
        total = tokens.numel()
        rows = dict(window=s.window, error_word=self.error_word)
        x = self.embed[tokens.flatten().long()]
        # KDA layer
        qkv = (x @ self.w_qkv).view(total, 3, s.kda_heads, 128)
        gate = (x @ self.w_gate).view(total, s.kda_heads, 128)
        y = torch.empty((total, s.kda_heads, 128), dtype=BF16, device=self.device)
        api.kda_verify(qkv[:, 0], qkv[:, 1], qkv[:, 2], gate, x @ self.w_beta, self.A_log,
                       self.g_bias, self.pool, self.cu_seqlens, self.slots, self.records, y,
                       record_slots=s.requests, **rows)
        x = x + y.flatten(1) @ self.w_kda_out
        # full-attention layer
        merged = (x @ self.w_merged).view(total, s.q_heads + 2 * s.kv_heads, s.head_dim)
        q = merged[:, :s.q_heads]
        k, v = merged[:, s.q_heads:].split(s.kv_heads, dim=1)
        where = (self.cu_seqlens, self.block_table, self.num_computed)
        q = api.kda_kv_append(q, k, v, self.key_cache, self.value_cache, *where,
                              inv_freq=self.inv_freq, error_word=self.error_word)
        y, _ = api.kda_window_attention(q, self.key_cache, self.value_cache, *where,
                                        self.workspace, **rows)
        x = x + y.flatten(1) @ self.w_out
        # what the target thinks of the drafts
        following = torch.cat([tokens[:, 1:], torch.full_like(tokens[:, :1], -1)], dim=1)
        return api.kda_token_logprobs(x @ self.w_head, following.flatten().contiguous(),
                                      num_top=1, error_word=self.error_word)

    def step(self, tokens: torch.Tensor):
        """One speculative step; returns the accepted counts (1..window), the
        next token of each request and what ``verify`` returned."""
        s = self.sizes
        seen = self.verify(tokens)
        choice = seen.top_index.view(s.requests, s.window)
        agreed = (tokens[:, 1:] == choice[:, :-1]).int().cumprod(dim=1).sum(dim=1)
        accepted = (agreed + 1).to(I32)
        api.kda_commit(self.A_log, self.g_bias, self.pool, self.cu_seqlens, self.slots, accepted,
                       self.records, window=s.window, record_slots=s.requests,
                       error_word=self.error_word)
        self.num_computed += accepted
        following = choice.gather(1, agreed[:, None]).squeeze(1)
        return accepted, following, seen


def main() -> None:
    sizes = Sizes()
    model = HybridModel(sizes)
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randint(0, sizes.vocab, (sizes.requests,), generator=gen, device="cuda", dtype=I32)
    for i in range(8):
        tokens = torch.randint(0, sizes.vocab, (sizes.requests, sizes.window), generator=gen,
                               device="cuda", dtype=I32)
        tokens[:, 0] = last
        # stand in for a drafter that is right once: ask the target itself
        tokens[:, 1] = model.verify(tokens).top_index.view(sizes.requests, sizes.window)[:, 0]
        accepted, last, seen = model.step(tokens)
        print(f"step {i}: accepted {accepted.tolist()}, lengths {model.num_computed.tolist()}, "
              f"mean entropy {seen.entropy.mean().item():.3f}")
    if int(model.error_word.item()) != 0:
        raise SystemExit(f"device error word {int(model.error_word.item())}")


if __name__ == "__main__":
    main()

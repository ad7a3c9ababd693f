"""Requests of a small hybrid model from their prompts on: admission, plain
decoding and speculative steps, all through the library.

    kda_prefill           the KDA layer over whole prompts, from no state
    kda_kv_norm_append    normed and rotated keys and values to the paged cache
    kda_window_attention  the prompts' tokens in windows over their own keys
    kda_decode            the KDA layer for one token of each request
    kda_verify, kda_commit and the others, as in hybrid_step.py

The model is hybrid_step.py's with norms of queries and keys in its
full-attention layer.  Weights and prompts are random.

    python examples/hybrid_requests.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.hybrid_step import BF16, I32, HybridModel, Sizes  # noqa: E402
from linear_attention_speculative_kda_gb300 import api  # noqa: E402


class NormedHybridModel(HybridModel):
    """The model of hybrid_step.py with head norms, and its requests' life
    before and between speculative steps."""

    def __init__(self, sizes: Sizes, device="cuda", seed: int = 0):
        super().__init__(sizes, device, seed)
        gen = torch.Generator().manual_seed(seed + 1)
        self.q_weight, self.k_weight = (
            (1.0 + 0.2 * torch.randn(sizes.head_dim, generator=gen)).to(BF16).to(self.device)
            for _ in range(2))

    def append(self, q, k, v, cu_seqlens, block_table, num_computed):
        return api.kda_kv_norm_append(q, k, v, self.key_cache, self.value_cache, cu_seqlens,
                                      block_table, num_computed, q_weight=self.q_weight,
                                      k_weight=self.k_weight, inv_freq=self.inv_freq,
                                      error_word=self.error_word)

    def _inputs(self, x):
        s = self.sizes
        qkv = (x @ self.w_qkv).view(-1, 3, s.kda_heads, 128)
        gate = (x @ self.w_gate).view(-1, s.kda_heads, 128)
        return (qkv[:, 0], qkv[:, 1], qkv[:, 2], gate, x @ self.w_beta, self.A_log, self.g_bias,
                self.pool)

    def _attention(self, x, where, pieces, workspace):
        """where: rows as the append takes them; pieces: the same tokens in rows
        of at most a window, for the attention."""
        s = self.sizes
        merged = (x @ self.w_merged).view(-1, s.q_heads + 2 * s.kv_heads, s.head_dim)
        k, v = merged[:, s.q_heads:].split(s.kv_heads, dim=1)
        q = self.append(merged[:, :s.q_heads], k, v, *where)
        y, _ = api.kda_window_attention(q, self.key_cache, self.value_cache, *pieces, workspace,
                                        window=s.window, error_word=self.error_word)
        return x + y.flatten(1) @ self.w_out

    def admit(self, prompts: list[torch.Tensor]) -> torch.Tensor:
        """Prompts, one of each request, into the states and the cache; returns
        the logits behind each prompt's last token."""
        s, d = self.sizes, self.device
        lens = [len(p) for p in prompts]
        cu = torch.tensor([0] + lens, dtype=I32, device=d).cumsum(0).to(I32)
        x = self.embed[torch.cat(prompts).to(d).long()]
        y = api.kda_prefill(*self._inputs(x), cu, self.slots,
                            initial_indices=torch.zeros_like(self.slots),
                            error_word=self.error_word)
        x = x + y.flatten(1) @ self.w_kda_out
        # a piece of a prompt is a row of its own, with its request's blocks
        starts = [(b, t) for b, n in enumerate(lens) for t in range(0, n, s.window)]
        begins = [sum(lens[:b]) + t for b, t in starts] + [sum(lens)]
        request = torch.tensor([b for b, _ in starts], device=d)
        pieces = (torch.tensor(begins, dtype=I32, device=d), self.block_table[request],
                  torch.tensor([t for _, t in starts], dtype=I32, device=d))
        workspace = api.allocate_attention_workspace(len(starts), s.q_heads, s.kv_heads, s.head_dim,
                                                     d, window=s.window)
        x = self._attention(x, (cu, self.block_table, torch.zeros_like(self.num_computed)), pieces,
                            workspace)
        self.num_computed = torch.tensor(lens, dtype=I32, device=d)
        return x[cu[1:].long() - 1] @ self.w_head

    def decode(self, tokens: torch.Tensor) -> torch.Tensor:
        """One token int32 of each request; returns the logits behind it."""
        x = self.embed[tokens.long()]
        y = api.kda_decode(*self._inputs(x), self.slots, error_word=self.error_word)
        x = x + y.flatten(1) @ self.w_kda_out
        cu = torch.arange(self.sizes.requests + 1, dtype=I32, device=self.device)
        where = (cu, self.block_table, self.num_computed)
        x = self._attention(x, where, where, self.workspace)
        self.num_computed = self.num_computed + 1
        return x @ self.w_head


def main() -> None:
    sizes = Sizes(max_len=400)
    model = NormedHybridModel(sizes)
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, sizes.vocab, (n,), generator=gen) for n in (7, 130, 33, 1, 64)]
    last = model.admit(prompts).argmax(1).to(I32)
    print(f"admitted {model.num_computed.tolist()}")
    for _ in range(4):
        last = model.decode(last).argmax(1).to(I32)
    print(f"decoded to {model.num_computed.tolist()}")
    for i in range(4):
        tokens = torch.randint(0, sizes.vocab, (sizes.requests, sizes.window), generator=gen).to(I32)
        tokens = tokens.to(model.device)
        tokens[:, 0] = last
        tokens[:, 1] = model.verify(tokens).top_index.view(sizes.requests, sizes.window)[:, 0]
        accepted, last, _ = model.step(tokens)
        print(f"step {i}: accepted {accepted.tolist()}, lengths {model.num_computed.tolist()}")
    if int(model.error_word.item()) != 0:
        raise SystemExit(f"device error word {int(model.error_word.item())}")


if __name__ == "__main__":
    main()

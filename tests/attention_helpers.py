"""Seeded cases of the full-attention layers' calls for the tests: tensors
for the library and the same numbers in float64 for the oracle."""

from __future__ import annotations

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LAYOUTS = ("tokens", "heads", "pairs")


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def cache_pair(blocks, block_size, heads, dim, dtype, layout, gen, device):
    """Key and value caches viewed as [blocks, block_size, heads, dim]: token
    major, head major, or key and value blocks side by side in one tensor."""
    def normal(*shape):
        return torch.randn(shape, generator=gen).to(dtype).to(device)
    if layout == "tokens":
        return normal(blocks, block_size, heads, dim), normal(blocks, block_size, heads, dim)
    if layout == "heads":
        return (normal(blocks, heads, block_size, dim).transpose(1, 2),
                normal(blocks, heads, block_size, dim).transpose(1, 2))
    both = normal(blocks, 2, block_size, heads, dim)
    return both[:, 0], both[:, 1]


class Case:
    """Rows with lens[b] new tokens after computed[b] earlier ones, blocks of
    the cache in random order, q, k, v as views of one merged buffer."""

    def __init__(self, lens, computed, q_heads, kv_heads, dim, block_size, dtype="bf16",
                 layout="tokens", seed=0, device="cuda", spare_blocks=3, extra_columns=1):
        gen = torch.Generator().manual_seed(seed)
        self.dtype = DTYPES[dtype]
        self.q_heads, self.kv_heads, self.dim, self.block_size = q_heads, kv_heads, dim, block_size
        B, total = len(lens), int(sum(lens))
        width = max([(c + n + block_size - 1) // block_size for c, n in zip(computed, lens)] + [1])
        need = [(c + n + block_size - 1) // block_size for c, n in zip(computed, lens)]
        blocks = 1 + sum(need) + spare_blocks
        order = (torch.randperm(blocks - 1, generator=gen) + 1).tolist()
        table = torch.zeros((B, width + extra_columns), dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                table[b, i] = order.pop()
        self.table = table.to(device)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32,
                               device=device)
        self.computed = torch.tensor(computed, dtype=torch.int32, device=device)
        self.keys, self.values = cache_pair(blocks, block_size, kv_heads, dim, self.dtype, layout,
                                            gen, device)
        merged = torch.randn((total, q_heads + 2 * kv_heads + 1, dim),
                             generator=gen).to(self.dtype).to(device)
        self.q = merged[:, :q_heads]
        self.k = merged[:, q_heads:q_heads + kv_heads]
        self.v = merged[:, q_heads + kv_heads:q_heads + 2 * kv_heads]
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def meta(self):
        return (self.cu.cpu().numpy(), self.table.cpu().numpy(), self.computed.cpu().numpy())


def frequencies(rotary_dim, base=10000.0, device="cuda"):
    return torch.tensor([base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)],
                        dtype=torch.float64, device=device)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest_half(dtype):
    """Half a step among the subnormals of the type."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2

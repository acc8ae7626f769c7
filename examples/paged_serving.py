"""Two attention layers over caches in pages, as a server would run them.

    python examples/paged_serving.py [--tokens 1000] [--steps 4]

GroupedLayer has grouped heads: positions are rotated into queries and keys, keys and values go to the pages of
their sequence, and prompts, later chunks and single tokens are one call over the pages. LatentLayer caches
one latent vector a token: prompts run in the expanded form, decode steps in the absorbed one, over the whole
cache or over the tokens that the KPool selection leaves. Every weight and token is random: the example shows
which calls belong together and what passes between them.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_attention_kpool_gb300 import kpool  # noqa: E402

BF = dict(dtype=torch.bfloat16, device="cuda")
INDEX_HEADS, INDEX_DIM = 32, 128


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pages:
    """Pages of a pool, handed to sequences as they grow."""

    def __init__(self, sequences: int, capacity: int, size: int):
        self.size, self.per = size, (capacity + size - 1) // size
        self.free = list(range(sequences * self.per))[::-1]
        self.table = torch.full((sequences, self.per), -1, dtype=torch.int32, device="cuda")
        self.held, self.lengths = [0] * sequences, [0] * sequences

    def __len__(self):
        return self.table.shape[0] * self.per

    def extend(self, b: int, n: int) -> torch.Tensor:
        """Places (page * size + token) of the next n tokens of sequence b."""
        start = self.lengths[b]
        while self.held[b] * self.size < start + n:
            self.table[b, self.held[b]] = self.free.pop()
            self.held[b] += 1
        self.lengths[b] = start + n
        j = torch.arange(start, start + n, device="cuda")
        return self.table[b, j // self.size].long() * self.size + j % self.size


class GroupedLayer:
    def __init__(self, sequences: int, capacity: int, q_heads: int = 32, kv_heads: int = 8, head_dim: int = 128,
                 page: int = 16):
        self.heads, self.scale = (q_heads, kv_heads, head_dim), 1.0 / math.sqrt(head_dim)
        self.pages = Pages(sequences, capacity, page)
        self.k = torch.zeros((len(self.pages), page, kv_heads, head_dim), **BF)
        self.v = torch.zeros_like(self.k)
        self.table = kpool.new_rotary_table(head_dim, base=500000.0)

    def step(self, q, k, v, new):
        """Rows of every sequence in turn, new[b] tokens each: rotated, cached, and attended with what came before."""
        starts = [self.pages.lengths[b] for b in range(len(new))]
        pos = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, new)]).to(torch.int32).cuda()
        q, k = kpool.kpool_rotary(q, pos, self.table, k=k)
        at = torch.cat([self.pages.extend(b, n) for b, n in enumerate(new)])
        self.k.flatten(0, 1)[at], self.v.flatten(0, 1)[at] = k, v
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        one = all(n == 1 for n in new)
        return kpool.kpool_attention_paged(q, self.k, self.v, self.pages.table, i32(self.pages.lengths), self.scale,
                                           cu_q=None if one else i32(cu))[0]


class LatentLayer:
    def __init__(self, capacity: int, heads: int = 16, latent: int = 512, nope: int = 128, rope: int = 64,
                 value: int = 128, page: int = 64, pool: int = 4, index_topk: int = 256, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dims, self.heads, self.scale = (latent, nope, rope, value), heads, 1.0 / math.sqrt(nope + rope)
        self.up_k = torch.randn((heads, nope, latent), generator=gen, device="cuda").div_(math.sqrt(latent)).to(torch.bfloat16)
        self.up_v = torch.randn((heads, value, latent), generator=gen, device="cuda").div_(math.sqrt(latent)).to(torch.bfloat16)
        self.pages = Pages(1, capacity, page)
        self.cache = torch.zeros((len(self.pages), page, latent + rope), **BF)
        self.table = kpool.new_rotary_table(rope, factor=40.0, original_length=4096.0)
        self.pool, self.topk, self.capacity = pool, index_topk, capacity
        self.index_k = torch.zeros((capacity, INDEX_DIM), **BF)

    def append(self, q, latent, k_rope, index_k):
        """Rotates the ends of q [n, H, nope + rope] and k_rope [n, rope], and caches the tokens; returns both."""
        n, start = latent.shape[0], self.pages.lengths[0]
        pos = torch.arange(start, start + n, dtype=torch.int32, device="cuda")
        q, k_rope = kpool.kpool_rotary(q, pos, self.table, k=k_rope[:, None], q_offset=self.dims[1], interleaved=True)
        self.cache.flatten(0, 1)[self.pages.extend(0, n)] = torch.cat((latent, k_rope[:, 0]), dim=-1)
        self.index_k[start:start + n] = index_k
        return q, k_rope[:, 0]

    def prompt(self, q, latent, k_rope):
        """The whole prompt in the expanded form: keys and values of every head from the latents."""
        cu = i32([0, q.shape[0]])
        k = torch.einsum("nl,hdl->nhd", latent, self.up_k)
        v = torch.einsum("nl,hdl->nhd", latent, self.up_v)
        return kpool.kpool_attention_latent_prompt(q, k, k_rope, v, cu, cu, self.scale)[0]

    def decode(self, q, token_ids=None):
        """The newest token in the absorbed form: the queries go into the latent space, the result comes back."""
        latent, nope = self.dims[:2]
        into = torch.cat((torch.einsum("rhd,hdl->rhl", q[..., :nope], self.up_k), q[..., nope:]), dim=-1)
        seq = None if token_ids is None else i32([0])
        low, _ = kpool.kpool_attention_latent(into, self.cache, self.pages.table, i32(self.pages.lengths), latent,
                                              self.scale, token_ids=token_ids, row_seq=seq)
        return torch.einsum("rhl,hdl->rhd", low, self.up_v)

    def select(self, index_q, index_w):
        """The token ids that the selection leaves the newest token."""
        cu = i32([0, self.capacity])
        pooled = kpool.kpool_pool_keys(self.index_k, cu, self.pool)
        return kpool.kpool_select_rows(index_q, index_w, i32([0]), i32([self.pages.lengths[0] - 1]), pooled, cu,
                                       self.capacity, self.pool, self.topk, 1.0 / math.sqrt(INDEX_DIM))[1]


def main(tokens: int = 1000, steps: int = 4):
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    grouped = GroupedLayer(2, tokens + steps)
    hq, hkv, d = grouped.heads
    new = [tokens, tokens // 3]
    n = sum(new)
    grouped.step(normal(n, hq, d), normal(n, hkv, d), normal(n, hkv, d), new)
    for _ in range(steps):
        out = grouped.step(normal(2, hq, d), normal(2, hkv, d), normal(2, hkv, d), [1, 1])
    print(f"grouped heads: {steps} steps over caches of {grouped.pages.lengths}, output norm {out.float().norm().item():.3f}")

    layer = LatentLayer(tokens + steps)
    latent, nope, rope, _ = layer.dims
    q, c, kr, ik = normal(tokens, layer.heads, nope + rope), normal(tokens, latent), normal(tokens, rope), normal(tokens, INDEX_DIM)
    q, kr = layer.append(q, c, kr, ik)
    whole = layer.prompt(q, c, kr)
    again = layer.decode(q[-1:])
    print(f"latent prompt of {tokens}: its last row expanded and absorbed differ by at most "
          f"{(whole[-1:].float() - again.float()).abs().max().item():.4f}")
    for _ in range(steps):
        y, _ = layer.append(normal(1, layer.heads, nope + rope), normal(1, latent), normal(1, rope), normal(1, INDEX_DIM))
        ids = layer.select(normal(1, INDEX_HEADS, INDEX_DIM), torch.rand((1, INDEX_HEADS), generator=gen, device="cuda"))
        sparse = layer.decode(y, ids)
    print(f"{steps} decode steps over {int((ids >= 0).sum())} selected tokens of {layer.pages.lengths[0]}, output norm "
          f"{sparse.float().norm().item():.3f}")
    return whole[-1:], again, layer, (q, c, kr)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    main(a.tokens, a.steps)

"""One attention layer with the KPool selection, as a server would run it.

    python examples/sparse_layer.py [--tokens 4096] [--steps 4]

The layer keeps a key/value cache and pooled index keys. It takes a prompt (selection, then
attention over the selected tokens), single decode steps against the cache, and the
verification of a drafted tree of tokens by dense attention over the cache. Every tensor
is random: the example shows which calls belong together and what passes between them.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_attention_kpool_gb300 import kpool  # noqa: E402

INDEX_HEADS, INDEX_DIM = 32, 128


class SparseLayer:
    """Cache and calls of one layer for a single sequence of up to `capacity` tokens."""

    def __init__(self, capacity: int, q_heads: int = 32, kv_heads: int = 8, head_dim: int = 128, pool: int = 4,
                 index_topk: int = 2048):
        self.capacity, self.pool, self.topk = capacity, pool, index_topk
        self.heads = (q_heads, kv_heads, head_dim)
        self.scale, self.index_scale = 1.0 / math.sqrt(head_dim), 1.0 / math.sqrt(INDEX_DIM)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.k = torch.zeros((capacity, kv_heads, head_dim), **bf)
        self.v = torch.zeros((capacity, kv_heads, head_dim), **bf)
        self.index_k = torch.zeros((capacity, INDEX_DIM), **bf)
        self.cu = torch.tensor([0, capacity], dtype=torch.int32, device="cuda")
        self.length = 0
        self.workspaces = {}

    def _workspace(self, rows: int) -> torch.Tensor:
        if rows not in self.workspaces:
            self.workspaces[rows] = kpool.new_attention_workspace(rows, 1, *self.heads, torch.bfloat16)
        return self.workspaces[rows]

    def append(self, k, v, index_k):
        n = k.shape[0]
        at = slice(self.length, self.length + n)
        self.k[at], self.v[at], self.index_k[at] = k, v, index_k
        self.length += n

    def prompt(self, q, index_q, index_w):
        """All rows of a prompt that was appended: each attends to the tokens its selection left it."""
        n = q.shape[0]
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        _, token_ids, _ = kpool.kpool_select(index_q, self.index_k[:n], index_w, cu, self.pool, self.topk,
                                             self.index_scale)
        return kpool.kpool_attention_selected(q, self.k[:n], self.v[:n], token_ids, cu, self.scale,
                                              workspace=self._workspace(n))[0]

    def prompt_dense(self, q):
        """The same prompt with every earlier token visible."""
        n = q.shape[0]
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        return kpool.kpool_attention_prompt(q, self.k[:n], self.v[:n], cu, cu, self.scale,
                                            workspace=self._workspace(n))[0]

    def decode(self, q, index_q, index_w):
        """One new token (appended before): selection over the pooled cache, attention over its ids."""
        # (pooled anew for brevity; a server keeps the pooled keys and adds a pool when one is complete)
        pooled = kpool.kpool_pool_keys(self.index_k, self.cu, self.pool)
        row_seq = torch.zeros(1, dtype=torch.int32, device="cuda")
        row_pos = torch.full((1,), self.length - 1, dtype=torch.int32, device="cuda")
        _, token_ids, _ = kpool.kpool_select_rows(index_q, index_w, row_seq, row_pos, pooled, self.cu, self.capacity,
                                                  self.pool, self.topk, self.index_scale)
        return kpool.kpool_attention_selected(q, self.k, self.v, token_ids, self.cu, self.scale, row_seq=row_seq,
                                              workspace=self._workspace(1))[0]

    def verify(self, q, parents):
        """A drafted tree whose nodes lie after the committed tokens: parents[i] < i, or -1 for a root."""
        n = len(parents)
        words = (n + 31) // 32
        seen, rows = [], []
        for i, parent in enumerate(parents):
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
            for w in range(words):
                x = (seen[i] >> (32 * w)) & 0xFFFFFFFF
                rows.append(x - (1 << 32) if x >= 1 << 31 else x)
        mask = torch.tensor(rows, dtype=torch.int32, device="cuda").reshape(n, words)
        cu_rows = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        prefix = torch.tensor([self.length - n], dtype=torch.int32, device="cuda")
        return kpool.kpool_attention_tree(q, self.k, self.v, cu_rows, self.cu, prefix, self.scale, mask=mask,
                                          workspace=self._workspace(n))[0]


def random_tokens(n, layer, gen):
    """Queries, keys, values and index inputs of n tokens."""
    hq, hkv, d = layer.heads

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    return {"q": normal(n, hq, d), "k": normal(n, hkv, d), "v": normal(n, hkv, d),
            "index_q": normal(n, INDEX_HEADS, INDEX_DIM), "index_k": normal(n, INDEX_DIM),
            "index_w": torch.rand((n, INDEX_HEADS), generator=gen, device="cuda")}


def main(tokens: int = 4096, steps: int = 4):
    gen = torch.Generator(device="cuda").manual_seed(0)
    layer = SparseLayer(capacity=tokens + steps + 64)
    x = random_tokens(tokens, layer, gen)
    layer.append(x["k"], x["v"], x["index_k"])
    sparse = layer.prompt(x["q"], x["index_q"], x["index_w"])
    dense = layer.prompt_dense(x["q"])
    same = min(tokens, layer.topk)  # rows that may keep every earlier token see what dense rows see
    print(f"prompt of {tokens}: first {same} rows differ from dense attention by at most "
          f"{(sparse[:same].float() - dense[:same].float()).abs().max().item():.4f}")
    for _ in range(steps):
        y = random_tokens(1, layer, gen)
        layer.append(y["k"], y["v"], y["index_k"])
        out = layer.decode(y["q"], y["index_q"], y["index_w"])
    print(f"{steps} decode steps, cache of {layer.length} tokens, last output norm {out.float().norm().item():.3f}")
    parents = [-1, 0, 0, 1, 1, 2, 3]
    z = random_tokens(len(parents), layer, gen)
    layer.append(z["k"], z["v"], z["index_k"])
    out = layer.verify(z["q"], parents)
    print(f"verified a tree of {len(parents)} nodes, output norm {out.float().norm().item():.3f}")
    return sparse, dense


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    main(a.tokens, a.steps)

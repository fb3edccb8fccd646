"""A decoder layer that serves a few sequences: prompts, then single tokens, with
the attention over an 8-bit paged cache and the MoE FFN behind it, and the cache
brought back to a budget where it grows past a limit.

    python examples/decode_with_cache.py

Per call of ``DecoderLayer``: q, k, v = norm(x) Wqkv^T; append k, v; x += attend(q)
Wo^T; x += MoEFFN(norm(x)).  (No positions and random weights: the layer shows
how the calls fit together.)  All matmuls are this library's.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_ffn_layer_gb300 import binding as B  # noqa: E402
from moe_ffn_layer_gb300 import synth  # noqa: E402
from moe_ffn_layer_gb300.kv_cache import KVCache8  # noqa: E402
from moe_ffn_layer_gb300.layer import MoEFFN  # noqa: E402


class Pages:
    """The cache's free pages, and a table of the sequences' own (the caller's part)."""

    def __init__(self, sequences: int, width: int, total: int, device):
        self.free = list(range(total))
        self.held = [[] for _ in range(sequences)]
        self.width, self.device = width, device

    def grow(self, lens, page):
        for own, n in zip(self.held, lens):
            while len(own) * page < n:
                own.append(self.free.pop())
        return self.table(self.held)

    def table(self, held):
        t = torch.zeros(len(held), self.width, dtype=torch.int32)
        for row, own in zip(t, held):
            row[:len(own)] = torch.tensor(own, dtype=torch.int32)
        return t.to(self.device)

    def take(self, lens, page):
        """Pages for sequences of those lengths, beside the ones they hold."""
        return [[self.free.pop() for _ in range(-(-n // page))] for n in lens]

    def replace(self, held):
        for own in self.held:
            self.free += own
        self.held = held


def norm(x):
    """Rows to a root mean square of one."""
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class DecoderLayer:
    """Weights bf16: w_qkv [(Hq + 2 Hkv) D, H], w_o [H, Hq D]; ffn a MoEFFN."""

    def __init__(self, w_qkv, w_o, ffn: MoEFFN, cache: KVCache8, heads: int):
        self.w_qkv, self.w_o, self.ffn, self.cache, self.heads = w_qkv, w_o, ffn, cache, heads

    def linear(self, x, w):
        out = torch.empty(x.shape[0], w.shape[0], dtype=torch.bfloat16, device=x.device)
        B.moe_grouped_gemm(x, w, None, 1, x.shape[0], w.shape[0], w.shape[1], 0, out, None, 0,
                           torch.cuda.current_stream())
        return out

    def __call__(self, x, table, lens, cu, max_new, max_len, weights=None):
        Hq, Hkv, D = self.heads, self.cache.kv_heads, self.cache.head_dim
        qkv = self.linear(norm(x), self.w_qkv).view(-1, Hq + 2 * Hkv, D)
        self.cache.append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], table, lens, cu)
        att = self.cache.attend(qkv[:, :Hq], table, lens, cu, max_new, max_len, weights=weights)
        x = x + self.linear(att.view(-1, Hq * D), self.w_o)
        return x + self.ffn(norm(x))


def make_layer(H=512, heads=8, kv_heads=2, D=64, page=32, pages=64, seed=0, device="cuda"):
    g = torch.Generator(device).manual_seed(seed)
    mat = lambda n, k: (torch.randn(n, k, generator=g, device=device) * k ** -0.5).bfloat16()  # noqa: E731
    w = synth.Workload("example", 8, H, 8, 2, 256, 256, sigma_router=0.1)
    ffn = MoEFFN.from_inputs(synth.make_inputs(w, seed), w.k, device)
    cache = KVCache8(pages, kv_heads, D, page, device)
    return DecoderLayer(mat((heads + 2 * kv_heads) * D, H), mat(H, heads * D), ffn, cache, heads)


def serve(layer, prompts, steps, limit, budget, sink=4, recent=16, seed=1):
    """Runs the prompts (lengths), then `steps` single tokens of each sequence.
    Returns (last outputs [B, H], lengths, evictions)."""
    n, page, dev = len(prompts), layer.cache.page, layer.cache.device
    H = layer.w_o.shape[0]
    g = torch.Generator(dev).manual_seed(seed)
    # room for every sequence at its limit, and for the pages an eviction writes beside it
    pages = Pages(n, -(-limit // page), layer.cache.num_pages, dev)
    weights = torch.zeros(n, layer.cache.kv_heads, limit, device=dev)
    lens, evictions = list(prompts), 0
    to = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    x = torch.randn(sum(prompts), H, generator=g, device=dev).bfloat16()
    cu = np.concatenate([[0], np.cumsum(prompts)]).tolist()
    y = layer(x, pages.grow(lens, page), to(lens), to(cu), max(prompts), max(lens), weights)
    y = y[torch.tensor(cu[1:], device=dev) - 1]
    one = to(list(range(n + 1)))
    for _ in range(steps):
        if max(lens) + 1 > limit:
            kept = [min(L, budget) for L in lens]
            new = pages.take(kept, page)
            _, w, _ = layer.cache.evict(weights, pages.table(pages.held), to(lens), max(lens), budget, sink, recent,
                                        pages.table(new))
            weights.zero_()
            weights[:, :, :budget] = w
            pages.replace(new)
            lens, evictions = kept, evictions + 1
        lens = [L + 1 for L in lens]
        y = layer(y, pages.grow(lens, page), to(lens), one, 1, max(lens), weights)
    return y, lens, evictions


if __name__ == "__main__":
    layer = make_layer()
    y, lens, evictions = serve(layer, [200, 75, 131], 120, limit=256, budget=128)
    torch.cuda.synchronize()
    print(f"lengths {lens}, {evictions} eviction(s), |y| = {float(y.float().norm()):.3f}, "
          f"device status {B.moe_last_device_error(torch.cuda.current_stream())}")

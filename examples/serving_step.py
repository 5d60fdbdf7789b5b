"""One attention block of a multi-LoRA serving step: requests on different adapters, their
keys and values in pages, prompts taken in by chunks and tokens decoded one by one.

    qkv = x W_qkv + s_k (x A_k) B_k          lora_base_fused
    keys, values -> pages                    lora_kv_write
    o = attention over the pages             lora_attention
    y = o W_o + s_k (o A'_k) B'_k            lora_base_fused

`python examples/serving_step.py` runs it on random weights and prints the time of a
decoding step.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import adapter_sgmv_bgmv_gb300 as L  # noqa: E402


class Block:
    """The block's weights, adapters and cache.  w_qkv [d, (heads + 2 kv_heads) dim] and
    w_o [heads dim, d] are bf16; `qkv_adapters` and `o_adapters` are L.AdapterTable's of
    the two projections, with the same adapter ids."""

    def __init__(self, ctx, w_qkv, w_o, qkv_adapters, o_adapters, heads, kv_heads, dim, n_pages,
                 page_size=16, cache_dtype=torch.bfloat16):
        self.ctx, self.w_qkv, self.w_o = ctx, w_qkv, w_o
        self.qkv_adapters, self.o_adapters = qkv_adapters, o_adapters
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        pool = torch.zeros((n_pages, 2, page_size, kv_heads, dim), dtype=cache_dtype, device=w_qkv.device)
        scales = (None, None)
        if cache_dtype != torch.bfloat16:
            scales = torch.zeros((n_pages, 2, kv_heads, page_size), device=w_qkv.device).transpose(2, 3).unbind(1)
        self.cache = L.KvCache(ctx, pool[:, 0], pool[:, 1], *scales)

    def __call__(self, x, ids, batch, window=0, sinks=0):
        """x [n, d] -> y [n, d] for the batch's new tokens; ids [n] are their adapters (-1: none)."""
        n, q = x.shape[0], self.heads * self.dim
        k = q + self.kv_heads * self.dim
        qkv = torch.empty((n, self.w_qkv.shape[1]), dtype=torch.bfloat16, device=x.device)
        L.lora_base_fused(self.ctx, self.qkv_adapters, ids, x, self.w_qkv, qkv)
        L.lora_kv_write(self.ctx, self.cache, batch, qkv[:, q:k], qkv[:, k:])
        o = torch.empty((n, q), dtype=torch.bfloat16, device=x.device)
        L.lora_attention(self.ctx, self.cache, batch, qkv[:, :q], o, window=window, sinks=sinks)
        y = torch.empty((n, self.w_o.shape[1]), dtype=torch.bfloat16, device=x.device)
        L.lora_base_fused(self.ctx, self.o_adapters, ids, o, self.w_o, y)
        return y


class Requests:
    """Which pages the requests have, and how long they are: a host-side list of free pages,
    and the tensors that the kernels read."""

    def __init__(self, n, n_pages, page_size, most, device="cuda"):
        self.page_size, self.free = page_size, list(range(n_pages))[::-1]
        self.table = np.full((n, -(-most // page_size)), -1, np.int32)
        self.lens = np.zeros(n, np.int32)
        self.device = device

    def grow(self, new):
        """The batch in which request s gets new[s] tokens."""
        for s, k in enumerate(new):
            have = -(-int(self.lens[s]) // self.page_size)
            self.lens[s] += k
            for j in range(have, -(-int(self.lens[s]) // self.page_size)):
                self.table[s, j] = self.free.pop()
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        to = lambda a: torch.from_numpy(a.copy()).to(self.device)  # noqa: E731
        return L.KvBatch(to(starts), to(self.lens), to(self.table), max_new=int(max(new)))


def random_block(ctx, d=512, heads=8, kv_heads=2, dim=64, rank=16, n_adapters=3, n_pages=64,
                 page_size=16, cache_dtype=torch.bfloat16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(rows, cols, std):
        return (torch.randn((rows, cols), generator=gen, device="cuda") * std).to(torch.bfloat16)

    def table(d_in, d_out):
        pages = np.arange(n_adapters * rank, dtype=np.int32).reshape(n_adapters, rank)
        return L.AdapterTable(ctx, rand(n_adapters * rank, d_in, d_in ** -0.5), rand(n_adapters * rank, d_out, rank ** -0.5),
                              np.full(n_adapters, rank, np.int32), np.full(n_adapters, 0.5, np.float32), pages, pages)
    wide = (heads + 2 * kv_heads) * dim
    return Block(ctx, rand(d, wide, d ** -0.5), rand(heads * dim, d, (heads * dim) ** -0.5),
                 table(d, wide), table(heads * dim, d), heads, kv_heads, dim, n_pages, page_size, cache_dtype)


def main():
    ctx = L.Context(0, max_rows=8192)
    n, d, page = 64, 4096, 16
    block = random_block(ctx, d=d, heads=32, kv_heads=8, dim=128, n_adapters=16, n_pages=64 * 70, page_size=page)
    req = Requests(n, 64 * 70, page, 1100)
    adapters = np.arange(n, dtype=np.int32) % 16
    rng = np.random.default_rng(0)
    lens = rng.integers(100, 1000, n)
    while lens.any():                                  # prompts, by chunks of up to 128 tokens
        new = np.minimum(lens, 128)
        lens = lens - new
        x = torch.randn((int(new.sum()), d), device="cuda").to(torch.bfloat16)
        block(x, np.repeat(adapters, new), req.grow(new))
    x = torch.randn((n, d), device="cuda").to(torch.bfloat16)
    for i in range(23):
        if i == 3:
            torch.cuda.synchronize()
            t0 = torch.cuda.Event(enable_timing=True)
            t0.record()
        block(x, adapters, req.grow(np.ones(n, np.int32)))
    t1 = torch.cuda.Event(enable_timing=True)
    t1.record()
    ctx.sync_status()
    print(f"{n} requests, {int(req.lens.sum())} tokens in the cache: {t0.elapsed_time(t1) / 20 * 1e3:.0f} us a decoding step of the block")


if __name__ == "__main__":
    main()

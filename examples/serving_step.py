"""One attention block of a multi-LoRA serving step: requests on different adapters, their
keys and values in pages, prompts taken in by chunks and tokens decoded one by one.

    qkv = x W_qkv + s_k (x A_k) B_k          lora_base_fused
    keys, values -> pages                    lora_kv_write, or with norms of heads and the
                                             rotation by position lora_kv_write_rope
    o = attention over the pages             lora_attention, or over the pages chosen for
                                             each token: lora_kv_bounds, lora_block_select,
                                             lora_block_attention
    y = o W_o + s_k (o A'_k) B'_k            lora_base_fused

Which pages the requests have is kept on the host (Requests) or in device memory
(PagedRequests: lora_pages_extend, _fork, _free, lora_kv_copy).

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
                 page_size=16, cache_dtype=torch.bfloat16, rope=None):
        self.ctx, self.w_qkv, self.w_o = ctx, w_qkv, w_o
        self.qkv_adapters, self.o_adapters = qkv_adapters, o_adapters
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        pool = torch.zeros((n_pages, 2, page_size, kv_heads, dim), dtype=cache_dtype, device=w_qkv.device)
        scales = (None, None)
        if cache_dtype != torch.bfloat16:
            scales = torch.zeros((n_pages, 2, kv_heads, page_size), device=w_qkv.device).transpose(2, 3).unbind(1)
        self.cache = L.KvCache(ctx, pool[:, 0], pool[:, 1], *scales)
        self.rope = rope
        dev = w_qkv.device
        self.cache.attach_bounds(torch.zeros((n_pages, kv_heads, 2, dim), dtype=torch.int8, device=dev),
                                 torch.zeros((n_pages, kv_heads), device=dev))

    def __call__(self, x, ids, batch, window=0, sinks=0, blocks=0):
        """x [n, d] -> y [n, d] for the batch's new tokens; ids [n] are their adapters (-1: none).
        With `blocks`, each token attends to that many pages at most (for steps of few tokens), and there is
        no window.  The bounds that choose them are kept up to date by every step, so that any later one
        can choose."""
        if blocks and window:
            raise ValueError("a token sees its chosen pages or a window, not both")
        n, q = x.shape[0], self.heads * self.dim
        k = q + self.kv_heads * self.dim
        qkv = torch.empty((n, self.w_qkv.shape[1]), dtype=torch.bfloat16, device=x.device)
        L.lora_base_fused(self.ctx, self.qkv_adapters, ids, x, self.w_qkv, qkv)
        if self.rope is None:
            L.lora_kv_write(self.ctx, self.cache, batch, qkv[:, q:k], qkv[:, k:])
        else:
            L.lora_kv_write_rope(self.ctx, self.cache, self.rope, batch, qkv[:, :q], qkv[:, q:k], qkv[:, k:])
        L.lora_kv_bounds(self.ctx, self.cache, batch, n)
        o = torch.empty((n, q), dtype=torch.bfloat16, device=x.device)
        if blocks:
            chosen = L.BlockSelection.empty(n, self.cache, blocks)
            L.lora_block_select(self.ctx, self.cache, batch, qkv[:, :q], chosen)
            L.lora_block_attention(self.ctx, self.cache, chosen, qkv[:, :q], o)
        else:
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


class PagedRequests:
    """The same in device memory: lengths, page table and the pages' counts of holders, changed by
    the library's calls; `caches` are the layers' that the pages belong to."""

    def __init__(self, ctx, caches, n, n_pages, page_size, most, device="cuda"):
        self.ctx, self.caches = ctx, caches
        new = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32, device=device)  # noqa: E731
        self.table = L.PageTable(new(n), new(n, -(-most // page_size), fill=-1), new(n_pages), page_size)
        self.got, self.src, self.dst, self.cells = new(n), new(n), new(n), new(n)

    def grow(self, new):
        """The batch in which request s gets new[s] tokens.  One that there is no room for stays as it was
        (got[s] is 0): the batch has a length of 0 for it, so that its rows have no position, nothing
        of them is stored and their attention is zeros; they can be offered again.  Nothing here waits for the GPU."""
        to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(self.got.device)  # noqa: E731
        asked = to(new)
        L.lora_pages_extend(self.ctx, self.table, asked, self.got, self.src, self.dst, self.cells)
        L.lora_kv_copy(self.ctx, self.caches, self.src, self.dst, self.cells)
        lens = torch.where(self.got == asked, self.table.lens, 0)
        return L.KvBatch(to(np.concatenate([[0], np.cumsum(new)])), lens, self.table.pages, max_new=int(max(new)))

    def fork(self, parents, children):
        to = lambda a: torch.tensor(a, dtype=torch.int32, device=self.got.device)  # noqa: E731
        L.lora_pages_fork(self.ctx, self.table, to(parents), to(children))

    def end(self, requests):
        L.lora_pages_free(self.ctx, self.table, torch.tensor(requests, dtype=torch.int32, device=self.got.device))


def random_block(ctx, d=512, heads=8, kv_heads=2, dim=64, rank=16, n_adapters=3, n_pages=64,
                 page_size=16, cache_dtype=torch.bfloat16, seed=0, rope=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(rows, cols, std):
        return (torch.randn((rows, cols), generator=gen, device="cuda") * std).to(torch.bfloat16)

    def table(d_in, d_out):
        pages = np.arange(n_adapters * rank, dtype=np.int32).reshape(n_adapters, rank)
        return L.AdapterTable(ctx, rand(n_adapters * rank, d_in, d_in ** -0.5), rand(n_adapters * rank, d_out, rank ** -0.5),
                              np.full(n_adapters, rank, np.int32), np.full(n_adapters, 0.5, np.float32), pages, pages)
    wide = (heads + 2 * kv_heads) * dim
    return Block(ctx, rand(d, wide, d ** -0.5), rand(heads * dim, d, (heads * dim) ** -0.5),
                 table(d, wide), table(heads * dim, d), heads, kv_heads, dim, n_pages, page_size, cache_dtype, rope)


def main():
    ctx = L.Context(0, max_rows=8192)
    n, d, page = 64, 4096, 16
    rope = L.HeadRope((1e4 ** (-torch.arange(64) / 64)).cuda(), 128)
    block = random_block(ctx, d=d, heads=32, kv_heads=8, dim=128, n_adapters=16, n_pages=64 * 70, page_size=page, rope=rope)
    req = PagedRequests(ctx, [block.cache], n, 64 * 70, page, 1100)
    adapters = np.arange(n, dtype=np.int32) % 16
    rng = np.random.default_rng(0)
    lens = rng.integers(100, 1000, n)
    while lens.any():                                  # prompts, by chunks of up to 128 tokens
        new = np.minimum(lens, 128)
        lens = lens - new
        x = torch.randn((int(new.sum()), d), device="cuda").to(torch.bfloat16)
        block(x, np.repeat(adapters, new), req.grow(new))
    for blocks in (0, 16):
        x = torch.randn((n, d), device="cuda").to(torch.bfloat16)
        for i in range(23):
            if i == 3:
                torch.cuda.synchronize()
                t0 = torch.cuda.Event(enable_timing=True)
                t0.record()
            block(x, adapters, req.grow(np.ones(n, np.int32)), blocks=blocks)
        t1 = torch.cuda.Event(enable_timing=True)
        t1.record()
        ctx.sync_status()
        print(f"{n} requests, {int(req.table.lens.sum())} tokens in the cache{f', {blocks} pages of each' if blocks else ''}: "
              f"{t0.elapsed_time(t1) / 20 * 1e3:.0f} us a decoding step of the block")


if __name__ == "__main__":
    main()

"""The operators around the cache together, as a serving step runs them: examples/serving_step.py with
rotated heads, pages kept in device memory, a request forked half way and one ended, attention over
all pages or over chosen ones, against the whole block in 64 bits; and the cache's part of a step
captured in a graph."""
import math

import numpy as np
import pytest
import torch

from tests._step_ref import rope as rope_model
from tests.test_gpu_serving_step import _example, _project

pytestmark = pytest.mark.gpu


def _whole(block, x, k, freqs, weights):
    """The block over one request's tokens at once, in 64 bits."""
    q, kv, d = block.heads, block.kv_heads, block.dim
    h = _project(x.double(), block.w_qkv, block.qkv_adapters, k)
    n = x.shape[0]
    pos = torch.arange(n, device="cuda")
    qs = rope_model(h[:, :q * d].view(n, q, d), weights[0], pos, freqs, 1e-6, False)[0]
    ks = rope_model(h[:, q * d:(q + kv) * d].view(n, kv, d), weights[1], pos, freqs, 1e-6, False)[0]
    vs = h[:, (q + kv) * d:].view(n, kv, d)
    o = torch.empty((n, q, d), dtype=torch.float64, device="cuda")
    for a in range(q):
        z = (qs[:, a] @ ks[:, a // (q // kv)].T / math.sqrt(d)).masked_fill(pos > pos[:, None], -math.inf)
        o[:, a] = torch.softmax(z, -1) @ vs[:, a // (q // kv)]
    return _project(o.reshape(n, q * d), block.w_o, block.o_adapters, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("blocks", [0, 12])
def test_requests_fork_end_and_go_on(dtype, blocks):
    import adapter_sgmv_bgmv_gb300 as L
    ex = _example()
    ctx = L.Context(0, max_rows=1024)
    gen = torch.Generator(device="cuda").manual_seed(3)
    freqs = (1e4 ** (-torch.arange(16) / 16)).cuda()
    weights = [1 + 0.2 * torch.randn(64, generator=gen, device="cuda") for _ in range(2)]
    block = ex.random_block(ctx, cache_dtype=dtype, n_pages=40, rope=L.HeadRope(freqs, 64, *weights))
    req = ex.PagedRequests(ctx, [block.cache], 5, 40, 16, 190)
    adapters = np.array([2, 0, -1, 1, 2], np.int32)
    # what each request has been given: request 3 forks from 0 after three steps, 4 from 0 as well, 1 ends there
    told, got = [[] for _ in range(5)], [[] for _ in range(5)]

    def step(new, sparse):
        xs = [torch.randn((k, 512), generator=gen, device="cuda").to(torch.bfloat16) for k in new]
        y = block(torch.cat(xs), np.repeat(adapters, new), req.grow(np.array(new)), blocks=sparse)
        at = 0
        for s, k in enumerate(new):
            told[s].append(xs[s])
            got[s].append(y[at:at + k])
            at += k
    step([64, 20, 33, 0, 0], 0)
    step([38, 7, 64, 0, 0], 0)
    step([1, 1, 1, 0, 0], blocks)
    adapters[3] = adapters[4] = adapters[0]                # a fork goes on with its parent's adapter
    req.fork([0, 0], [3, 4])
    req.end([1])
    for s in (3, 4):
        told[s], got[s] = list(told[0]), list(got[0])
    told[1], got[1] = [], []
    for _ in range(20):
        step([1, 1, 1, 1, 1], blocks)
    ctx.sync_status()
    assert req.table.lens.tolist() == [123, 20, 118, 123, 123] and req.got.tolist() == [1] * 5
    refs = req.table.refs.tolist()
    # 103 tokens shared: six full pages of them held three times
    assert sorted(refs, reverse=True)[:7] == [3] * 6 + [1] and sum(refs) == 8 + 2 + 8 + 8 + 8
    # four roundings to bf16 of at most 2^-8 each (qkv with its rotation, weights, o, y); int8 keys and
    # values add a step of max / 127, a hundredth of a vector's size, each
    bound = 2e-2 if dtype == torch.bfloat16 else 4e-2
    for s in range(5):
        want = _whole(block, torch.cat(told[s]), int(adapters[s]), freqs, weights)
        have = torch.cat(got[s]).double()
        assert ((have - want).norm() / want.norm()).item() < bound
    ctx.close()


def test_a_captured_step_follows_table_and_lengths():
    """extend, copy, rotate and store, bounds, choice, attention: one graph, replayed while requests grow
    across pages, fork between replays and end; against eager steps on a second set of pools."""
    import adapter_sgmv_bgmv_gb300 as L
    ctx = L.Context(0, max_rows=64)
    n, page, heads, kv, dim, n_pages = 4, 8, 4, 2, 64, 60
    freqs = (1e4 ** (-torch.arange(32) / 32)).cuda()
    rope = L.HeadRope(freqs, dim)
    one = lambda v: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = (torch.empty((n, h, dim), dtype=torch.bfloat16, device="cuda") for h in (heads, kv, kv))

    class Side:
        def __init__(self):
            self.pool = torch.zeros((2, n_pages, page, kv, dim), dtype=torch.bfloat16, device="cuda")
            self.cache = L.KvCache(ctx, self.pool[0], self.pool[1])
            self.cache.attach_bounds(torch.zeros((n_pages, kv, 2, dim), dtype=torch.int8, device="cuda"), torch.zeros((n_pages, kv), device="cuda"))
            self.table = L.PageTable(one(0), torch.full((n, 12), -1, dtype=torch.int32, device="cuda"),
                                     torch.zeros(n_pages, dtype=torch.int32, device="cuda"), page)
            self.batch = L.KvBatch(torch.arange(n + 1, dtype=torch.int32, device="cuda"), self.table.lens, self.table.pages, max_new=1)
            self.sel = L.BlockSelection.empty(n, self.cache, 4)
            self.lists = [one(0) for _ in range(4)]
            self.qr, self.out = torch.empty_like(q), torch.empty_like(q)

        def step(self):
            L.lora_pages_extend(ctx, self.table, one_each, *self.lists)
            L.lora_kv_copy(ctx, self.cache, *self.lists[1:])
            L.lora_kv_write_rope(ctx, self.cache, rope, self.batch, q, k, v, self.qr)
            L.lora_kv_bounds(ctx, self.cache, self.batch, n)
            L.lora_block_select(ctx, self.cache, self.batch, self.qr, self.sel, 1, 1)
            L.lora_block_attention(ctx, self.cache, self.sel, self.qr, self.out)
    one_each = one(1)
    a, b = Side(), Side()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    gen = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for i in range(60):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        for side in (a, b):
            if i in (20, 41):
                L.lora_pages_free(ctx, side.table, ints(2, 3))
                L.lora_pages_fork(ctx, side.table, ints(0, 1), ints(2, 3))
        graph.replay()
        b.step()
        ctx.sync_status()
        for x, y in ((a.out, b.out), (a.qr, b.qr), (a.sel.pages, b.sel.pages), (a.table.pages, b.table.pages), (a.table.refs, b.table.refs)):
            assert torch.equal(x, y), i
    assert torch.equal(a.pool, b.pool) and a.table.lens.tolist() == [60] * 4
    ctx.close()

"""Steps for which the pool has too few pages: requests that get none keep every token that they
and those they share pages with have, eagerly and in a captured step, and go on once there is room."""
import numpy as np
import pytest
import torch

from tests.test_gpu_serving_step import _example
from tests.test_gpu_step_run import _whole

pytestmark = pytest.mark.gpu


def _cells(cache, table, lens):
    """Each sequence's keys and values, [tokens, 2, heads, dim]."""
    out = []
    for s, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        page, cell = table.pages[s].long()[j // table.page_size], j % table.page_size
        out.append(torch.stack([cache.k_pool[page, cell], cache.v_pool[page, cell]], 1))
    return out


def _kept(before, after):
    return all(torch.equal(b, a[:b.shape[0]]) for b, a in zip(before, after))


@pytest.mark.parametrize("blocks", [0, 12])
def test_a_refused_request_overwrites_nothing(blocks):
    import adapter_sgmv_bgmv_gb300 as L
    ex = _example()
    ctx = L.Context(0, max_rows=1024)
    gen = torch.Generator(device="cuda").manual_seed(11)
    freqs = (1e4 ** (-torch.arange(16) / 16)).cuda()
    block = ex.random_block(ctx, n_pages=6, rope=L.HeadRope(freqs, 64))
    req = ex.PagedRequests(ctx, [block.cache], 3, 6, 16, 80)
    adapters = np.array([2, 1, 2], np.int32)
    told, got = [[] for _ in range(3)], [[] for _ in range(3)]

    def step(new):
        lens = req.table.lens.tolist()
        before = _cells(block.cache, req.table, lens)
        xs = [torch.randn((k, 512), generator=gen, device="cuda").to(torch.bfloat16) for k in new]
        y = block(torch.cat(xs), np.repeat(adapters, new), req.grow(np.array(new)), blocks=blocks)
        ctx.sync_status()
        granted = req.got.tolist()
        assert req.table.lens.tolist() == [a + b for a, b in zip(lens, granted)]
        assert _kept(before, _cells(block.cache, req.table, lens))
        at = 0
        for s, k in enumerate(new):
            if granted[s]:
                told[s].append(xs[s])
                got[s].append(y[at:at + k])
            at += k
        return granted
    assert step([20, 30, 0]) == [20, 30, 0]
    req.fork([0], [2])
    told[2], got[2] = list(told[0]), list(got[0])
    # two pages are left: request 0 takes both, one of them in place of the page it shares, and 2 gets none;
    # later it asks for more than its row of five pages holds
    assert step([20, 1, 30]) == [20, 1, 0]
    assert step([8, 0, 1]) == [8, 0, 1]
    assert step([1, 0, 70]) == [0, 0, 0]
    req.end([1])
    assert step([0, 0, 33]) == [0, 0, 33]
    for s in (0, 2):
        want = _whole(block, torch.cat(told[s]), int(adapters[s]), freqs, [None, None])
        have = torch.cat(got[s]).double()
        # four roundings to bf16 of at most 2^-8 each (qkv with its rotation, weights, o, y)
        assert ((have - want).norm() / want.norm()).item() < 2e-2
    ctx.close()


def test_a_captured_step_without_pages_changes_no_token():
    """extend, lengths from what was got, copy, store, attention in one graph; three requests that share
    their last page and a pool with one page to spare: replays past its end leave every cell as it was."""
    import adapter_sgmv_bgmv_gb300 as L
    ctx = L.Context(0, max_rows=64)
    n, page, heads, kv, dim, n_pages = 3, 4, 4, 2, 64, 5
    one = lambda v: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(5)
    pool = torch.zeros((2, n_pages, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    cache = L.KvCache(ctx, pool[0], pool[1])
    table = L.PageTable(one(0), torch.full((n, 6), -1, dtype=torch.int32, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda"), page)
    lists, ask, lens, none = [one(0) for _ in range(4)], one(1), one(0), one(0)
    q, out = (torch.randn((n, heads, dim), generator=gen, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((n, kv, dim), generator=gen, device="cuda").bfloat16() for _ in range(2))
    # a prompt of 6 tokens, held by all three
    L.lora_pages_extend(ctx, table, ints(6, 0, 0), *lists)
    rows = [torch.randn((6, kv, dim), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    L.lora_kv_write(ctx, cache, L.KvBatch(ints(0, 6), table.lens[:1], table.pages[:1]), *rows)
    L.lora_pages_fork(ctx, table, ints(0, 0), ints(1, 2))
    batch = L.KvBatch(ints(0, 1, 2, 3), lens, table.pages, max_new=1)
    ctx.sync_status()

    def step():
        L.lora_pages_extend(ctx, table, ask, *lists)
        torch.where(lists[0] == ask, table.lens, none, out=lens)
        L.lora_kv_copy(ctx, cache, *lists[1:])
        L.lora_kv_write(ctx, cache, batch, k, v)
        L.lora_attention(ctx, cache, batch, q, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    granted = []
    for _ in range(7):
        for t in (k, v):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        had = table.lens.tolist()
        before = _cells(cache, table, had)
        graph.replay()
        ctx.sync_status()
        got = lists[0].tolist()
        granted.append(got)
        now = _cells(cache, table, table.lens.tolist())
        assert _kept(before, now)
        for s in range(n):
            if got[s]:
                assert torch.equal(now[s][-1], torch.stack([k[s], v[s]]))
            assert bool(out[s].any()) == bool(got[s])      # no position: zeros
    # 3 free pages: 0 and 1 take copies, 2 keeps the shared page; at 8 tokens each wants a page, and one is left
    assert granted == [[1, 1, 1], [1, 1, 1], [1, 0, 0], [1, 0, 0], [1, 0, 0], [1, 0, 0], [0, 0, 0]]
    cache.close()
    ctx.close()

"""Pages that something other than the table's sequences uses: pinned ones are neither handed out nor
moved, and keep what they hold; the others are compacted around them."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PIN = 1 << 30


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    assert L.PAGE_PINNED == PIN
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _compacted(refs, rows, n):
    """moves, refs, rows of pages and the end of the highest held page, one move after another."""
    refs = list(refs)
    held = [p for p, r in enumerate(refs) if 0 < r < PIN]
    free = [p for p, r in enumerate(refs) if r == 0]
    moves = [(a, b) for a, b in zip(held[::-1], free) if a > b][:n]
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    to = dict(moves)
    return moves, refs, [[to.get(p, p) for p in row] for row in rows], max([p + 1 for p, r in enumerate(refs) if r], default=0)


@pytest.mark.parametrize("n_pages", [1, 2, 33, 1000, 16384, 16385, 40000])
@pytest.mark.parametrize("seed", range(6))
def test_compaction_around_pinned_pages(ctx, n_pages, seed):
    """Pools of one CTA and of clusters; pins alone, in runs and all over; lists too short for all moves."""
    import adapter_sgmv_bgmv_gb300 as L
    rng, gen = random.Random(seed * 100003 + n_pages), np.random.default_rng(seed * 7 + n_pages)
    refs = (gen.random(n_pages) < rng.choice([0.02, 0.5, 0.97])).astype(np.int64)
    if seed % 3 == 2:
        refs[n_pages // 3:] = 0
    pins = gen.random(n_pages) < [0.0, 0.01, 0.3, 0.9, 0.2, 0.05][seed]
    if seed == 4:
        pins[: n_pages // 2] = False                       # all in the upper half, some where nobody else is
    if seed == 5:
        pins[n_pages // 4:n_pages // 2] = True
    # a sequence holds every other held page, pinned or not; something else has a count on the rest
    held = np.flatnonzero(refs)
    mine = gen.permutation(held)[: min(len(held) // 2, 4000)]
    refs = refs + PIN * pins
    refs = refs.tolist()
    moves = len(_compacted(refs, [], n_pages)[0])
    for n in {0, 1, min(moves, 7), moves // 2, moves, moves + 3}:
        table = L.PageTable(ints([len(mine)]), ints([mine.tolist() + [-1]]), ints(refs), 1)
        src, dst, top = ints([55] * n), ints([55] * n), ints([-5])
        L.lora_pages_compact(ctx, table, src, dst, top)
        ctx.sync_status()
        want, refs_after, rows, end = _compacted(refs, [mine.tolist()], n)
        pad = [-1] * (n - len(want))
        assert src.tolist() == [a for a, _ in want] + pad and dst.tolist() == [b for _, b in want] + pad
        assert table.refs.tolist() == refs_after and table.pages[0].tolist() == rows[0] + [-1]
        assert top.tolist() == [end]


def test_sequences_on_a_pinned_page(ctx):
    """Forks and ends count on it; who writes into it gets a copy; one too many gives back nothing."""
    import adapter_sgmv_bgmv_gb300 as L
    from adapter_sgmv_bgmv_gb300 import LoraError
    table = L.PageTable(ints([6, 0, 0]), ints([[1, 4, -1], [-1] * 3, [-1] * 3]), ints([PIN, 1, 0, 0, PIN + 1, 0]), 4)
    L.lora_pages_fork(ctx, table, ints([0]), ints([1]))
    ctx.sync_status()
    assert table.refs.tolist() == [PIN, 2, 0, 0, PIN + 2, 0]
    lists = [ints([0] * 3) for _ in range(4)]
    L.lora_pages_extend(ctx, table, ints([1, 1, 0]), *lists)
    ctx.sync_status()
    assert [v.tolist() for v in lists] == [[1, 1, 0], [4, 4, -1], [2, 3, -1], [2, 2, 0]]
    assert table.refs.tolist() == [PIN, 2, 1, 1, PIN, 0] and table.pages.tolist() == [[1, 2, -1], [1, 3, -1], [-1] * 3]
    for s in ([1], [0, 1]):                                # a table that is wrong: nobody's count to give back
        table.lens[:2] = 7
        table.pages[:2, 1] = 4
        L.lora_pages_free(ctx, table, ints(s), ints([4] * len(s)))
        with pytest.raises(LoraError) as e:
            ctx.sync_status()
        assert e.value.name == "LORA_E_PAGE" and table.refs.tolist()[4] == PIN
    L.lora_pages_free(ctx, table, ints([0, 1]))
    ctx.sync_status()
    assert table.refs.tolist() == [PIN, 0, 1, 1, PIN, 0]


def test_an_adapter_in_the_cache_s_pool_stays(ctx):
    """Compaction, then growth over the whole pool: the pinned pages hold what they held."""
    import adapter_sgmv_bgmv_gb300 as L
    n_pages, page, heads, dim = 40, 4, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    pool = torch.randn((n_pages, 2, page, heads, dim), generator=gen, device="cuda").bfloat16()
    cache = L.KvCache(ctx, pool[:, 0], pool[:, 1])
    adapter = [3, 17, 38, 39]
    refs = ints([0] * n_pages)
    for _ in range(2):                                     # once is enough
        refs[adapter] |= L.PAGE_PINNED
    was = pool[adapter].clone()
    table = L.PageTable(ints([0] * 3), torch.full((3, 40), -1, dtype=torch.int32, device="cuda"), refs, page)
    lists = [ints([0] * 3) for _ in range(4)]
    src, dst, top = ints([0] * n_pages), ints([0] * n_pages), ints([0])

    def grow(*new):
        L.lora_pages_extend(ctx, table, ints(list(new)), *lists)
        L.lora_kv_copy(ctx, cache, *lists[1:])
        rows = [torch.randn((sum(new), heads, dim), generator=gen, device="cuda").bfloat16() for _ in range(2)]
        L.lora_kv_write(ctx, cache, L.KvBatch(ints(np.cumsum([0, *new]).tolist()), table.lens, table.pages), *rows)
        ctx.sync_status()
        assert lists[0].tolist() == list(new)
        return rows
    grow(40, 30, 0)
    kept = grow(0, 0, 30)
    L.lora_pages_free(ctx, table, ints([0, 1]))
    L.lora_pages_compact(ctx, table, src, dst, top)
    L.lora_kv_copy(ctx, cache, src, dst)
    ctx.sync_status()
    # eight pages at the first eight places that are not the adapter's
    assert sorted(table.pages[2, :8].tolist()) == [0, 1, 2, 4, 5, 6, 7, 8] and top.tolist() == [40]
    grow(28 * page, 0, 0)                                  # all the rest of the pool
    assert torch.equal(pool[adapter], was)
    back = [torch.empty_like(r) for r in kept]
    L.lora_kv_read(ctx, cache, L.KvBatch(ints([0, 0, 0, 30]), table.lens, table.pages), *back)
    ctx.sync_status()
    assert torch.equal(back[0], kept[0]) and torch.equal(back[1], kept[1])
    cache.close()

"""Bounds of pages, the choice of pages by them and attention over what is chosen, against the models
in integers and 64 bits."""
import math
import random

import pytest
import torch

from tests._kv_ref import Case, assert_attention, raw
from tests._step_ref import bounds, chosen_attention, select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


class Step:
    """A Case with its cache and bounds, those of every page filled as earlier steps would have."""

    def __init__(self, ctx, case, max_new=None):
        import adapter_sgmv_bgmv_gb300 as L
        self.L, self.ctx, self.c = L, ctx, case
        self.cache = L.KvCache(ctx, case.k_pool, case.v_pool, case.k_scale, case.v_scale)
        n = case.k_pool.shape[0]
        self.codes = torch.full((n, case.kv_heads, 2, case.dim), 55, dtype=torch.int8, device="cuda")
        self.unit = torch.full((n, case.kv_heads), 3.0, device="cuda")
        self.cache.attach_bounds(self.codes, self.unit)
        self.batch = L.KvBatch(case.starts, case.lens_t, case.pages, max_new=max_new)

    def fill(self):
        """Bounds of all pages, by calls in which every token is new."""
        c = self.c
        starts = torch.tensor([0] + c.lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        if sum(c.lens):
            self.L.lora_kv_bounds(self.ctx, self.cache, self.L.KvBatch(starts, c.lens_t, c.pages), sum(c.lens))

    def choose(self, blocks, first, last):
        sel = self.L.BlockSelection.empty(self.c.n + 2, self.cache, blocks)
        sel.lens.fill_(-7)
        sel.pages.fill_(-7)
        self.L.lora_block_select(self.ctx, self.cache, self.batch, self.c.q, sel, first, last)
        return sel

    def close(self):
        self.cache.close()


def draw(seed):
    rng = random.Random(seed)
    kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
    seqs, hi = rng.choice([(1, 1), (1, 5), (3, 1), (5, 3), (17, 1), (2, 40)])
    page = rng.choice([1, 3, 16, 16, 24, 64])
    longest = rng.choice([20, 300, 1200]) * (1 if page < 16 else 2)
    new = [rng.randint(0 if seqs > 1 else 1, hi) for _ in range(seqs)]
    lens = [max(n, rng.randint(1, longest)) for n in new]
    for s in rng.sample(range(seqs), rng.choice([0, seqs // 3])):
        lens[s], new[s] = 0, 1
    if sum(new) == 0:
        new[0] = 1
        lens[0] = max(1, lens[0])
    blocks = rng.choice([1, 2, 5, 16, 40])
    first = rng.randint(0, min(3, blocks - 1))
    last = rng.randint(1, min(3, blocks - first))
    return dict(new=new, lens=lens, heads=kv_heads * rng.choice([1, 2, 3, 5, 8, 16, 20]), kv_heads=kv_heads, dim=rng.choice([64, 128]), page=page,
                fmt=rng.choice(["bf16", "int8", "fp8"]), layout=rng.choice(["split", "joint", "heads", "gaps"])), (blocks, first, last)


@pytest.mark.parametrize("seed", range(60))
def test_random_steps(ctx, seed):
    shape, how = draw(seed)
    c = Case(seed, **shape)
    st = Step(ctx, c)
    was = st.codes.clone(), st.unit.clone()
    st.L.lora_kv_bounds(ctx, st.cache, st.batch, c.n)
    ctx.sync_status()
    assert ctx.last_path() == (2048, 1)
    want = bounds(c, *was)
    assert torch.equal(st.codes, want[0]) and torch.equal(st.unit, want[1])
    st.fill()
    sel = st.choose(*how)
    ctx.sync_status()
    lens, pages = select(c, st.codes, st.unit, *how)
    assert torch.equal(sel.lens[:c.n].cpu(), lens) and torch.equal(sel.pages[:c.n].cpu(), pages)
    assert bool((sel.lens[c.n:] == -7).all()) and bool((sel.pages[c.n:] == -7).all())
    st.L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
    ctx.sync_status()
    assert ctx.last_path() == (64, 1)
    assert_attention(c.out, *chosen_attention(c, lens, pages))
    st.close()


@pytest.mark.parametrize("n_cols,page,heads,kv_heads", [(2000, 1, 4, 1), (9000, 1, 1, 1), (45056, 1, 2, 2), (1500, 16, 28, 4)])
def test_long_lists(ctx, n_cols, page, heads, kv_heads):
    """One (row, head) over a cluster of CTAs."""
    c = Case(n_cols, [2], [n_cols * page - page // 2], heads, kv_heads, 64, page)
    st = Step(ctx, c)
    st.fill()
    for how in ((7, 2, 3), (300, 0, 1)):
        sel = st.choose(*how)
        ctx.sync_status()
        lens, pages = select(c, st.codes, st.unit, *how)
        assert torch.equal(sel.lens[:2].cpu(), lens) and torch.equal(sel.pages[:2].cpu(), pages)
        st.L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
        ctx.sync_status()
        assert_attention(c.out, *chosen_attention(c, lens, pages))
    st.close()


def test_ties_go_to_the_first_pages(ctx):
    """Equal keys everywhere, queries of zero, and scores of either sign of zero."""
    c = Case(3, [1, 1], [1000, 900], 4, 2, 64, 4)
    raw(c.k_pool).copy_(raw(c.k_pool[:1, :1]).expand_as(c.k_pool))
    c.q[1] = 0
    st = Step(ctx, c)
    st.fill()
    sel = st.choose(9, 2, 3)
    ctx.sync_status()
    for s, cols in ((0, 250), (1, 225)):
        want = c.pages[s][list(range(6)) + list(range(cols - 3, cols))]
        assert torch.equal(sel.pages[s], want.expand(2, -1))
    st.close()


def test_keys_that_are_not_finite(ctx):
    """A page with one is chosen ahead of all others; NaNs behind a sequence's end are nobody's."""
    c = Case(4, [1], [64 * 16 + 3], 2, 1, 64, 16)
    k, v = c.rand(1, 1, 64), c.rand(1, 1, 64)
    k[0, 0, 5] = -math.inf
    c.put(0, [16 * 20 + 7], k, v)
    k[0, 0, 5] = math.nan
    c.put(0, [16 * 40 + 2], k, v)
    st = Step(ctx, c)
    was = st.codes.clone(), st.unit.clone()
    st.fill()
    ctx.sync_status()
    full = Case.__new__(Case)
    full.__dict__.update(c.__dict__, new=c.lens)
    want = bounds(full, *was)
    assert torch.equal(st.codes, want[0]) and torch.equal(st.unit.nan_to_num(-1), want[1].nan_to_num(-1))
    sel = st.choose(4, 1, 1)
    lens, pages = select(c, st.codes, st.unit, 4, 1, 1)
    assert torch.equal(sel.pages[:1].cpu(), pages)
    assert sel.pages[0, 0].tolist()[1:3] == [int(c.table[0, 20]), int(c.table[0, 40])]
    st.L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
    ctx.sync_status()
    assert bool(torch.isnan(c.out[0]).all())
    # a query head that is not finite has no say; alone, the first pages are as good as any
    c.q[0, 0, 1] = math.inf
    sel = st.choose(4, 1, 1)
    lens, pages = select(c, st.codes, st.unit, 4, 1, 1)
    ctx.sync_status()
    assert torch.equal(sel.pages[:1].cpu(), pages)
    st.close()


def test_values_of_chosen_pages_only(ctx):
    """NaNs in the pages that were not chosen, and behind the row's position, never reach the result."""
    c = Case(5, [1, 1], [50 * 16 + 5, 30 * 16], 8, 2, 128, 16)
    st = Step(ctx, c)
    st.fill()
    sel = st.choose(6, 1, 2)
    ctx.sync_status()
    lens, pages = sel.lens[:2].cpu(), sel.pages[:2].cpu()
    want = chosen_attention(c, lens, pages)
    for h in range(2):
        lost = torch.ones(c.k_pool.shape[0], dtype=torch.bool)
        lost[pages[:, h].flatten().long()] = False
        for pool in (c.k_pool, c.v_pool):
            pool[lost.cuda(), :, h] = math.nan
    st.L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
    ctx.sync_status()
    assert_attention(c.out, *want)
    st.close()


@pytest.mark.parametrize("gain", [1e-37, 1e-20, 1e18])
def test_extreme_sizes(ctx, gain):
    c = Case(6, [1], [500], 4, 2, 64, 8, gain=gain if gain > 1 else 1.0)
    if gain < 1:
        c.k_pool.mul_(gain)
    st = Step(ctx, c)
    was = st.codes.clone(), st.unit.clone()
    st.fill()
    ctx.sync_status()
    full = Case.__new__(Case)
    full.__dict__.update(c.__dict__, new=c.lens)
    want = bounds(full, *was)
    assert torch.equal(st.codes, want[0]) and torch.equal(st.unit, want[1])
    sel = st.choose(10, 1, 1)
    lens, pages = select(c, st.codes, st.unit, 10, 1, 1)
    ctx.sync_status()
    assert torch.equal(sel.pages[:1].cpu(), pages)
    st.close()


def test_rows_of_no_sequence_bad_pages_and_bad_sequences(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    from adapter_sgmv_bgmv_gb300 import LoraError
    c = Case(7, [1, 2, 1], [400, 300, 200], 4, 2, 64, 16)
    st = Step(ctx, c)
    st.fill()
    ctx.sync_status()
    q = torch.cat([c.q, c.rand(2, 4, 64)])
    out = torch.full_like(q, 7)
    c.lens_t[1] = 10 ** 6
    sel = L.BlockSelection.empty(6, st.cache, 5)
    for call in (lambda: L.lora_kv_bounds(ctx, st.cache, st.batch, 4),
                 lambda: L.lora_block_select(ctx, st.cache, st.batch, q, sel)):
        call()
        with pytest.raises(LoraError) as e:
            ctx.sync_status()
        assert e.value.name == "LORA_E_INVAL"
    assert sel.lens.tolist() == [(4 * 16) + (399 % 16) + 1, -1, -1, 4 * 16 + 199 % 16 + 1, -1, -1]
    L.lora_block_attention(ctx, st.cache, sel, q, out)
    ctx.sync_status()
    assert bool((out[[1, 2, 4, 5]] == 7).all()) and bool((out[[0, 3]] != 7).any(-1).all())
    c.lens_t[1] = 300
    c.pages[0, 3], c.pages[2, 12] = -1, 10 ** 6
    L.lora_kv_bounds(ctx, st.cache, st.batch, 4)
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_PAGE"
    L.lora_block_select(ctx, st.cache, st.batch, q, sel)
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_PAGE"
    assert -1 not in sel.pages[0].tolist()[0]              # chosen last
    L.lora_block_attention(ctx, st.cache, sel, q, out)     # the last row's own page is not there
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_PAGE"
    st.close()


def test_all_pages_chosen_is_attention(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(8, [1, 3, 1], [100, 77, 0], 8, 2, 128, 16, fmt="int8")
    st = Step(ctx, c)
    sel = st.choose(7, 3, 2)
    L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
    ctx.sync_status()
    want, bound = c.reference()
    assert_attention(c.out, want, bound)
    st.close()


def test_scale_and_many_heads(ctx):
    """More query heads than one unit has rows, and a scale of one's own."""
    c = Case(9, [2], [700], 128, 1, 64, 16, fmt="fp8")
    st = Step(ctx, c)
    st.fill()
    sel = st.choose(12, 1, 1)
    lens, pages = select(c, st.codes, st.unit, 12, 1, 1)
    assert torch.equal(sel.pages[:2].cpu(), pages)
    st.L.lora_block_attention(ctx, st.cache, sel, c.q, c.out, scale=0.31)
    ctx.sync_status()
    assert_attention(c.out, *chosen_attention(c, lens, pages, scale=0.31))
    st.close()


def test_results_repeat_and_replay(ctx):
    """The same bits on every run, on a stream and in replays that follow the lengths; two graphs in turn."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(10, [1] * 4, [5000, 3000, 40, 2500], 8, 2, 128, 16)
    st = Step(ctx, c, max_new=1)
    st.fill()
    ctx.sync_status()
    sels = [L.BlockSelection.empty(4, st.cache, b) for b in (20, 6)]
    outs = [torch.empty_like(c.out) for _ in sels]

    def step(i):
        L.lora_kv_bounds(ctx, st.cache, st.batch, 4)
        L.lora_block_select(ctx, st.cache, st.batch, c.q, sels[i], 1, 1)
        L.lora_block_attention(ctx, st.cache, sels[i], c.q, outs[i])
    graphs = [torch.cuda.CUDAGraph() for _ in sels]
    for i, g in enumerate(graphs):
        step(i)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            step(i)
    for lens in ([5000, 3000, 40, 2500], [4800, 0, 33, 17], [4801, 1, 34, 18]):
        c.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
        want = []
        for i in range(2):
            step(i)
            ctx.sync_status()
            want.append((outs[i].clone(), sels[i].pages.clone(), sels[i].lens.clone()))
        for _ in range(3):
            for g in graphs:
                g.replay()
        ctx.sync_status()
        for i in range(2):
            assert torch.equal(outs[i], want[i][0]) and torch.equal(sels[i].pages, want[i][1]) and torch.equal(sels[i].lens, want[i][2])
    st.close()


def test_batches_without_rows_or_sequences(ctx):
    """Every row of a call without sequences belongs to none: its length is -1, and attention leaves it alone."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(11, [1], [40], 4, 2, 64, 16)
    st = Step(ctx, c)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    empty = L.KvBatch(none, none[:0], torch.zeros((0, 3), dtype=torch.int32, device="cuda"))
    q = c.rand(3, 4, 64)
    out = torch.full_like(q, 7)
    sel = L.BlockSelection.empty(3, st.cache, 2)
    sel.lens.fill_(5)
    L.lora_kv_bounds(ctx, st.cache, empty, 3)
    L.lora_block_select(ctx, st.cache, empty, q, sel)
    L.lora_block_attention(ctx, st.cache, sel, q, out)
    ctx.sync_status()
    assert sel.lens.tolist() == [-1] * 3 and bool((out == 7).all())
    L.lora_kv_bounds(ctx, st.cache, st.batch, 0)
    L.lora_block_select(ctx, st.cache, st.batch, q[:0], sel)
    L.lora_block_attention(ctx, st.cache, sel, q[:0], out[:0])
    ctx.sync_status()
    assert ctx.last_path() == (0, 0)
    st.close()


def test_a_selection_of_ones_own(ctx):
    """Any pages in any order, one of them twice, lengths that end inside a page; one too long is refused."""
    import adapter_sgmv_bgmv_gb300 as L
    from adapter_sgmv_bgmv_gb300 import LoraError
    c = Case(12, [1, 1, 1], [200, 90, 40], 4, 2, 64, 16)
    st = Step(ctx, c)
    ids = [[[5, 0, 3], [0, 5, 5]], [[1, 2, 4], [2, 1, 0]], [[2, -1, -1], [0, -1, -1]]]
    sel = L.BlockSelection(torch.tensor([37, 48, 1], dtype=torch.int32, device="cuda"), torch.tensor(ids, dtype=torch.int32, device="cuda"))
    # pages of the table: those have been written
    for s in range(3):
        for h in range(2):
            for i in range(3):
                if ids[s][h][i] >= 0:
                    sel.pages[s, h, i] = int(c.table[0, ids[s][h][i]])
    L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
    ctx.sync_status()
    assert_attention(c.out, *chosen_attention(c, sel.lens.cpu(), sel.pages.cpu()))
    before = c.out.clone()
    sel.lens[1] = 49
    L.lora_block_attention(ctx, st.cache, sel, c.q, c.out.fill_(3))
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_INVAL"
    assert torch.equal(c.out[[0, 2]], before[[0, 2]]) and bool((c.out[1] == 3).all())
    st.close()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_values_that_are_not_finite(ctx, fmt):
    """An infinity among the values of a token that a row sees reaches its own element only; a NaN, as an
    8-bit vector keeps it, the whole vector's elements; tokens behind the row's length neither."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(13, [1, 1], [200, 100], 12, 2, 128, 16, fmt=fmt)
    k, v = c.rand(1, 2, 128), c.rand(1, 2, 128)
    v[0, 1, 7] = math.inf
    c.put(0, [50], k, v)                                    # its page is listed for both heads
    c.put(1, [99], *(x.clone() for x in (k, v)))            # behind the second row's length
    st = Step(ctx, c)
    ids = c.pages[:, [0, 1, 3, 6]].clone()
    sel = L.BlockSelection(torch.tensor([61, 51], dtype=torch.int32, device="cuda"), ids[:, None].expand(2, 2, 4).contiguous())
    L.lora_block_attention(ctx, st.cache, sel, c.q, c.out)
    ctx.sync_status()
    lost = ~torch.isfinite(c.out)
    want = torch.zeros_like(lost)
    if fmt == "bf16":
        want[0, 6:, 7] = True
        assert bool((c.out[0, 6:, 7] == math.inf).all())
    else:
        want[0, 6:] = True
    assert torch.equal(lost, want)
    st.close()


def test_offsets_beyond_32_bits(ctx):
    """Pages beyond 2^32 bytes of a 6 GB pool, for the store, the bounds, the choice and the attention."""
    import adapter_sgmv_bgmv_gb300 as L
    n_pages, page, kv, dim = 24000, 16, 64, 128
    pool = torch.empty((n_pages, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    cache = L.KvCache(ctx, pool, torch.empty_like(pool))
    cache.attach_bounds(torch.zeros((n_pages, kv, 2, dim), dtype=torch.int8, device="cuda"), torch.zeros((n_pages, kv), device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(0)
    m = 16 * 9 + 5
    rows = [torch.randn((m, kv, dim), generator=gen, device="cuda").bfloat16() for _ in range(3)]
    outs = []
    rope = L.HeadRope((1e4 ** (-torch.arange(64) / 64)).cuda(), dim)
    for first in (0, 23990):                                # the same tokens at both ends of the pool
        pages = torch.arange(first, first + 10, dtype=torch.int32, device="cuda")[None]
        lens = torch.tensor([m], dtype=torch.int32, device="cuda")
        batch = L.KvBatch(torch.tensor([0, m], dtype=torch.int32, device="cuda"), lens, pages)
        q = torch.empty_like(rows[0])
        L.lora_kv_write_rope(ctx, cache, rope, batch, rows[0], rows[1], rows[2], q)
        L.lora_kv_bounds(ctx, cache, batch, m)
        sel = L.BlockSelection.empty(m, cache, 4)
        L.lora_block_select(ctx, cache, batch, q, sel)
        out = torch.empty_like(q)
        L.lora_block_attention(ctx, cache, sel, q, out)
        ctx.sync_status()
        chosen = torch.where(sel.pages >= 0, sel.pages - first, -1)
        outs.append((q, chosen, sel.lens, out, pool[first:first + 9].clone(), cache.bounds[0][first:first + 10].clone()))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    cache.close()

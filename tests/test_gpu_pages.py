"""Page tables and copies of pages, against lists that change one sequence after another."""
import random

import numpy as np
import pytest
import torch

from tests._kv_ref import DTYPE, pools, raw
from tests._step_ref import Pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """A model and the library's table, held to one another after every call."""

    def __init__(self, ctx, n_seqs, n_cols, n_pages, page):
        import adapter_sgmv_bgmv_gb300 as L
        self.L, self.ctx, self.m = L, ctx, Pages(n_seqs, n_cols, n_pages, page)
        wide = torch.full((n_seqs, n_cols + 3), -9, dtype=torch.int32, device="cuda")     # a row stride of its own
        self.lens, self.pages, self.refs = ints([0] * n_seqs), wide[:, :n_cols], ints([0] * n_pages)
        self.pages.fill_(-1)
        self.wide = wide
        self.table = L.PageTable(self.lens, self.pages, self.refs, page)
        self.lists = [torch.full((n_seqs,), 99, dtype=torch.int32, device="cuda") for _ in range(4)]

    def same(self):
        self.ctx.sync_status()
        for got, want in zip((self.lens, self.pages, self.refs), self.m.arrays()):
            assert np.array_equal(got.cpu().numpy(), want)
        assert bool((self.wide[:, self.pages.shape[1]:] == -9).all())

    def extend(self, grow):
        self.L.lora_pages_extend(self.ctx, self.table, ints(grow), *self.lists)
        want = self.m.extend(grow)
        self.same()
        assert [v.tolist() for v in self.lists] == [list(v) for v in want]
        return want

    def fork(self, parents, children):
        self.L.lora_pages_fork(self.ctx, self.table, ints(parents), ints(children))
        self.m.fork(parents, children)
        self.same()

    def free(self, seqs, keep=None):
        self.L.lora_pages_free(self.ctx, self.table, ints(seqs), None if keep is None else ints(keep))
        self.m.free(seqs, keep)
        self.same()

    def compact(self, n, with_top=True):
        src, dst, top = ints([55] * n), ints([55] * n), ints([-5])
        self.L.lora_pages_compact(self.ctx, self.table, src, dst, top if with_top else None)
        want = self.m.compact(n)
        self.same()
        assert src.tolist() == want[0] and dst.tolist() == want[1]
        assert top.tolist() == [want[2] if with_top else -5]
        return src, dst


@pytest.mark.parametrize("seed", range(30))
def test_random_lives(ctx, seed):
    rng = random.Random(seed)
    n, page = rng.choice([1, 3, 17, 70]), rng.choice([1, 3, 16, 64])
    cols = rng.choice([4, 9, 40])
    b = Both(ctx, n, cols, rng.choice([5, 40, 200, 1500]), page)
    for _ in range(25):
        what = rng.choice(["extend", "extend", "extend", "fork", "free", "trim", "compact"])
        if what == "extend":
            hi = rng.choice([1, 2, 2 * page + 1, cols * page + 2])
            b.extend([rng.choice([0, -1, 1, rng.randint(1, hi)]) for _ in range(n)])
        elif what == "fork":
            empty = [s for s in range(n) if not b.m.lens[s]]
            full = [s for s in range(n) if b.m.lens[s]] or [s for s in range(n) if s not in empty[:1]]
            if empty and full:
                some = rng.sample(empty, rng.randint(1, len(empty)))
                some = [s for s in some if s not in full]
                b.fork([rng.choice(full) for _ in some], some)
        elif what == "free":
            b.free(rng.sample(range(n), rng.randint(0, n)))
        elif what == "trim":
            some = rng.sample(range(n), rng.randint(1, n))
            b.free(some, [rng.randint(0, b.m.lens[s] + 2) for s in some])
        else:
            b.compact(rng.choice([1, 2, 7, len(b.m.refs)]), rng.random() < 0.8)


@pytest.mark.parametrize("n_pages", [1, 31, 32, 16384, 16385, 100003, 400000, 1 << 20])
def test_pools_of_every_size(ctx, n_pages):
    """One CTA up to a cluster of eight; most pages are held by something else."""
    b = Both(ctx, 5, 300, n_pages, 2)
    held = np.random.default_rng(n_pages).random(n_pages) < 0.97
    held[: n_pages // 2] |= n_pages > 1000
    b.refs.copy_(torch.from_numpy(held.astype(np.int32)))
    b.m.refs = held.astype(int).tolist()
    b.extend([3, 0, 500, 1, 101])
    b.extend([3, 1, 7, 1, 101])
    b.free([2, 0])
    b.compact(min(n_pages, 4000))
    b.compact(5)
    b.extend([50, 50, 50, 50, 50])


def test_many_sequences(ctx):
    rng = random.Random(1)
    b = Both(ctx, 5000, 3, 9000, 4)
    b.extend([rng.randint(0, 9) for _ in range(5000)])
    b.free(rng.sample(range(5000), 2500))
    b.extend([rng.randint(0, 12) for _ in range(5000)])
    b.compact(9000)
    left = [s for s in range(5000) if b.m.lens[s]]
    empty = [s for s in range(5000) if not b.m.lens[s]]
    b.fork([rng.choice(left[:3]) for _ in empty], empty)
    b.extend([1] * 5000)                                   # hundreds write into one shared page


def test_the_last_writer_keeps_a_shared_page(ctx):
    b = Both(ctx, 6, 4, 20, 4)
    b.extend([6, 0, 0, 0, 0, 0])
    b.fork([0, 0, 0], [2, 4, 5])
    got, src, dst, cells = b.extend([1, 0, 1, 0, 1, 1])
    assert src == [1, -1, 1, -1, 1, -1] and cells == [2, 0, 2, 0, 2, 0] and dst == [2, -1, 3, -1, 4, -1]
    b.fork([5], [1])
    got, src, dst, cells = b.extend([0, 0, 0, 0, 0, 1])    # sequence 1 holds it too
    assert src[5] == 1 and cells[5] == 3


def test_out_of_pages_leaves_the_rest_as_it_was(ctx):
    b = Both(ctx, 4, 8, 5, 4)
    assert b.extend([8, 9, 5, 1])[0] == [8, 9, 0, 0]
    b.free([0])
    assert b.extend([0, 3, 30, 1])[0] == [0, 3, 0, 0]
    assert b.extend([0, 30, 1, 1])[0] == [0, 0, 1, 1]      # a row too short does not stop the others


def test_bad_lists_and_tables_change_nothing(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    from adapter_sgmv_bgmv_gb300 import LoraError

    def refuses(name, call):
        before = [t.clone() for t in (b.lens, b.pages, b.refs)]
        call()
        with pytest.raises(LoraError) as e:
            ctx.sync_status()
        assert e.value.name == name
        return [torch.equal(x, y) for x, y in zip(before, (b.lens, b.pages, b.refs))]
    b = Both(ctx, 4, 4, 12, 4)
    b.extend([7, 5, 0, 0])
    all_same = [True] * 3
    fork = lambda a, c: (lambda: L.lora_pages_fork(ctx, b.table, ints(a), ints(c)))  # noqa: E731
    free = lambda s, k=None: (lambda: L.lora_pages_free(ctx, b.table, ints(s), None if k is None else ints(k)))  # noqa: E731
    for call in (fork([0], [1]), fork([0], [0]), fork([0], [4]), fork([-1], [2]), fork([4], [2]), fork([0], [-1]),
                 free([4]), free([-1]), free([1], [-1])):
        assert refuses("LORA_E_INVAL", call) == all_same
    # a child that is another's parent in the same call: neither order would be right
    assert refuses("LORA_E_INVAL", fork([0, 2], [2, 3])) == [False] * 3
    b.m.fork([0], [2])
    b.ctx.sync_status()
    for got, want in zip((b.lens, b.pages, b.refs), b.m.arrays()):
        assert np.array_equal(got.cpu().numpy(), want)
    # the same index twice: the first one counts
    refuses("LORA_E_INVAL", fork([1, 0], [3, 3]))
    b.m.fork([1], [3])
    refuses("LORA_E_INVAL", free([3, 0, 3], [2, 3, 0]))
    b.m.free([3, 0], [2, 3])
    b.same()
    # a page that the pool does not have, and one that nobody holds
    b.pages[0, 0] = 12
    refuses("LORA_E_PAGE", free([0]))
    b.m.refs[b.m.rows[0][0]] += 1                          # still counted
    b.m.free([0])
    b.same()
    b.refs[b.m.rows[1][0]] = 0
    refuses("LORA_E_PAGE", free([1]))
    b.m.refs[b.m.rows[1][0]] = 1
    b.m.free([1])
    b.same()
    b.lens[2] = 1000
    got = refuses("LORA_E_INVAL", lambda: L.lora_pages_extend(ctx, b.table, ints([1] * 4), *b.lists))
    assert b.lists[0].tolist() == [1, 1, 0, 1] and int(b.lens[2]) == 1000, got


def test_empty_calls(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    none = ints([])
    t = L.PageTable(none, torch.empty((0, 4), dtype=torch.int32, device="cuda"), ints([1, 0, 2]), 16)
    L.lora_pages_extend(ctx, t, none, none, none, none, none)
    L.lora_pages_fork(ctx, t, none, none)
    L.lora_pages_free(ctx, t, none)
    src, dst, top = ints([7, 7]), ints([7, 7]), ints([7])
    L.lora_pages_compact(ctx, t, src, dst, top)            # pages that others hold move as well
    ctx.sync_status()
    assert src.tolist() == [2, -1] and dst.tolist() == [1, -1] and top.tolist() == [2] and t.refs.tolist() == [1, 2, 0]
    t = L.PageTable(none, torch.empty((0, 4), dtype=torch.int32, device="cuda"), ints([1, 0, 2]), 16)
    L.lora_pages_compact(ctx, t, none, none, top)          # room for no move: only the end
    ctx.sync_status()
    assert top.tolist() == [3]


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("layout", ["split", "joint", "heads", "gaps"])
@pytest.mark.parametrize("page,heads,dim", [(16, 8, 128), (1, 1, 64), (24, 3, 64), (128, 5, 128), (7, 33, 128)])
def test_copies(ctx, fmt, layout, page, heads, dim):
    import adapter_sgmv_bgmv_gb300 as L
    gen = torch.Generator(device="cuda").manual_seed(page * heads + dim)
    n_pages, caches, kept = 40, [], []
    for _ in range(3):
        k, v, ks, vs = pools(n_pages, page, heads, dim, fmt, layout, "cuda")
        for t in (k, v):
            raw(t).copy_(torch.randint(-100, 100, t.shape, generator=gen, device="cuda"))
        for t in (ks, vs):
            if t is not None:
                t.copy_(torch.rand(t.shape, generator=gen, device="cuda"))
        caches.append(L.KvCache(ctx, k, v, ks, vs))
        kept.append([t for t in (k, v, ks, vs) if t is not None])
    codes = torch.randint(-127, 127, (n_pages, heads, 2, dim), generator=gen, device="cuda").to(torch.int8)
    unit = torch.rand((n_pages, heads), generator=gen, device="cuda")
    caches[1].attach_bounds(codes, unit)
    order = np.random.default_rng(page).permutation(n_pages)
    src, dst = order[:12].copy(), order[12:24]
    src[[3, 4, 9]] = -1
    cells = np.array([0, 1, page, page + 5, 1, page - 1, page, page, 2, 3, 4, -2])
    for use in (None, cells):
        want = []
        for t in [x for ts in kept for x in ts]:
            w = (raw(t) if t.dim() == 4 else t).clone()
            for i in range(12):
                if src[i] >= 0:
                    m = page if use is None else min(max(int(use[i]), 0), page)
                    w[dst[i], :m] = w[src[i], :m]
            want.append(w)
        c2, u2 = codes.clone(), unit.clone()
        on = src >= 0
        c2[dst[on]], u2[dst[on]] = c2[src[on]], u2[src[on]]
        L.lora_kv_copy(ctx, caches, ints(src.tolist()), ints(dst.tolist()), None if use is None else ints(use.tolist()))
        ctx.sync_status()
        assert ctx.last_path() == (1024, 1)
        for t, w in zip([x for ts in kept for x in ts], want):
            assert torch.equal(raw(t) if t.dim() == 4 else t, w)
        assert torch.equal(codes, c2) and torch.equal(unit, u2)
    for c in caches:
        c.close()


def test_copies_of_many_caches_and_long_lists(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    pool = torch.randn((70, 2, 9001, 2, 1, 64), device="cuda").bfloat16()
    caches = [L.KvCache(ctx, p[0], p[1]) for p in pool]
    src, dst = np.full(4500 * 2, -1), np.full(4500 * 2, -1)
    at = np.random.default_rng(0).choice(9000, 3000, replace=False)
    order = np.random.default_rng(1).permutation(9001)
    src[at], dst[at] = order[:3000], order[3000:6000]
    want = pool.clone()
    want[:, :, torch.from_numpy(dst[at]).cuda()] = pool[:, :, torch.from_numpy(src[at]).cuda()]
    L.lora_kv_copy(ctx, caches, ints(src.tolist()), ints(dst.tolist()))
    ctx.sync_status()
    assert ctx.last_path() == (1024, 2)                    # 64 caches a launch
    assert torch.equal(pool, want)
    for c in caches:
        c.close()


def test_copies_of_pages_that_are_not_there(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    from adapter_sgmv_bgmv_gb300 import LoraError
    pool = torch.randn((2, 8, 4, 2, 64), device="cuda").bfloat16()
    cache = L.KvCache(ctx, pool[0], pool[1])
    want = pool.clone()
    want[:, 5] = pool[:, 2]
    L.lora_kv_copy(ctx, cache, ints([8, 1, 2, 1 << 30, 3]), ints([0, 8, 5, 1, -1]))
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_PAGE" and torch.equal(pool, want)
    cache.close()


def test_copies_beyond_32_bits(ctx):
    """Pools of 6 GB: offsets beyond 2^32 bytes, elements beyond 2^31."""
    import adapter_sgmv_bgmv_gb300 as L
    k = torch.empty((24000, 16, 64, 128), dtype=torch.int8, device="cuda")
    ks = torch.ones((24000, 16, 64), device="cuda")
    cache = L.KvCache(ctx, k, k, ks, ks)
    gen = torch.Generator(device="cuda").manual_seed(0)
    k[23999] = torch.randint(-99, 99, k.shape[1:], generator=gen, device="cuda").to(torch.int8)
    k[1].zero_()
    L.lora_kv_copy(ctx, cache, ints([23999]), ints([1]))
    L.lora_kv_copy(ctx, cache, ints([1]), ints([23998]))
    ctx.sync_status()
    assert torch.equal(k[1], k[23999]) and torch.equal(k[23998], k[23999]) and bool(k[1].any())
    cache.close()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_sequences_keep_their_tokens(ctx, fmt):
    """Prompts, forks, writes into shared pages, ends and compactions, in two layers: what is read
    back for each sequence is what was written for it and for what it forked from."""
    import adapter_sgmv_bgmv_gb300 as L
    rng = random.Random(4)
    n, cols, page, heads, dim = 9, 20, 4, 2, 64
    b = Both(ctx, n, cols, 150, page)
    layers = []
    for _ in range(2):
        pool = torch.zeros((2, 150, page, heads, dim), dtype=DTYPE[fmt], device="cuda")
        sc = (None, None) if fmt == "bf16" else torch.zeros((2, 150, page, heads), device="cuda").unbind(0)
        layers.append(L.KvCache(ctx, pool[0], pool[1], *sc))
    told = [[] for _ in range(n)]                          # a number for each token
    count = 0

    def vectors(tokens, layer):
        # distinct for each token, exact in bf16 and in 8 bits (largest magnitude 127)
        t = torch.tensor(tokens, device="cuda", dtype=torch.int64)
        x = torch.stack([(t // 255 ** i % 255 - 127).float() for i in range(3)], -1)
        x = torch.cat([x, torch.full((len(tokens), 1), 127.0, device="cuda"), torch.full((len(tokens), dim - 4), float(layer), device="cuda")], -1)
        return x[:, None].expand(-1, heads, -1).bfloat16().contiguous()
    for step in range(40):
        grow = [rng.choice([0, 1, 1, rng.randint(1, 9)]) if len(told[s]) < 60 else 0 for s in range(n)]
        got, src, dst, cells = b.extend(grow)
        lists = b.lists
        L.lora_kv_copy(ctx, layers, lists[1], lists[2], lists[3])
        starts = ints(np.concatenate([[0], np.cumsum(got)]).tolist())
        batch = L.KvBatch(starts, b.lens, b.pages)
        new = []
        for s in range(n):
            mine = list(range(count, count + got[s]))
            count += got[s]
            told[s] += mine
            new += mine
        if new:
            for i, cache in enumerate(layers):
                x = vectors(new, i)
                L.lora_kv_write(ctx, cache, batch, x, -x)
        empty = [s for s in range(n) if not told[s]]
        full = [s for s in range(n) if told[s]]
        if empty and full and rng.random() < 0.6:
            some = rng.sample(empty, rng.randint(1, len(empty)))
            parents = [rng.choice(full) for _ in some]
            b.fork(parents, some)
            for a, c in zip(parents, some):
                told[c] = list(told[a])
        if rng.random() < 0.5:
            some = rng.sample(range(n), rng.randint(1, 4))
            keep = [rng.choice([0, 0, rng.randint(0, len(told[s]))]) for s in some]
            b.free(some, keep)
            for s, k in zip(some, keep):
                told[s] = told[s][:k]
        if rng.random() < 0.4:
            m1, m2 = b.compact(rng.choice([3, 150]))
            L.lora_kv_copy(ctx, layers, m1, m2)
        all_rows = [t for s in range(n) for t in told[s]]
        if not all_rows:
            continue
        whole = L.KvBatch(ints(np.concatenate([[0], np.cumsum([len(t) for t in told])]).tolist()), b.lens, b.pages)
        for i, cache in enumerate(layers):
            want = vectors(all_rows, i)
            back = [torch.empty_like(want) for _ in range(2)]
            L.lora_kv_read(ctx, cache, whole, *back)
            ctx.sync_status()
            assert torch.equal(back[0], want) and torch.equal(back[1], -want), step
    for c in layers:
        c.close()


def test_captured_steps(ctx):
    """extend and the copies it asks for, captured once: replays follow the table."""
    import adapter_sgmv_bgmv_gb300 as L
    b = Both(ctx, 3, 8, 30, 4)
    b.extend([6, 0, 0])
    b.fork([0, 0], [1, 2])
    grow = ints([1, 1, 1])
    pool = torch.randn((2, 30, 4, 2, 64), device="cuda").bfloat16()
    cache = L.KvCache(ctx, pool[0], pool[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            L.lora_pages_extend(ctx, b.table, grow, *b.lists)
            L.lora_kv_copy(ctx, cache, *b.lists[1:])
        for _ in range(6):
            before = pool.clone()
            graph.replay()
            want = b.m.extend([1, 1, 1])
            side.synchronize()
            b.same()
            assert [v.tolist() for v in b.lists] == [list(v) for v in want]
            for s, d, m in zip(*want[1:]):
                if s >= 0:
                    before[:, d, :m] = before[:, s, :m]
            assert torch.equal(pool, before)
    cache.close()

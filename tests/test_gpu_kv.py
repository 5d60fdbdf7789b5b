"""The paged key/value cache and attention over it, against the 64-bit model: formats,
layouts, page sizes, shared heads, ragged and empty rows, windows, values that must not
leak out of masked places, bad device data, streams and graphs."""
import math

import numpy as np
import pytest
import torch

from tests._kv_ref import DTYPE, Case, assert_attention, quantise, random_batch, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def handles(ctx, c, max_new=None):
    import adapter_sgmv_bgmv_gb300 as L
    return (L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale),
            L.KvBatch(c.starts, c.lens_t, c.pages, max_new=max_new))


def attend(ctx, c, max_new=None, **kw):
    import adapter_sgmv_bgmv_gb300 as L
    cache, batch = handles(ctx, c, max_new)
    L.lora_attention(ctx, cache, batch, c.q, c.out, **kw)
    ctx.sync_status()
    return c.out


def check(ctx, c, max_new=None, **kw):
    want, bound = c.reference(**kw)
    assert_attention(attend(ctx, c, max_new, **kw), want, bound)


# ---------------------------------------------------------------- write and read

@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("layout", ["split", "joint", "heads", "gaps"])
@pytest.mark.parametrize("dim,heads,page", [(128, 8, 16), (64, 3, 24), (128, 1, 1), (64, 32, 64), (128, 33, 7)])
def test_write_then_read(ctx, fmt, layout, dim, heads, page):
    import adapter_sgmv_bgmv_gb300 as L
    new, lens = random_batch(dim + heads, 9, 40, 130, released=2)
    new[3] = lens[3] + 5                       # five rows ahead of position 0
    c = Case(5, new, lens, heads, heads, dim, page, fmt, layout, fill=False)
    k, v = c.rand(c.n, heads, dim), c.rand(c.n, heads, dim)
    v[1] *= 1e-3
    k[0, 0] = 0
    cache, batch = handles(ctx, c)
    L.lora_kv_write(ctx, cache, batch, k, v)
    ctx.sync_status()
    got = [None if t is None else t.clone() for t in (c.k_pool, c.v_pool, c.k_scale, c.v_scale)]
    # the same stores by the model, on pools in their first state
    m = Case(5, new, lens, heads, heads, dim, page, fmt, layout, fill=False)
    back = []
    for x, what in ((k, "k"), (v, "v")):
        y = torch.zeros((c.n, heads, dim), dtype=torch.bfloat16, device="cuda")
        for s in range(len(lens)):
            n = min(new[s], lens[s])
            if n:
                rows = slice(int(c.start[s + 1]) - n, int(c.start[s + 1]))
                js = range(lens[s] - n, lens[s])
                m.put(s, js, k[rows], v[rows])
                y[rows] = m.get(s, lens[s], what)[lens[s] - n:].float().to(torch.bfloat16)
        back.append(y)
    for a, b in zip(got, (m.k_pool, m.v_pool, m.k_scale, m.v_scale)):
        if a is not None:
            assert torch.equal(raw(a) if a.dtype != torch.float32 else a.contiguous().view(torch.int32),
                               raw(b) if b.dtype != torch.float32 else b.contiguous().view(torch.int32))
    kb, vb = torch.full_like(k, 9), torch.full_like(v, 9)
    L.lora_kv_read(ctx, cache, batch, kb, vb)
    ctx.sync_status()
    assert torch.equal(raw(kb), raw(back[0])) and torch.equal(raw(vb), raw(back[1]))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_read_is_exact_over_every_code(ctx, fmt):
    """Every 8-bit code (NaN codes of e4m3 too) times a scale, rounded once to bf16."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(1, [4], [4], 1, 1, 64, 4, fmt)
    p, cell = c.cells(0, range(4))
    codes = torch.arange(256, dtype=torch.int16, device="cuda").to(torch.int8).view(4, 1, 64)
    for pool, scale in ((c.k_pool, c.k_scale), (c.v_pool, c.v_scale)):
        raw(pool)[p, cell] = codes
        scale[p, cell] = torch.tensor([[0.0123], [1.0], [3e-39], [7e30]], device="cuda")
    k, v = torch.empty((4, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache, batch = handles(ctx, c)
    L.lora_kv_read(ctx, cache, batch, k, v)
    ctx.sync_status()
    want = (raw(c.k_pool)[p, cell].view(DTYPE[fmt]).float() * c.k_scale[p, cell][..., None]).to(torch.bfloat16)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(k), nan) and torch.equal(k[~nan], want[~nan]) and torch.equal(raw(k), raw(v))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_write_quantises_extreme_vectors(ctx, fmt):
    """Subnormal, huge and exact-tie vectors as the model; a vector with an infinity or a
    NaN reads back as NaN and leaves its neighbours alone."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(2, [8], [8], 2, 2, 128, 8, fmt, fill=False)
    k, v = c.rand(8, 2, 128), c.rand(8, 2, 128)
    k[0, 0] *= 2.0 ** -130
    k[1, 1] *= 2.0 ** 120
    k[2, 0] = torch.arange(128, device="cuda").to(torch.bfloat16) / 2 + 0.5     # ties of int8 steps of 1
    k[2, 0, 0] = 127
    k[3, 0, 5] = math.inf
    k[4, 1, 127] = math.nan
    v[5, 0, 64] = -math.inf
    cache, batch = handles(ctx, c)
    L.lora_kv_write(ctx, cache, batch, k, v)
    ctx.sync_status()
    p, cell = c.cells(0, range(8))
    for x, pool, scale in ((k, c.k_pool, c.k_scale), (v, c.v_pool, c.v_scale)):
        code, sc = quantise(x, fmt)
        assert torch.equal(raw(pool)[p, cell], raw(code))
        assert torch.equal(torch.isnan(scale[p, cell]), torch.isnan(sc))
        assert torch.equal(torch.nan_to_num(scale[p, cell]), torch.nan_to_num(sc))
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    L.lora_kv_read(ctx, cache, batch, kb, vb)
    ctx.sync_status()
    bad = ~torch.isfinite(k).all(-1)
    assert torch.isnan(kb[bad]).all() and torch.isfinite(kb[~bad]).all()


def test_write_from_strided_rows(ctx):
    """k and v as slices of one fused projection output."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(3, [3, 1, 5], [30, 1, 17], 4, 2, 64, 16, fill=False)
    qkv = c.rand(c.n, (4 + 2 + 2) * 64)
    k, v = qkv[:, 256:384], qkv[:, 384:]
    cache, batch = handles(ctx, c)
    L.lora_kv_write(ctx, cache, batch, k, v)
    kb, vb = torch.empty((c.n, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((c.n, 128), dtype=torch.bfloat16, device="cuda")
    L.lora_kv_read(ctx, cache, batch, kb, vb)
    ctx.sync_status()
    assert torch.equal(kb.view(c.n, 128), k) and torch.equal(vb, v)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 2), (12, 4), (7, 1), (40, 2)])
@pytest.mark.parametrize("new_hi", [1, 6])
def test_few_new_tokens(ctx, fmt, dim, heads, kv_heads, new_hi):
    new, lens = random_batch(heads * 7 + new_hi, 11, new_hi, 700, released=2)
    check(ctx, Case(heads + dim, new, lens, heads, kv_heads, dim, 16, fmt))


@pytest.mark.parametrize("length", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_one_row_at_every_edge_of_a_tile(ctx, fmt, length):
    check(ctx, Case(length, [1], [length], 4, 2, 128, 16, fmt))


@pytest.mark.parametrize("page", [1, 3, 16, 100, 256])
@pytest.mark.parametrize("layout", ["split", "joint", "heads", "gaps"])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_pages_and_layouts(ctx, fmt, layout, page):
    new, lens = random_batch(page, 5, 3, 400)
    check(ctx, Case(page, new, lens, 6, 3, 64, page, fmt, layout))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,lens", [([17], [17]), ([130, 1, 64], [130, 500, 64]), ([255, 33], [700, 33]),
                                      ([128, 129, 1, 1], [128, 129, 900, 1])])
def test_chunks(ctx, fmt, dim, new, lens):
    check(ctx, Case(sum(new), new, lens, 8, 2, dim, 16, fmt))


@pytest.mark.parametrize("heads,kv_heads", [(3, 3), (5, 1), (12, 4), (48, 2)])
def test_chunks_of_shared_heads(ctx, heads, kv_heads):
    check(ctx, Case(heads, [200, 77, 1], [300, 77, 450], heads, kv_heads, 128, 32))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (5, 1), (64, 4), (100, 0), (130, 200), (10 ** 9, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 1, 2, 5], [150, 260, 1, 70]])
def test_window_and_sinks(ctx, fmt, window, sinks, new):
    lens = [max(a, b) for a, b in zip(new, [40, 777, 3, 513])]
    check(ctx, Case(window % 1000, new, lens, 4, 2, 64, 16, fmt), window=window, sinks=sinks)


def test_sinks_without_a_window_change_nothing(ctx):
    c = Case(4, [3, 60], [90, 200], 4, 2, 64, 16)
    a = attend(ctx, c).clone()
    assert torch.equal(a, attend(ctx, c, sinks=9))


def test_rows_without_a_position_and_rows_of_nobody(ctx):
    """Released slots and rows ahead of position 0 become zeros; rows past the last
    sequence are left alone; sequences without rows are fine."""
    import adapter_sgmv_bgmv_gb300 as L
    for new, lens in (([1, 0, 1, 4, 0, 2], [0, 50, 33, 2, 0, 2]), ([40, 0, 90, 1], [3, 9, 60, 0])):
        c = Case(6, new, lens, 4, 2, 64, 16)
        want, bound = c.reference()
        q = torch.cat([c.q, c.rand(3, 4, 64)])
        out = torch.full_like(q, 7.0)
        cache, batch = handles(ctx, c)
        L.lora_attention(ctx, cache, batch, q, out)
        ctx.sync_status()
        assert_attention(out[:c.n], want, bound)
        for s, (n, m) in enumerate(zip(new, lens)):
            if n > m:
                assert (out[c.start[s]:c.start[s] + n - m] == 0).all()
        assert (out[c.n:] == 7).all()


def test_no_rows_and_no_sequences(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(6, [0, 0], [5, 0], 4, 2, 64, 16)
    cache, batch = handles(ctx, c)
    empty = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    L.lora_attention(ctx, cache, batch, empty, empty)
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lora_attention(ctx, cache, batch, out.clone(), out)      # rows, but none belongs to a sequence
    nobody = L.KvBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                       torch.zeros((0, 4), dtype=torch.int32, device="cuda"))
    L.lora_attention(ctx, cache, nobody, out.clone(), out)
    ctx.sync_status()
    assert (out == 7).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("new", [[6, 1], [190, 1]])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_hidden_values_do_not_leak(ctx, fmt, new, value):
    """A value or key that is not finite reaches exactly the rows that see it: later
    tokens of the chunk, and tokens behind the window, are not in a row's sums."""
    c = Case(8, new, [250, 300], 4, 2, 64, 16, fmt)
    bad = c.rand(1, 2, 64)
    bad[0, :, 3] = value
    good = c.rand(1, 2, 64)
    c.put(0, [247], good, bad)                  # seen by the last three rows of the chunk
    c.put(0, [100], bad, bad)                   # behind the window of every row
    c.put(1, [200], good, bad)                  # behind the window
    check(ctx, c, window=40, sinks=2)


def test_an_infinite_score_is_a_nan_only_where_seen(ctx):
    c = Case(9, [5, 70], [40, 70], 2, 1, 64, 16)
    c.q[:, :, 0] = 1.0
    k = c.rand(1, 1, 64)
    k[0, 0, 0] = math.inf
    v = c.rand(1, 1, 64)
    c.put(0, [38], k, v)
    c.put(1, [30], k, v)
    out = attend(ctx, c)
    assert torch.isfinite(out[:3]).all() and torch.isnan(out[3:5]).all()
    assert torch.isfinite(out[5:35]).all() and torch.isnan(out[35:]).all()


def test_keys_of_minus_infinite_score_have_no_weight(ctx):
    c = Case(10, [1], [3], 2, 1, 64, 16)
    c.q[:, :, 0] = 1.0
    k = c.rand(1, 1, 64)
    k[0, 0, 0] = -math.inf
    v = c.rand(1, 1, 64)
    c.put(0, [1], k, v)
    want, bound = c.reference()
    assert_attention(attend(ctx, c), want, bound)
    c.put(0, [0], k, v)
    c.put(0, [2], k, v)
    assert (attend(ctx, c) == 0).all()          # no key has a weight


def test_large_scores(ctx):
    """Scores of some hundreds: the maximum is taken out before the exponential.  The
    bound's score term scales with them."""
    for new in ([2], [150]):
        c = Case(11, new, [600], 4, 4, 64, 16, gain=40.0)
        want, bound = c.reference()
        got = attend(ctx, c)
        assert_attention(got, want, bound + 2.0 ** -9 * c.get(0, 600, "v").abs().amax())


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_scale_is_the_callers(ctx, scale):
    check(ctx, Case(12, [2, 100], [80, 130], 4, 2, 64, 16), scale=scale)


def test_strided_queries_and_outputs(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    for new, lens in (([2, 1, 3], [70, 9, 200]), ([90, 130], [90, 333])):
        c = Case(13, new, lens, 4, 2, 64, 16)
        want, bound = c.reference()
        qkv = c.rand(c.n, 512)
        qkv[:, :256] = c.q.view(c.n, 256)
        out = torch.full((c.n, 320), 7.0, dtype=torch.bfloat16, device="cuda")
        cache, batch = handles(ctx, c)
        L.lora_attention(ctx, cache, batch, qkv[:, :256], out[:, 64:])
        ctx.sync_status()
        assert_attention(out[:, 64:].reshape(c.n, 4, 64), want, bound)
        assert (out[:, :64] == 7).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_one_long_sequence_is_split_and_joined_in_a_fixed_order(ctx, fmt):
    for new in (1, 20, 300):
        c = Case(14, [new], [70001], 8, 2, 128, 64, fmt)
        want, bound = c.reference()
        first = attend(ctx, c).clone()
        assert_attention(first, want, bound)
        for _ in range(3):
            assert torch.equal(first, attend(ctx, c))


def test_many_short_sequences(ctx):
    new, lens = random_batch(15, 900, 2, 90, released=300)
    check(ctx, Case(15, new, lens, 4, 2, 64, 16))


def test_offsets_beyond_32_bits(ctx):
    """Cells more than 2^32 bytes into the pools."""
    import adapter_sgmv_bgmv_gb300 as L
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB free")
    n, page, heads, dim = 70000, 16, 16, 128            # 4.6 GB a pool
    pools = [torch.zeros((n, page, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for new in ([1, 1], [80, 1]):
        c = Case(16, new, [100, 60], heads, heads, dim, page)
        far = np.array([[69999, 3, 69990, 68000, 12, 69000, 66000], [65999, 69998, 1, 67001, -1, -1, -1]], np.int32)
        for s in range(2):
            for j in range(-(-c.lens[s] // page)):
                for a, b in zip(pools, (c.k_pool, c.v_pool)):
                    a[far[s, j]] = b[int(c.table[s, j])]
        want, bound = c.reference()
        cache = L.KvCache(ctx, pools[0], pools[1])
        batch = L.KvBatch(c.starts, c.lens_t, torch.from_numpy(far).cuda())
        L.lora_attention(ctx, cache, batch, c.q, c.out)
        ctx.sync_status()
        assert_attention(c.out, want, bound)
        k, v = c.rand(c.n, heads, dim), c.rand(c.n, heads, dim)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        L.lora_kv_write(ctx, cache, batch, k, v)
        L.lora_kv_read(ctx, cache, batch, kb, vb)
        ctx.sync_status()
        assert torch.equal(k, kb) and torch.equal(v, vb)


# ---------------------------------------------------------------- device data, streams, graphs

def test_bad_device_data_is_reported_and_skipped(ctx):
    import adapter_sgmv_bgmv_gb300 as L

    def fails(c, name, max_new=None):
        cache, batch = handles(ctx, c, max_new)
        k = c.rand(c.n, c.kv_heads, c.dim)
        for call in (lambda: L.lora_attention(ctx, cache, batch, c.q, c.out),
                     lambda: L.lora_kv_read(ctx, cache, batch, k, k.clone()),
                     lambda: L.lora_kv_write(ctx, cache, batch, k, k)):
            call()
            with pytest.raises(L.LoraError) as e:
                ctx.sync_status()
            assert e.value.name == name
            ctx.sync_status()                   # reported once

    for new in ([1, 2, 1], [1, 90, 1]):
        lens = [50, 100, 70]
        c = Case(17, new, lens, 4, 2, 64, 16)
        want, bound = c.reference()
        for row, col, bad in ((1, 2, -1), (1, 6, 10 ** 6), (1, 6, -5)):
            keep = c.pages.clone()
            c.pages[row, col] = bad
            cache, batch = handles(ctx, c)
            L.lora_attention(ctx, cache, batch, c.q, c.out)
            with pytest.raises(L.LoraError) as e:
                ctx.sync_status()
            assert e.value.name == "LORA_E_PAGE"
            assert_attention(c.out[:1], want[:1], bound[:1])           # the others have their results
            assert_attention(c.out[-1:], want[-1:], bound[-1:])
            c.pages.copy_(keep)
        for what, index, bad in (("lens_t", 1, -3), ("lens_t", 1, 10 ** 6), ("starts", 1, -1), ("starts", 1, 10 ** 8),
                                 ("starts", 3, 10 ** 9)):
            keep = getattr(c, what).clone()
            getattr(c, what)[index] = bad
            fails(c, "LORA_E_INVAL")
            getattr(c, what).copy_(keep)
        fails(c, "LORA_E_INVAL", max_new=1)
        check(ctx, Case(17, new, lens, 4, 2, 64, 16))                  # and the context goes on


def test_a_captured_step_follows_the_lengths(ctx):
    """Write and attention in one CUDA graph; each replay stores a new token."""
    import adapter_sgmv_bgmv_gb300 as L
    lens = [5, 63, 127, 300]
    c = Case(18, [1] * 4, [m + 6 for m in lens], 8, 2, 128, 16, "int8")
    c.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
    cache, batch = handles(ctx, c, max_new=1)
    k, v = c.rand(4, 2, 128), c.rand(4, 2, 128)

    def step():
        L.lora_kv_write(ctx, cache, batch, k, v)
        L.lora_attention(ctx, cache, batch, c.q, c.out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in range(1, 6):
        k.copy_(c.rand(4, 2, 128))
        v.copy_(c.rand(4, 2, 128))
        c.q.copy_(c.rand(4, 8, 128))
        c.lens_t += 1
        g.replay()
        ctx.sync_status()
        c.lens = [m + t for m in lens]
        want, bound = c.reference()
        assert_attention(c.out, want, bound)


def test_another_stream(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(19, [1, 100], [500, 120], 8, 2, 128, 16)
    want, bound = c.reference()
    cache, batch = handles(ctx, c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    L.lora_attention(ctx, cache, batch, c.q, c.out, stream=s)
    ctx.sync_status(s)
    assert_attention(c.out, want, bound)


def test_calls_count_their_launches_and_name_their_path(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(20, [1, 1], [40, 50], 4, 2, 64, 16)
    cache, batch = handles(ctx, c, max_new=1)
    n = ctx.launch_count()
    k = c.rand(2, 2, 64)
    L.lora_kv_write(ctx, cache, batch, k, k)
    assert ctx.last_path() == (32, 1)
    L.lora_attention(ctx, cache, batch, c.q, c.out)
    path, launches = ctx.last_path()
    assert path & 64 and launches >= 1 and ctx.launch_count() == n + 1 + launches
    ctx.sync_status()


def test_adapters_and_cache_share_one_pool(ctx):
    """S-LoRA's unified paging: 4096-wide pages, some hold adapter vectors, others two
    tokens' keys and values each; the delta and the attention both read the pool."""
    import adapter_sgmv_bgmv_gb300 as L
    heads, dim, width = 8, 128, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randn((64, width), generator=gen, device="cuda").to(torch.bfloat16)
    ap = np.arange(0, 16, 2, dtype=np.int32)[None]
    bp = np.arange(1, 17, 2, dtype=np.int32)[None]
    table = L.AdapterTable(ctx, pool, pool, [8], [0.5], ap, bp)
    cells = pool.view(64, 2, 2, heads, dim)              # [page, token, k / v, head, d]
    k_pool, v_pool = cells[:, :, 0], cells[:, :, 1]
    c = Case(21, [1, 2], [21, 30], 8, 8, 128, 2)
    free = np.random.default_rng(2).permutation(np.arange(17, 64)).astype(np.int32)
    pages = np.full((2, 15), -1, np.int32)
    pages[0, :11], pages[1] = free[:11], free[11:26]
    for s in range(2):
        for j in range(-(-c.lens[s] // 2)):
            k_pool[int(pages[s, j])] = c.k_pool[int(c.table[s, j])]
            v_pool[int(pages[s, j])] = c.v_pool[int(c.table[s, j])]
    x = torch.randn((3, width), generator=gen, device="cuda").to(torch.bfloat16)
    y = torch.zeros((3, width), dtype=torch.bfloat16, device="cuda")
    want, bound = c.reference()
    cache = L.KvCache(ctx, k_pool, v_pool)
    batch = L.KvBatch(c.starts, c.lens_t, torch.from_numpy(pages).cuda())
    L.lora_attention(ctx, cache, batch, c.q, c.out)
    L.lora_fused(ctx, table, np.zeros(3, np.int32), x, y)
    ctx.sync_status()
    assert_attention(c.out, want, bound)
    a, b = pool[torch.from_numpy(ap[0]).long().cuda()].double(), pool[torch.from_numpy(bp[0]).long().cuda()].double()
    ref = 0.5 * (x.double() @ a.T) @ b
    assert ((y.double() - ref).norm() / ref.norm()).item() < 5e-3

"""Norms of heads and their rotation, alone and with the store into the cache, against the 64-bit model."""
import math
import random

import pytest
import torch

from tests._kv_ref import TOP, Case, raw
from tests._step_ref import rope, rope_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def freqs_of(rot, theta=1e4):
    return (theta ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float().cuda() if rot else None


def positions(case):
    return torch.cat([torch.arange(m - n, m) for n, m in zip(case.new, case.lens)]).cuda()


def make(ctx, case, rot, norm="qk", interleaved=False, theta=1e4, eps=1e-6):
    import adapter_sgmv_bgmv_gb300 as L
    w = {s: (1 + 0.3 * torch.randn(case.dim, generator=case.gen, device="cuda")) if s in norm else None for s in "qk"}
    f = freqs_of(rot, theta)
    return L.HeadRope(f, case.dim, w["q"], w["k"], eps=eps, interleaved=interleaved), w, f


def check(got, x, w, pos, f, eps, interleaved):
    y, size = rope(x, w, pos.clamp(min=0), f, eps, interleaved)
    y = torch.where((pos >= 0)[:, None, None], y, torch.zeros_like(y))
    off = (got.double() - y).abs()
    assert bool((off <= rope_bound(y, size)).all()), float((off - rope_bound(y, size)).max())


@pytest.mark.parametrize("dim,rot,interleaved", [
    (128, 128, False), (128, 128, True), (128, 64, False), (128, 32, True), (128, 0, False), (64, 64, False), (64, 16, True), (64, 48, False),
    (256, 256, False), (256, 128, True), (96, 96, False), (96, 32, True), (80, 80, False), (8, 0, False), (16, 16, False), (200, 160, False)])
@pytest.mark.parametrize("norm", ["qk", "", "k"])
def test_heads(ctx, dim, rot, interleaved, norm):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(dim + rot, [3, 1, 0, 9], [40, 1, 5, 4097], 6, 2, 64, 16, fill=False)
    c.dim = dim
    r, w, f = make(ctx, c, rot, norm, interleaved)
    q, k = c.rand(c.n, 6, dim), c.rand(c.n, 2, dim)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages)
    L.lora_head_rope(ctx, r, batch, q, k, qo, ko)
    ctx.sync_status()
    assert ctx.last_path() == (256, 1)
    check(qo, q, w["q"], positions(c), f, 1e-6, interleaved)
    check(ko, k, w["k"], positions(c), f, 1e-6, interleaved)
    # one side alone, and in place: the same bits
    q2, k2 = q.clone(), k.clone()
    L.lora_head_rope(ctx, r, batch, q2, None)
    L.lora_head_rope(ctx, r, batch, None, k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("far", [32767, 131071, (1 << 24) + 1, (1 << 30) - 1])
def test_far_positions(ctx, far):
    """fp32 angles would be off by far * 2^-24 radians here."""
    import adapter_sgmv_bgmv_gb300 as L
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    lens = torch.tensor([far + 1], dtype=torch.int32, device="cuda")
    batch = L.KvBatch(starts, lens, torch.zeros((1, 0), dtype=torch.int32, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(far)
    q = torch.randn((4, 5, 128), generator=gen, device="cuda").bfloat16()
    for theta in (1e4, 1e6):
        f = freqs_of(128, theta)
        out = torch.empty_like(q)
        L.lora_head_rope(ctx, L.HeadRope(f, 128), batch, q, None, out)
        ctx.sync_status()
        check(out, q, None, torch.arange(far - 3, far + 1, device="cuda"), f, 0.0, False)


def test_odd_frequencies(ctx):
    """Negative, zero, above a turn a token, tiny; one that is no number turns its pair alone into NaN."""
    import adapter_sgmv_bgmv_gb300 as L
    f = torch.tensor([-0.7, 0.0, 9.5, 1e-30, 700.25, -1e5, 0.1, 1.0], device="cuda")
    starts, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 50], [50]))
    batch = L.KvBatch(starts, lens, torch.zeros((1, 0), dtype=torch.int32, device="cuda"))
    q = torch.randn((50, 2, 64), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    out = torch.empty_like(q)
    L.lora_head_rope(ctx, L.HeadRope(f, 64), batch, q, None, out)
    check(out, q, None, torch.arange(50, device="cuda"), f, 0.0, False)
    for bad in (math.nan, math.inf, 2.0 ** 21):
        f[6] = bad
        L.lora_head_rope(ctx, L.HeadRope(f, 64, interleaved=True), batch, q, None, out)
        lost = torch.zeros(64, dtype=torch.bool, device="cuda")
        lost[12:14] = True
        assert torch.equal(torch.isnan(out), lost.expand_as(out))
    ctx.sync_status()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("layout", ["split", "joint", "heads", "gaps"])
@pytest.mark.parametrize("dim,rot,interleaved,norm", [(128, 128, False, "qk"), (64, 32, True, "q"), (128, 64, True, ""), (64, 64, False, "k")])
def test_store(ctx, fmt, layout, dim, rot, interleaved, norm):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(7 * dim + rot, [5, 1, 0, 33, 1], [70, 1, 9, 33, 0], 12, 3, dim, 16, fmt=fmt, layout=layout, fill=False)
    r, w, f = make(ctx, c, rot, norm, interleaved)
    qkv = c.rand(c.n, 18, dim)                             # one projection's rows
    q, k, v = qkv[:, :12], qkv[:, 12:15], qkv[:, 15:]
    cache = L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages)
    # apart: rotation, then the write
    q1, k1 = torch.full_like(q, 7).contiguous(), torch.empty((c.n, 3, dim), dtype=torch.bfloat16, device="cuda")
    L.lora_head_rope(ctx, r, batch, q, k, q1, k1)
    L.lora_kv_write(ctx, cache, batch, k1, v)
    apart = [raw(c.k_pool).clone(), raw(c.v_pool).clone()]
    raw(c.k_pool).fill_(3)
    raw(c.v_pool).fill_(3)
    blank = [raw(c.k_pool).clone(), raw(c.v_pool).clone()]
    q2 = torch.empty_like(q1)
    L.lora_kv_write_rope(ctx, cache, r, batch, q, k, v, q2)
    ctx.sync_status()
    assert ctx.last_path() == (256, 1)
    assert torch.equal(q1, q2)
    pos = positions(c)
    y, size = rope(k, w["k"], pos.clamp(min=0), f, 1e-6, interleaved)
    written = torch.zeros(c.k_pool.shape[:2], dtype=torch.bool, device="cuda")
    row = 0
    for s, (n, m) in enumerate(zip(c.new, c.lens)):
        for i in range(n):
            p = m - n + i
            if p >= 0:
                at = int(c.table[s, p // 16]), p % 16
                written[at] = True
                if fmt == "bf16":
                    assert torch.equal(raw(c.k_pool)[at], apart[0][at])
                else:
                    sc = c.k_scale[at].double()[:, None]
                    got = raw(c.k_pool)[at].view(c.k_pool.dtype).float().double() * sc
                    top = y[row].abs().amax(-1, keepdim=True)
                    assert bool(((sc * TOP[fmt] - top).abs() <= 2.0 ** -16 * size[row].amax(-1, keepdim=True)).all())
                    # half a step of the code (int8 a step is the scale, e4m3 2^-3 of the value or 2^-9 scales), and fp32 ahead of it
                    half = sc / 2 if fmt == "int8" else torch.maximum(y[row].abs() * 2.0 ** -4, sc * 2.0 ** -10)
                    assert bool(((got - y[row]).abs() <= half * (1 + 2.0 ** -10) + 2.0 ** -15 * size[row].amax(-1, keepdim=True)).all())
                assert torch.equal(raw(c.v_pool)[at], apart[1][at])
            row += 1
    for now, was in zip((raw(c.k_pool), raw(c.v_pool)), blank):
        assert torch.equal(now[~written], was[~written])
    # keys and values alone: the same codes
    after = raw(c.k_pool).clone()
    L.lora_kv_write_rope(ctx, cache, r, batch, None, k, v)
    ctx.sync_status()
    assert torch.equal(raw(c.k_pool), after)
    cache.close()


@pytest.mark.parametrize("n,heads,kv_heads", [(1, 1, 1), (1, 64, 8), (304, 8, 1), (700, 40, 10), (3000, 4, 4), (2500, 28, 4)])
def test_rows_of_every_count(ctx, n, heads, kv_heads):
    """One row a CTA, cut over several, and up to eight rows a CTA."""
    import adapter_sgmv_bgmv_gb300 as L
    rng = random.Random(n)
    new, left = [], n
    while left:
        new.append(rng.randint(1, min(left, 600)))
        left -= new[-1]
    c = Case(n, new, [m + rng.randint(0, 50) for m in new], heads, kv_heads, 128, 24, fill=False)
    r, w, f = make(ctx, c, 128)
    k, v = c.rand(n, kv_heads, 128), c.rand(n, kv_heads, 128)
    cache = L.KvCache(ctx, c.k_pool, c.v_pool)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages)
    L.lora_kv_write_rope(ctx, cache, r, batch, c.q, k, v, c.out)
    back = [torch.empty_like(k) for _ in range(2)]
    L.lora_kv_read(ctx, cache, batch, *back)
    ctx.sync_status()
    check(c.out, c.q, w["q"], positions(c), f, 1e-6, False)
    check(back[0], k, w["k"], positions(c), f, 1e-6, False)
    assert torch.equal(back[1], v)
    cache.close()


def test_rows_of_no_sequence_and_bad_pages(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    from adapter_sgmv_bgmv_gb300 import LoraError
    c = Case(5, [2, 3, 2], [20, 3, 40], 4, 2, 64, 16, fmt="int8", fill=False)
    r, _, _ = make(ctx, c, 64)
    q, k, v = c.rand(c.n + 3, 4, 64), c.rand(c.n + 3, 2, 64), c.rand(c.n + 3, 2, 64)
    out = torch.full_like(q, 7)
    cache = L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    c.pages[1, 0] = 1000
    c.lens_t[2] = 10 ** 6
    batch = L.KvBatch(c.starts, c.lens_t, c.pages)
    L.lora_kv_write_rope(ctx, cache, r, batch, q, k, v, out)
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_INVAL"
    assert bool((out[5:] == 7).all())                      # a sequence out of range, rows past the last one
    assert bool((out[:5] != 7).any(-1).all())
    c.lens_t[2] = 40
    L.lora_kv_write_rope(ctx, cache, r, batch, q, k, v, out)
    with pytest.raises(LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_PAGE"
    cache.close()


def test_values_that_are_not_finite(ctx):
    """They stay with their own head; an 8-bit vector with one reads back as NaN."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(6, [4], [4], 2, 2, 128, 16, fmt="fp8", fill=False)
    r, w, f = make(ctx, c, 64)
    q, k, v = c.rand(4, 2, 128), c.rand(4, 2, 128), c.rand(4, 2, 128)
    q[1, 0, 100], k[2, 1, 3], v[3, 0, 9] = math.inf, math.nan, -math.inf
    cache = L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages)
    L.lora_kv_write_rope(ctx, cache, r, batch, q, k, v, c.out)
    back = [torch.empty_like(k) for _ in range(2)]
    L.lora_kv_read(ctx, cache, batch, *back)
    ctx.sync_status()
    for x, bad in ((c.out, (1, 0)), (back[0], (2, 1)), (back[1], (3, 0))):
        lost = ~torch.isfinite(x).all(-1)
        want = torch.zeros_like(lost)
        want[bad] = True
        assert torch.equal(lost, want)
    cache.close()


def test_captured_and_on_a_stream(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(8, [1, 1, 1], [5, 17, 40], 8, 2, 128, 16, fill=False)
    r, w, f = make(ctx, c, 128)
    k, v = c.rand(3, 2, 128), c.rand(3, 2, 128)
    cache = L.KvCache(ctx, c.k_pool, c.v_pool)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages, max_new=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.lora_kv_write_rope(ctx, cache, r, batch, c.q, k, v, c.out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(c.out, c.q, w["q"], positions(c), f, 1e-6, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lora_kv_write_rope(ctx, cache, r, batch, c.q, k, v, c.out)
    for lens in ([1, 2, 3], [16, 0, 48]):
        c.lens_t.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ctx.sync_status()
        pos = c.lens_t.long() - 1
        check(c.out, c.q, w["q"], pos, f, 1e-6, False)
    cache.close()


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_wider_buffer(ctx, interleaved):
    """Queries and keys of one projection's rows, turned where they are: nothing else of the rows changes."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(9, [700, 1, 33], [700, 50, 40], 5, 2, 128, 16, fill=False)
    r, w, f = make(ctx, c, 64, "qk", interleaved)
    rows = c.rand(c.n, 5 + 2 + 2, 128)
    was = rows.clone()
    L.lora_head_rope(ctx, r, L.KvBatch(c.starts, c.lens_t, c.pages), rows[:, :5], rows[:, 5:7])
    ctx.sync_status()
    check(rows[:, :5], was[:, :5], w["q"], positions(c), f, 1e-6, interleaved)
    check(rows[:, 5:7], was[:, 5:7], w["k"], positions(c), f, 1e-6, interleaved)
    assert torch.equal(rows[:, 7:], was[:, 7:])


def test_calls_without_rows_or_heads(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(10, [2], [9], 2, 2, 64, 16, fill=False)
    r, _, _ = make(ctx, c, 64)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages)
    L.lora_head_rope(ctx, r, batch, c.q[:0], None)
    assert ctx.last_path() == (0, 0)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    was = c.q.clone()
    L.lora_head_rope(ctx, r, L.KvBatch(none, none[:0], torch.zeros((0, 3), dtype=torch.int32, device="cuda")), c.q, None)
    ctx.sync_status()
    assert torch.equal(c.q, was)
    for bad in (lambda: L.lora_head_rope(ctx, r, batch, None, None), lambda: L.lora_head_rope(ctx, r, batch, c.q, None, c.q[:1]),
                lambda: L.lora_head_rope(ctx, r, batch, c.q[..., :32], None), lambda: L.lora_head_rope(ctx, r, batch, c.q.float(), None),
                lambda: L.lora_kv_write_rope(ctx, L.KvCache(ctx, c.k_pool, c.v_pool), L.HeadRope(None, 128), batch, None, c.q, c.q)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        L.lora_head_rope(ctx, r, batch, c.q.cpu(), None)

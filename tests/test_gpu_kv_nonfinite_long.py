"""One value that is not finite at the start of a long context: every row that sees it is
computed on its own, over the whole context, which takes longer than the kernels' bounded
waits.  The rows get their results, and so do the other sequences of the same CTAs."""
import math

import pytest
import torch

from tests._kv_ref import Case, assert_attention, raw

pytestmark = pytest.mark.gpu

SEQS, NEW, LENGTH = 80, 200, 131003


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def spoil(c, page, fmt, value):
    """The value at the first cell of `page`, in one element of the second head."""
    c.v_pool.view(torch.int8 if fmt != "bf16" else torch.bfloat16)[page, 0, 1, 5] = 3 if fmt != "bf16" else value
    if fmt != "bf16":
        c.v_scale[page, 0, 1] = value


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_a_chunk_over_a_bad_value_beside_clean_ones(ctx, fmt):
    """160 units of 200 rows and 131,003 keys, somewhat less than one a CTA, so that a piece has
    parts of two.  All sequences share their pages but for the first one's first page."""
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(3, [NEW], [LENGTH], 2, 2, 64, 64, fmt)
    own = next(i for i in range(c.k_pool.shape[0]) if i not in set(c.table[0].tolist()))
    first = int(c.table[0, 0])
    for pool in (c.k_pool, c.v_pool):
        raw(pool)[own] = raw(pool)[first]
    if fmt != "bf16":
        c.k_scale[own], c.v_scale[own] = c.k_scale[first], c.v_scale[first]
    pages = c.pages.expand(SEQS, -1).contiguous()
    pages[0, 0] = own
    starts = (torch.arange(SEQS + 1, device="cuda") * NEW).to(torch.int32)
    lens = torch.full((SEQS,), LENGTH, dtype=torch.int32, device="cuda")
    q = c.rand(SEQS * NEW, 2, 64)
    out = torch.full_like(q, 7.0)
    cache, batch = L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale), L.KvBatch(starts, lens, pages, max_new=NEW)

    def check(s):
        c.q, c.pages = q[s * NEW:(s + 1) * NEW], pages[s:s + 1]
        want, bound = c.reference()
        assert_attention(out[s * NEW:(s + 1) * NEW], want, bound)

    L.lora_attention(ctx, cache, batch, q, out)
    ctx.sync_status()
    clean = out.clone()
    check(1)
    spoil(c, own, fmt, math.inf if fmt == "bf16" else math.nan)
    out.fill_(7.0)
    L.lora_attention(ctx, cache, batch, q, out)
    ctx.sync_status()
    # every other row is what it was, bit for bit; so is the first sequence's other head
    assert torch.equal(raw(out[NEW:]), raw(clean[NEW:])) and torch.equal(raw(out[:NEW, 0]), raw(clean[:NEW, 0]))
    check(0)


@pytest.mark.parametrize("new", [1, 3, 60])
def test_few_rows_and_a_joined_chunk_over_a_bad_value(ctx, new):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(4, [new, 2, 40], [LENGTH, 50, 300], 4, 2, 64, 64)
    spoil(c, int(c.table[0, 0]), "bf16", -math.inf)
    want, bound = c.reference()
    cache, batch = L.KvCache(ctx, c.k_pool, c.v_pool), L.KvBatch(c.starts, c.lens_t, c.pages)
    L.lora_attention(ctx, cache, batch, c.q, c.out)
    ctx.sync_status()
    assert_attention(c.out, want, bound)

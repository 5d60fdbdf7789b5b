"""The choice of pages at any magnitude: scores whose units' product lies below or above what fp32 holds."""
import math

import pytest
import torch

from tests._kv_ref import Case
from tests._step_ref import select
from tests.test_gpu_blocks import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def _chosen_as_modelled(ctx, c, how):
    st = Step(ctx, c)
    st.fill()
    sel = st.choose(*how)
    ctx.sync_status()
    lens, pages = select(c, st.codes, st.unit, *how)       # float64: no product leaves its range
    got = sel.pages[:c.n].cpu()
    st.close()
    assert torch.equal(sel.lens[:c.n].cpu(), lens) and torch.equal(got, pages)
    return got


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 2), (128, 24, 2)])
@pytest.mark.parametrize("keys,queries", [(1e-25, 1e-25), (1e-28, 1e-12), (1e-12, 1e-28), (1e-30, 1e-30), (1e-36, 1e-36), (1e20, 1e20),
                                          (1e37, 1e37), (1e37, 1e-30), (1e37, 1e-36), (1e-36, 1e37), (1.0, 1.0)])
def test_keys_and_queries_of_any_size(ctx, keys, queries, dim, heads, kv_heads):
    c = Case(int(math.log10(keys) * 100 + math.log10(queries)) % 9973, [1, 2], [900, 640], heads, kv_heads, dim, 8)
    c.k_pool.mul_(keys)
    c.q.mul_(queries)
    pages = _chosen_as_modelled(ctx, c, (11, 1, 2))
    # Something was chosen, not the first pages for want of a score.  (Units go down to 2^-106: of numbers
    # around 1e-36, none above 6e-36, the codes are at most 6e-36 * 2^106 < 1e-3, zeros by definition.)
    if min(keys, queries) > 1e-35:
        assert not torch.equal(pages[0, 0, 1:9].long(), torch.from_numpy(c.table[0, 1:9]).long())


def test_heads_and_pages_of_very_different_sizes(ctx):
    """Query heads 2^200 apart of which the large ones score 0 or less, and pages 2^200 apart: what is
    far smaller still decides where nothing larger does."""
    c = Case(21, [1], [1200], 8, 2, 64, 8)
    c.q[0, 0::4].mul_(2.0 ** 90)
    c.q[0, 0::4, :] = c.q[0, 0::4, :].abs()
    c.q[0, 1::4] = 0
    c.q[0, 2::4].mul_(2.0 ** -95)
    c.q[0, 3::4].mul_(2.0 ** -105)
    # keys: half of the pages have no component along the large heads' query but a little below zero
    k = c.k_pool
    k[:] = -k.abs()
    k[1::2].mul_(2.0 ** -100)
    k[::5] = 0
    _chosen_as_modelled(ctx, c, (9, 0, 1))
    c.q[0, 0::4] = 0
    _chosen_as_modelled(ctx, c, (9, 0, 1))


def test_scores_below_zero_and_heads_without_a_say(ctx):
    c = Case(22, [1], [1500], 6, 2, 128, 8)
    c.k_pool[:] = -c.k_pool.abs()
    c.q[:] = c.q.abs() * 2.0 ** -60
    c.k_pool.mul_(2.0 ** -60)
    c.q[0, 1, 5] = math.inf
    _chosen_as_modelled(ctx, c, (20, 1, 1))
    c.q[0, :3] = math.nan                                  # key head 0: nobody has a say, the first pages do
    pages = _chosen_as_modelled(ctx, c, (20, 1, 1))
    assert pages[0, 0, :19].tolist() == c.table[0, :19].tolist()


def test_infinite_scores_do_not_tie_with_pages_that_are_not_finite(ctx):
    c = Case(23, [1], [800], 2, 1, 64, 8)
    c.k_pool.mul_(1e37)
    c.q.mul_(1e37)
    k, v = c.rand(1, 1, 64), c.rand(1, 1, 64)
    k[0, 0, 3] = math.nan
    c.put(0, [8 * 77], k, v)
    pages = _chosen_as_modelled(ctx, c, (3, 1, 1))
    assert int(pages[0, 0, 1]) == int(c.table[0, 77])

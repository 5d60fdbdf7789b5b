"""Values that are not finite in long contexts: rows that see them get them, in time that
the kernels' bounded waits allow."""
import math

import pytest
import torch

from tests._kv_ref import Case, assert_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


def attend(ctx, c, **kw):
    import adapter_sgmv_bgmv_gb300 as L
    cache = L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    L.lora_attention(ctx, cache, L.KvBatch(c.starts, c.lens_t, c.pages), c.q, c.out, **kw)
    ctx.sync_status()
    return c.out


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("new", [1, 3, 300])
def test_a_bad_first_token_of_a_long_context(ctx, fmt, new):
    c = Case(1, [new, 2], [40000, 50], 8, 2, 128, 64, fmt)
    bad = c.rand(1, 2, 128)
    bad[0, :, 7] = math.nan
    c.put(0, [0], bad, bad)
    out = attend(ctx, c)
    assert torch.isnan(out[:new]).all() and torch.isfinite(out[new:]).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 1), (3000, 0)])
def test_an_infinite_value_in_one_element(ctx, fmt, new, window, sinks):
    """Only a value: the other elements keep their sums (bf16), or the vector is a NaN (8 bits)."""
    c = Case(2, [new], [5000], 4, 2, 64, 16, fmt)
    bad = c.rand(1, 2, 64)
    bad[0, :, 5] = math.inf
    c.put(0, [0], c.rand(1, 2, 64), bad)
    want, bound = c.reference(window=window, sinks=sinks)
    assert_attention(attend(ctx, c, window=window, sinks=sinks), want, bound)

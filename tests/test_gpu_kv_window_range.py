"""Windows and numbers of first tokens that do not fit in 32 bits: no position is that far
away, so they are as good as the largest that fits; negative ones are refused."""
import pytest
import torch

from tests._kv_ref import Case, assert_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=64)
    yield c
    c.close()


def attend(ctx, c, **kw):
    import adapter_sgmv_bgmv_gb300 as L
    L.lora_attention(ctx, L.KvCache(ctx, c.k_pool, c.v_pool), L.KvBatch(c.starts, c.lens_t, c.pages), c.q, c.out, **kw)
    ctx.sync_status()
    return c.out.clone()


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 5, 2 ** 33, 2 ** 63 - 1, 2 ** 64 + 3])
def test_large_ones_see_everything(ctx, big):
    c = Case(1, [1, 30], [70, 60], 4, 2, 64, 16)
    most = 2 ** 31 - 1
    assert torch.equal(attend(ctx, c), attend(ctx, c, window=big))
    assert torch.equal(attend(ctx, c, window=3, sinks=most), attend(ctx, c, window=3, sinks=big))
    assert_attention(c.out, *c.reference())


@pytest.mark.parametrize("small", [-1, -2 ** 31, -2 ** 32 + 5, -2 ** 32, -2 ** 63])
def test_negative_ones_are_refused(ctx, small):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(1, [1], [70], 4, 2, 64, 16)
    for kw in (dict(window=small), dict(window=3, sinks=small)):
        with pytest.raises(L.LoraError) as e:
            attend(ctx, c, **kw)
        assert e.value.name == "LORA_E_INVAL"

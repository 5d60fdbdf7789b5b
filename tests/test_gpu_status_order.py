"""A bounded wait that ran out is reported whatever bad device data was found before it, and
the context's next calls are right."""
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


def bad_page(ctx, c):
    c.pages[0, 0] = 10 ** 6


def bad_batch(ctx, c):
    c.lens_t[0] = -3


@pytest.mark.parametrize("spoil", [bad_page, bad_batch])
@pytest.mark.parametrize("timeout_first", [False, True])
def test_a_timeout_is_not_hidden_by_bad_data(ctx, spoil, timeout_first):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(1, [1, 40], [50, 90], 4, 2, 64, 16)
    want, bound = c.reference()
    cache, batch = L.KvCache(ctx, c.k_pool, c.v_pool), L.KvBatch(c.starts, c.lens_t, c.pages)
    keep = c.pages.clone(), c.lens_t.clone()
    spoil(ctx, c)
    if timeout_first:
        ctx.selftest_timeout(1000)
    L.lora_attention(ctx, cache, batch, c.q, c.out)
    if not timeout_first:
        ctx.selftest_timeout(1000)
    with pytest.raises(L.LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_TIMEOUT"
    ctx.sync_status()                                  # reported once
    c.pages.copy_(keep[0])
    c.lens_t.copy_(keep[1])
    L.lora_attention(ctx, cache, batch, c.q, c.out)
    ctx.sync_status()
    assert_attention(c.out, want, bound)


def test_bad_data_alone_keeps_its_name(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    for spoil, name in ((bad_page, "LORA_E_PAGE"), (bad_batch, "LORA_E_INVAL")):
        c = Case(2, [1, 1], [50, 90], 4, 2, 64, 16)
        spoil(ctx, c)
        L.lora_attention(ctx, L.KvCache(ctx, c.k_pool, c.v_pool), L.KvBatch(c.starts, c.lens_t, c.pages), c.q, c.out)
        with pytest.raises(L.LoraError) as e:
            ctx.sync_status()
        assert e.value.name == name
    torch.cuda.synchronize()

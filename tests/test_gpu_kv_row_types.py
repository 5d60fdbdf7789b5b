"""The rows of the cache's calls are bf16 on the context's device; anything else is refused
before a launch."""
from types import SimpleNamespace

import pytest
import torch

from tests._kv_ref import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=64)
    yield c
    c.close()


def made(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(1, [2, 1], [30, 9], 4, 2, 64, 16)
    return c, L.KvCache(ctx, c.k_pool, c.v_pool), L.KvBatch(c.starts, c.lens_t, c.pages), c.rand(c.n, 2, 64)


@pytest.mark.parametrize("dtype", [torch.float16, torch.int16, torch.uint16])
@pytest.mark.parametrize("shape", ["heads", "flat"])
def test_other_16_bit_rows_are_refused(ctx, dtype, shape):
    import adapter_sgmv_bgmv_gb300 as L
    c, cache, batch, k = made(ctx)
    before = c.k_pool.clone(), c.v_pool.clone(), c.out.clone()

    def other(t):
        t = t.view(dtype)
        return t.view(t.shape[0], -1) if shape == "flat" else t

    for call in (lambda: L.lora_kv_write(ctx, cache, batch, other(k), k), lambda: L.lora_kv_write(ctx, cache, batch, k, other(k)),
                 lambda: L.lora_kv_read(ctx, cache, batch, other(k), k.clone()),
                 lambda: L.lora_kv_read(ctx, cache, batch, k.clone(), other(k)),
                 lambda: L.lora_attention(ctx, cache, batch, other(c.q), c.out),
                 lambda: L.lora_attention(ctx, cache, batch, c.q, other(c.out))):
        with pytest.raises(ValueError, match="bf16"):
            call()
    ctx.sync_status()
    for a, b in zip(before, (c.k_pool, c.v_pool, c.out)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_tensors_of_another_device_are_refused(ctx):
    """A context or cache that says it is on the next device stands for one."""
    import adapter_sgmv_bgmv_gb300 as L
    c, cache, batch, k = made(ctx)
    with pytest.raises(ValueError, match="k_pool must be on the context's device"):
        L.KvCache(SimpleNamespace(device=torch.device("cuda", 1), handle=None), c.k_pool, c.v_pool)
    cache.device_index = batch.device_index = 1
    for what, call in (("k", lambda: L.lora_kv_write(ctx, cache, batch, k, k)), ("k", lambda: L.lora_kv_read(ctx, cache, batch, k, k.clone())),
                       ("q", lambda: L.lora_attention(ctx, cache, batch, c.q, c.out))):
        with pytest.raises(ValueError, match=f"{what} must be on the context's device"):
            call()


def test_a_batch_of_another_device_is_refused(ctx):
    import adapter_sgmv_bgmv_gb300 as L
    c, cache, batch, k = made(ctx)
    batch.device_index = 1
    for call in (lambda: L.lora_kv_write(ctx, cache, batch, k, k), lambda: L.lora_kv_read(ctx, cache, batch, k, k.clone()),
                 lambda: L.lora_attention(ctx, cache, batch, c.q, c.out)):
        with pytest.raises(ValueError, match="device"):
            call()

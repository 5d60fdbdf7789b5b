"""A context's first attention, on a stream that does not wait for the default one: what the
library zeroes when the first cache is made is zero by then."""
import pytest
import torch

from tests._kv_ref import Case, assert_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,lens", [([1], [20000]), ([200, 1], [9000, 3000])])
def test_first_attention_on_a_side_stream(new, lens):
    import adapter_sgmv_bgmv_gb300 as L
    c = Case(1, new, lens, 8, 2, 128, 16)              # units cut over several CTAs
    want, bound = c.reference()
    ctx = L.Context(0, max_rows=64)
    # memory that is not zero, handed back to the driver for the library to get
    dirty = [torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del dirty
    torch.cuda.empty_cache()
    torch.cuda._sleep(200_000_000)                     # about 0.1 s of work on the default stream
    cache, batch = L.KvCache(ctx, c.k_pool, c.v_pool), L.KvBatch(c.starts, c.lens_t, c.pages)
    side = torch.cuda.Stream()
    for _ in range(3):
        L.lora_attention(ctx, cache, batch, c.q, c.out, stream=side)
    ctx.sync_status(side)
    assert_attention(c.out, want, bound)
    torch.cuda.synchronize()
    ctx.close()

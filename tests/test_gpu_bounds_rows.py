"""lora_kv_bounds takes a number of rows and no tensor of them: the largest one it allows, over a short batch."""
import pytest
import torch

from tests._kv_ref import Case
from tests._step_ref import bounds
from tests.test_gpu_blocks import Step

pytestmark = pytest.mark.gpu


# a CTA has 17 (or 15) rows, and the last one's go past 2^31: below zero in 32 bits, where they were looked up
@pytest.mark.parametrize("page", [18, 16])
def test_the_largest_number_of_rows(page):
    import adapter_sgmv_bgmv_gb300 as L
    ctx = L.Context(0, max_rows=64)
    c = Case(page, [40], [101], 4, 2, 64, page)
    st = Step(ctx, c)
    was = st.codes.clone(), st.unit.clone()
    L.lora_kv_bounds(ctx, st.cache, st.batch, (1 << 31) - 1)
    ctx.sync_status()
    want = bounds(c, *was)
    assert torch.equal(st.codes, want[0]) and torch.equal(st.unit, want[1])
    st.close()
    ctx.close()

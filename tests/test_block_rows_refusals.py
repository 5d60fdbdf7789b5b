"""Numbers of rows of a selection's calls whose product with the heads leaves 64 bits are refused as others are."""
import ctypes

import pytest

import adapter_sgmv_bgmv_gb300 as L
from adapter_sgmv_bgmv_gb300 import _lib
from tests.test_step_refusals import A, B, CAPACITY, UNSUPPORTED, ctx, kv  # noqa: F401  (fixtures)


@pytest.mark.parametrize("n,rc", [(1 << 62, CAPACITY), ((1 << 62) + 1, CAPACITY), ((1 << 61) + 3, CAPACITY), (1 << 26, CAPACITY), ((1 << 26) - 1, UNSUPPORTED)])
def test_rows_beyond_the_limit(ctx, kv, n, rc):  # noqa: F811
    s = _lib.BlockSel(lens=4096, pages=8192, n_rows=n, blocks=6)
    assert L._L.lora_block_attention(ctx.handle, kv, ctypes.byref(s), n, A, 1024, 4, 0.1, B, 1024, None) == rc

"""Angles of far positions, for frequencies of either sign: the last positions of the range, against
angles in 64-bit fixed point."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _pi(bits):
    """pi in units of 2^-bits: 16 atan(1/5) - 4 atan(1/239) (Machin)."""
    def atan(x):
        t = (1 << bits + 16) // x
        total, k = t, 1
        while t:
            t //= x * x
            k += 2
            total += -(t // k) if k % 4 == 3 else t // k
        return total
    return 16 * atan(5) - 4 * atan(239) >> 16


def _turns(freqs, pos):
    """pos * f / 2 pi modulo 1, float64 [positions, freqs]: the fraction of a turn a token is rounded to 2^-64,
    which 2^30 positions make 2^-35."""
    per = Fraction(1 << 200, 2 * _pi(200))
    f = [round(Fraction(float(v)) * per * (1 << 64)) % (1 << 64) for v in freqs]
    return (pos[:, None] * np.array(f, np.uint64)).astype(np.float64) * 2.0 ** -64


@pytest.mark.parametrize("sign", [1, -1])
def test_the_last_positions(sign):
    """Rows (1, 0) become (cos t, sin t).  Near their zeros these show t's own error: at most 2^-34 turns of
    the product, 2^-33 of its 32 bits and 2^-26 of the fp32 number, and the model's 2^-35 and 2^-53:
    below 2^-25.9 turns.  Apart from that the cosine's own error (4 steps of fp32 are counted, 2^-22) and half
    a step of bf16, at most 2^-8 of the value."""
    import adapter_sgmv_bgmv_gb300 as L
    ctx = L.Context(0, max_rows=64)
    n, end = 1 << 19, 1 << 30
    freqs = sign * torch.tensor([0.01, 0.031622775, 1.7782794e-4, 3.1622778e-5, 5.6234132e-3, 3.1622776e-4, 0.7, 1.0])
    batch = L.KvBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([end], dtype=torch.int32, device="cuda"),
                      torch.zeros((1, 0), dtype=torch.int32, device="cuda"))
    x = torch.zeros((n, 1, 16), dtype=torch.bfloat16, device="cuda")
    x[..., :8] = 1
    L.lora_head_rope(ctx, L.HeadRope(freqs.cuda(), 16), batch, x, None)
    ctx.sync_status()
    got = x[:, 0].double().cpu().numpy()
    t = _turns(freqs.tolist(), np.arange(end - n, end, dtype=np.uint64))
    for have, want in ((got[:, :8], np.cos(2 * np.pi * t)), (got[:, 8:], np.sin(2 * np.pi * t))):
        off = np.abs(have - want) - (2.0 ** -8 * 1.001 + 2.0 ** -22) * np.abs(want)
        assert off.max() <= 2 * np.pi * 2.0 ** -25.9, np.log2(off.max() / (2 * np.pi))
    ctx.close()

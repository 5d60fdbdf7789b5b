"""examples/serving_step.py against the whole block in 64 bits: prompts by chunks, then
tokens one by one, requests on different adapters, one of them on none."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("serving_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _project(x, w, table, k):
    y = x @ w.double()
    if k >= 0:
        a = table.a_pool[torch.from_numpy(table.a_pages[k]).long().cuda()].double()
        b = table.b_pool[torch.from_numpy(table.b_pages[k]).long().cuda()].double()
        y = y + float(table.scale[k]) * (x @ a.T) @ b
    return y


def _whole(block, x, k, window, sinks):
    """The block over one request's tokens at once, in 64 bits."""
    q, kv, d = block.heads, block.kv_heads, block.dim
    h = _project(x.double(), block.w_qkv, block.qkv_adapters, k)
    n = x.shape[0]
    qs, ks, vs = h[:, :q * d].view(n, q, d), h[:, q * d:(q + kv) * d].view(n, kv, d), h[:, (q + kv) * d:].view(n, kv, d)
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
    seen = j <= i
    if window:
        seen &= (j > i - window) | (j < sinks)
    o = torch.empty((n, q, d), dtype=torch.float64, device="cuda")
    for a in range(q):
        z = (qs[:, a] @ ks[:, a // (q // kv)].T / math.sqrt(d)).masked_fill(~seen, -math.inf)
        o[:, a] = torch.softmax(z, -1) @ vs[:, a // (q // kv)]
    return _project(o.reshape(n, q * d), block.w_o, block.o_adapters, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_chunks_then_tokens_are_the_whole_block(dtype, window, sinks):
    import adapter_sgmv_bgmv_gb300 as L
    ex = _example()
    ctx = L.Context(0, max_rows=1024)
    block = ex.random_block(ctx, cache_dtype=dtype)
    total, adapters = [150, 33, 70, 6], np.array([2, 0, -1, 1], np.int32)
    req = ex.Requests(4, 64, 16, 160)
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn((n, 512), generator=gen, device="cuda").to(torch.bfloat16) for n in total]
    done, got = [0] * 4, [[] for _ in total]
    steps = [[64, 20, 64, 1], [80, 7, 0, 1]] + [[1, 1, 1, 1]] * 4 + [[1, 1, 1, 0], [1, 1, 1, 0]]
    for new in steps:
        x = torch.cat([xs[s][done[s]:done[s] + k] for s, k in enumerate(new)])
        y = block(x, np.repeat(adapters, new), req.grow(new), window, sinks)
        at = 0
        for s, k in enumerate(new):
            got[s].append(y[at:at + k])
            at += k
            done[s] += k
    ctx.sync_status()
    assert done == [150, 33, 70, 6]
    # four roundings to bf16 of at most 2^-8 each (qkv, weights, o, y); int8 keys and values
    # add a step of max / 127, a hundredth of a vector's size, each
    bound = 2e-2 if dtype == torch.bfloat16 else 4e-2
    for s in range(4):
        want = _whole(block, xs[s], int(adapters[s]), window, sinks)
        have = torch.cat(got[s]).double()
        assert ((have - want).norm() / want.norm()).item() < bound

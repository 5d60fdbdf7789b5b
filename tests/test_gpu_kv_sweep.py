"""Seeded sweep over the cache's shapes: heads, dims, pages, layouts, formats, lengths, new
tokens, windows and released slots drawn at random; each step writes its new tokens and
attends, against the 64-bit model."""
import random

import pytest
import torch

from tests._kv_ref import Case, assert_attention

pytestmark = pytest.mark.gpu


def draw(seed):
    rng = random.Random(seed)
    kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    seqs = rng.choice([1, 2, 5, 17])
    hi = rng.choice([1, 1, 3, 9, 40, 170, 300])
    longest = rng.choice([20, 130, 700, 2500])
    new = [rng.randint(0 if seqs > 1 else 1, hi) for _ in range(seqs)]
    lens = [max(n, rng.randint(1, longest)) for n in new]
    for s in rng.sample(range(seqs), rng.choice([0, 0, seqs // 3])):
        lens[s], new[s] = 0, 1
    if sum(new) == 0:
        new[0] = 1
    window = rng.choice([0, 0, rng.randint(1, 400)])
    return dict(new=new, lens=lens, heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]),
                page=rng.choice([1, 5, 16, 24, 64, 128]), fmt=rng.choice(["bf16", "int8", "fp8"]),
                layout=rng.choice(["split", "joint", "heads", "gaps"])), dict(window=window, sinks=rng.choice([0, 1, 6, 200]))


@pytest.fixture(scope="module")
def ctx():
    import adapter_sgmv_bgmv_gb300 as L
    c = L.Context(0, max_rows=1024)
    yield c
    c.close()


@pytest.mark.parametrize("seed", range(60))
def test_random_steps(ctx, seed):
    import adapter_sgmv_bgmv_gb300 as L
    shape, how = draw(1000 + seed)
    c = Case(seed, **shape)
    cache = L.KvCache(ctx, c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    batch = L.KvBatch(c.starts, c.lens_t, c.pages, max_new=random.Random(seed).choice([None, max(c.new)]))
    k, v = c.rand(c.n, c.kv_heads, c.dim), c.rand(c.n, c.kv_heads, c.dim)
    L.lora_kv_write(ctx, cache, batch, k, v)
    L.lora_attention(ctx, cache, batch, c.q, c.out, **how)
    ctx.sync_status()
    got = c.out.clone()
    # the model's own stores of the same tokens, over what the write left
    for s in range(len(c.lens)):
        n = min(c.new[s], c.lens[s])
        if n:
            rows = slice(int(c.start[s + 1]) - n, int(c.start[s + 1]))
            c.put(s, range(c.lens[s] - n, c.lens[s]), k[rows], v[rows])
    want, bound = c.reference(**how)
    assert_attention(got, want, bound)

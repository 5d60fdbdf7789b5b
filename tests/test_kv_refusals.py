"""What the cache's entry points refuse, without a GPU: the checks run on the host ahead of
any launch, so a host-only context sees all of them."""
import ctypes

import pytest
import torch

import adapter_sgmv_bgmv_gb300 as L
from adapter_sgmv_bgmv_gb300 import _lib

INVAL, CAPACITY, UNSUPPORTED = -1, -9, -10


@pytest.fixture()
def ctx():
    c = L.Context(-1, max_rows=64)
    yield c
    c.close()


def desc(**over):
    d = dict(k_pool=1 << 20, v_pool=1 << 21, k_scale=0, v_scale=0, n_pages=8, page_size=16, n_heads=4,
             head_dim=128, format=0, page_stride=8192, cell_stride=512, head_stride=128,
             scale_page_stride=64, scale_cell_stride=4, scale_head_stride=1)
    d.update(over)
    return _lib.KvDesc(**d)


def create(ctx, **over):
    h = ctypes.c_void_p()
    rc = L._L.lora_kv_create(ctx.handle, ctypes.byref(desc(**over)), ctypes.byref(h))
    if rc == 0:
        L._L.lora_kv_destroy(h)
    return rc


@pytest.mark.parametrize("over", [
    dict(k_pool=0), dict(v_pool=0), dict(k_pool=(1 << 20) + 8), dict(n_pages=0), dict(page_size=0), dict(n_heads=0),
    dict(n_pages=-1), dict(format=3), dict(format=-1), dict(page_stride=4), dict(page_stride=8193), dict(cell_stride=-512),
    dict(head_stride=127), dict(head_stride=132), dict(format=1), dict(format=2, k_scale=4096),
    dict(format=1, k_scale=4098, v_scale=4096), dict(format=1, k_scale=4096, v_scale=4096, scale_cell_stride=0),
    dict(format=1, k_scale=4096, v_scale=4096, head_stride=136)])
def test_descriptions_that_are_refused(ctx, over):
    assert create(ctx, **over) == INVAL


@pytest.mark.parametrize("over,rc", [
    ({}, 0), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(n_pages=1 << 31), CAPACITY),
    (dict(page_size=1 << 21), CAPACITY), (dict(n_heads=1, head_stride=0), 0), (dict(n_pages=1, page_stride=0), 0),
    (dict(page_size=1, cell_stride=3), 0), (dict(format=2, k_scale=4096, v_scale=4096), 0)])
def test_other_descriptions(ctx, over, rc):
    assert create(ctx, **over) == rc


def test_null_arguments(ctx):
    h = ctypes.c_void_p()
    d = desc()
    assert L._L.lora_kv_create(None, ctypes.byref(d), ctypes.byref(h)) == INVAL
    assert L._L.lora_kv_create(ctx.handle, None, ctypes.byref(h)) == INVAL
    assert L._L.lora_kv_create(ctx.handle, ctypes.byref(d), None) == INVAL
    assert L._L.lora_kv_destroy(None) == INVAL


@pytest.fixture()
def kv(ctx):
    h = ctypes.c_void_p()
    d = desc()
    assert L._L.lora_kv_create(ctx.handle, ctypes.byref(d), ctypes.byref(h)) == 0
    yield h
    L._L.lora_kv_destroy(h)


def batch(**over):
    b = dict(starts=4096, lens=8192, pages=12288, n_seqs=3, n_cols=5, ld_pages=5, max_new=4)
    b.update(over)
    return _lib.KvBatchArgs(**b)


BAD_BATCHES = [(dict(starts=0), INVAL), (dict(lens=0), INVAL), (dict(pages=0), INVAL), (dict(starts=4097), INVAL),
               (dict(n_seqs=-1), INVAL), (dict(n_cols=-1), INVAL), (dict(ld_pages=4), INVAL), (dict(max_new=-1), INVAL),
               (dict(n_seqs=1 << 31), CAPACITY)]


@pytest.mark.parametrize("over,rc", BAD_BATCHES)
def test_batches_that_are_refused(ctx, kv, over, rc):
    b = ctypes.byref(batch(**over))
    big = 1 << 22
    assert L._L.lora_kv_write(ctx.handle, kv, b, 3, big, 512, big, 512, None) == rc
    assert L._L.lora_kv_read(ctx.handle, kv, b, 3, big, 512, big, 512, None) == rc
    assert L._L.lora_attention(ctx.handle, kv, b, 3, big, 1024, 8, 0.1, 0, 0, big, 1024, None) == rc


@pytest.mark.parametrize("k,ldk,v,ldv,n,rc", [
    (0, 512, 1 << 22, 512, 3, INVAL), (1 << 22, 512, 0, 512, 3, INVAL), (1 << 22, 511, 1 << 22, 512, 3, INVAL),
    (1 << 22, 516, 1 << 22, 512, 3, INVAL), ((1 << 22) + 2, 512, 1 << 22, 512, 3, INVAL), (1 << 22, 512, 1 << 22, 504, 3, INVAL),
    (1 << 22, 512, 1 << 22, 512, -1, INVAL), (1 << 22, 512, 1 << 22, 512, 1 << 31, CAPACITY),
    (1 << 22, 512, 1 << 22, 512, 3, UNSUPPORTED)])       # nothing wrong: a host-only context launches nothing
def test_rows_that_are_refused(ctx, kv, k, ldk, v, ldv, n, rc):
    b = ctypes.byref(batch())
    assert L._L.lora_kv_write(ctx.handle, kv, b, n, k, ldk, v, ldv, None) == rc
    assert L._L.lora_kv_read(ctx.handle, kv, b, n, k, ldk, v, ldv, None) == rc


@pytest.mark.parametrize("over,rc", [
    (dict(q=0), INVAL), (dict(out=0), INVAL), (dict(ldq=1023), INVAL), (dict(ldo=1016), INVAL), (dict(heads=0), INVAL),
    (dict(heads=6), INVAL), (dict(heads=-4), INVAL), (dict(window=-1), INVAL), (dict(sinks=-1), INVAL),
    (dict(scale=float("nan")), INVAL), (dict(scale=float("inf")), INVAL), (dict(n=1 << 28, heads=8), CAPACITY), ({}, UNSUPPORTED)])
def test_attention_arguments_that_are_refused(ctx, kv, over, rc):
    a = dict(q=1 << 22, ldq=1024, heads=8, scale=0.1, window=0, sinks=0, out=1 << 23, ldo=1024, n=3)
    a.update(over)
    got = L._L.lora_attention(ctx.handle, kv, ctypes.byref(batch()), a["n"], a["q"], a["ldq"], a["heads"], a["scale"],
                              a["window"], a["sinks"], a["out"], a["ldo"], None)
    assert got == rc


def test_a_cache_belongs_to_its_context(ctx, kv):
    other = L.Context(-1, max_rows=64)
    b = ctypes.byref(batch())
    assert L._L.lora_kv_write(other.handle, kv, b, 3, 1 << 22, 512, 1 << 22, 512, None) == INVAL
    assert L._L.lora_attention(other.handle, kv, b, 3, 1 << 22, 1024, 8, 0.1, 0, 0, 1 << 23, 1024, None) == INVAL
    assert L._L.lora_attention(ctx.handle, kv, None, 3, 1 << 22, 1024, 8, 0.1, 0, 0, 1 << 23, 1024, None) == INVAL
    other.close()


def test_the_binding_checks_shapes_and_types(ctx):
    pool = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    scale = torch.ones((4, 16, 2))
    code = torch.zeros((4, 16, 2, 64), dtype=torch.int8)
    L.KvCache(ctx, pool, pool).close()
    L.KvCache(ctx, code, code, scale, scale).close()
    for bad in (lambda: L.KvCache(ctx, pool[0], pool[0]), lambda: L.KvCache(ctx, pool.float(), pool.float()),
                lambda: L.KvCache(ctx, pool, code), lambda: L.KvCache(ctx, code, code),
                lambda: L.KvCache(ctx, code, code, scale, scale.double()), lambda: L.KvCache(ctx, pool, pool, scale, scale),
                lambda: L.KvCache(ctx, pool, torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16).transpose(1, 2)),
                lambda: L.KvCache(ctx, pool.transpose(2, 3), pool.transpose(2, 3))):
        with pytest.raises(ValueError):
            bad()
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.KvBatch(i, i, torch.zeros((3, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        L.KvBatch(i.long(), i[:2], torch.zeros((2, 2), dtype=torch.int32))
    with pytest.raises(TypeError):
        L.KvBatch(i, i[:2], torch.zeros((2, 2), dtype=torch.int32))      # not device memory

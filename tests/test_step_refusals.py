"""What the entry points around the cache refuse, without a GPU: the checks run on the host ahead
of any launch, so a host-only context sees all of them."""
import ctypes

import pytest
import torch

import adapter_sgmv_bgmv_gb300 as L
from adapter_sgmv_bgmv_gb300 import _lib

INVAL, CAPACITY, UNSUPPORTED = -1, -9, -10
A, B = 1 << 22, 1 << 24          # addresses that nothing looks at


@pytest.fixture()
def ctx():
    c = L.Context(-1, max_rows=64)
    yield c
    c.close()


def make_kv(ctx, **over):
    d = dict(k_pool=1 << 20, v_pool=1 << 21, k_scale=0, v_scale=0, n_pages=8, page_size=16, n_heads=4,
             head_dim=128, format=0, page_stride=8192, cell_stride=512, head_stride=128,
             scale_page_stride=64, scale_cell_stride=4, scale_head_stride=1)
    d.update(over)
    h, desc = ctypes.c_void_p(), _lib.KvDesc(**d)
    assert L._L.lora_kv_create(ctx.handle, ctypes.byref(desc), ctypes.byref(h)) == 0
    return h


@pytest.fixture()
def kv(ctx):
    h = make_kv(ctx)
    yield h
    L._L.lora_kv_destroy(h)


def batch(**over):
    return _lib.KvBatchArgs(**{**dict(starts=4096, lens=8192, pages=12288, n_seqs=3, n_cols=5, ld_pages=5, max_new=4), **over})


def rope(**over):
    return _lib.Rope(**{**dict(q_weight=4096, k_weight=4096, freqs=4096, eps=1e-6, head_dim=128, rot_dim=128, interleaved=0), **over})


BAD_ROPES = [(dict(head_dim=0), INVAL), (dict(rot_dim=-16), INVAL), (dict(rot_dim=144), INVAL), (dict(eps=-1.0), INVAL),
             (dict(eps=float("nan")), INVAL), (dict(eps=float("inf")), INVAL), (dict(q_weight=4100), INVAL), (dict(k_weight=4104), INVAL),
             (dict(freqs=0), INVAL), (dict(freqs=4098), INVAL), (dict(rot_dim=24), UNSUPPORTED), (dict(rot_dim=2), UNSUPPORTED)]


@pytest.mark.parametrize("over,rc", BAD_ROPES + [(dict(head_dim=100, rot_dim=96), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED)])
def test_rotations_that_are_refused(ctx, kv, over, rc):
    r, b = rope(**over), batch()
    if "head_dim" not in over:
        assert L._L.lora_kv_write_rope(ctx.handle, kv, ctypes.byref(r), ctypes.byref(b), 3, A, 1024, 8, A, 1024, A, 512, A, 512, None) == rc
    assert L._L.lora_head_rope(ctx.handle, ctypes.byref(r), ctypes.byref(b), 3, A, 4096, 8, A, 4096, A, 4096, 4, A, 4096, None) == rc


@pytest.mark.parametrize("over,rc", [
    (dict(q=0), INVAL), (dict(q_out=0), INVAL), (dict(ldq=1016), INVAL), (dict(ldqo=1020), INVAL), (dict(k=A + 8), INVAL),
    (dict(v=0), INVAL), (dict(ldk=508), INVAL), (dict(heads=-1), INVAL), (dict(n=-1), INVAL), (dict(n=1 << 31), CAPACITY),
    (dict(heads=20000, ldq=1 << 22, ldqo=1 << 22), CAPACITY), (dict(heads=0, q=0, q_out=0), UNSUPPORTED), ({}, UNSUPPORTED)])
def test_rows_of_the_rotation_that_are_refused(ctx, kv, over, rc):
    a = dict(q=A, ldq=1024, heads=8, q_out=B, ldqo=1024, k=A, ldk=512, v=A, ldv=512, n=3)
    a.update(over)
    r, b = rope(), batch()
    head = [ctx.handle, kv, ctypes.byref(r), ctypes.byref(b), a["n"], a["q"], a["ldq"], a["heads"], a["q_out"], a["ldqo"]]
    assert L._L.lora_kv_write_rope(*head, a["k"], a["ldk"], a["v"], a["ldv"], None) == rc
    if "v" in over:
        return
    head.pop(1)
    assert L._L.lora_head_rope(*head, a["k"], a["ldk"], 4, B, 512, None) == rc


def test_the_rotation_needs_its_cache_and_head_dim(ctx, kv):
    r, b = rope(head_dim=64, rot_dim=64), batch()
    tail = [ctypes.byref(r), ctypes.byref(b), 3, A, 1024, 8, A, 1024, A, 512, A, 512, None]
    assert L._L.lora_kv_write_rope(ctx.handle, kv, *tail) == INVAL
    assert L._L.lora_kv_write_rope(ctx.handle, None, *tail) == INVAL
    other = L.Context(-1, max_rows=64)
    tail[0] = ctypes.byref(rope())
    assert L._L.lora_kv_write_rope(other.handle, kv, *tail) == INVAL
    other.close()
    # without a cache nothing looks at the pages
    assert L._L.lora_head_rope(ctx.handle, ctypes.byref(rope()), ctypes.byref(batch(pages=0, n_cols=0)), 3, A, 1024, 8, A, 1024, None, 0, 0,
                               None, 0, None) == UNSUPPORTED


def table(**over):
    return _lib.PageTableArgs(**{**dict(lens=4096, pages=8192, refs=12288, n_seqs=3, n_cols=5, ld_pages=5, n_pages=64, page_size=16), **over})


BAD_TABLES = [(dict(lens=0), INVAL), (dict(pages=0), INVAL), (dict(refs=0), INVAL), (dict(refs=4098), INVAL), (dict(n_seqs=-1), INVAL),
              (dict(n_cols=-1), INVAL), (dict(ld_pages=4), INVAL), (dict(n_pages=0), INVAL), (dict(page_size=0), INVAL),
              (dict(n_seqs=16385), CAPACITY), (dict(n_pages=(1 << 30) + 1), CAPACITY), (dict(page_size=1 << 21), CAPACITY),
              ({}, UNSUPPORTED)]


@pytest.mark.parametrize("over,rc", BAD_TABLES)
def test_tables_that_are_refused(ctx, over, rc):
    t = ctypes.byref(table(**over))
    assert L._L.lora_pages_extend(ctx.handle, t, A, A, A, A, A, None) == rc
    assert L._L.lora_pages_fork(ctx.handle, t, A, A, 2, None) == rc
    assert L._L.lora_pages_free(ctx.handle, t, A, None, 2, None) == rc
    assert L._L.lora_pages_compact(ctx.handle, t, A, A, 8, None, None) == rc


@pytest.mark.parametrize("n,rc", [(-1, INVAL), (16385, CAPACITY), (0, UNSUPPORTED)])
def test_lists_that_are_refused(ctx, n, rc):
    t = ctypes.byref(table())
    assert L._L.lora_pages_fork(ctx.handle, t, A, A, n, None) == rc
    assert L._L.lora_pages_free(ctx.handle, t, A, A, n, None) == rc


def test_arrays_of_the_table_calls(ctx):
    t = ctypes.byref(table())
    for i in range(5):
        a = [A] * 5
        a[i] = A + 2 if i % 2 else 0
        assert L._L.lora_pages_extend(ctx.handle, t, *a, None) == INVAL
    assert L._L.lora_pages_fork(ctx.handle, t, 0, A, 1, None) == INVAL
    assert L._L.lora_pages_fork(ctx.handle, t, A, A + 1, 1, None) == INVAL
    assert L._L.lora_pages_free(ctx.handle, t, A, A + 1, 1, None) == INVAL
    assert L._L.lora_pages_compact(ctx.handle, t, 0, A, 8, None, None) == INVAL
    assert L._L.lora_pages_compact(ctx.handle, t, A, A, -1, None, None) == INVAL
    assert L._L.lora_pages_compact(ctx.handle, t, A, A, 8, A + 1, None) == INVAL
    assert L._L.lora_pages_compact(ctx.handle, t, A, A, (1 << 30) + 1, None, None) == CAPACITY
    assert L._L.lora_pages_extend(None, t, A, A, A, A, A, None) == INVAL
    assert L._L.lora_pages_extend(ctx.handle, None, A, A, A, A, A, None) == INVAL


def test_copies_that_are_refused(ctx, kv):
    def call(kvs, n_kv=None, src=A, dst=A, cells=None, n=3):
        arr = (ctypes.c_void_p * len(kvs))(*[k.value if k else None for k in kvs])
        return L._L.lora_kv_copy(ctx.handle, arr, len(kvs) if n_kv is None else n_kv, src, dst, cells, n, None)
    assert call([kv]) == UNSUPPORTED
    assert call([kv], n_kv=0) == INVAL and call([kv], n=-1) == INVAL and call([kv], src=0) == INVAL
    assert call([kv], dst=A + 2) == INVAL and call([kv], cells=A + 2) == INVAL and call([kv, None]) == INVAL
    assert call([kv], n=(1 << 30) + 1) == CAPACITY
    assert L._L.lora_kv_copy(ctx.handle, None, 1, A, A, None, 1, None) == INVAL
    for over in (dict(page_size=8), dict(n_heads=2), dict(head_dim=64), dict(format=1, k_scale=4096, v_scale=4096)):
        other = make_kv(ctx, **over)
        assert call([kv, other]) == INVAL
        L._L.lora_kv_destroy(other)
    big = make_kv(ctx, page_size=1 << 20, n_heads=32, cell_stride=4096, page_stride=1 << 32)
    assert call([big]) == CAPACITY
    L._L.lora_kv_destroy(big)
    far = L.Context(-1, max_rows=64)
    other = make_kv(far)
    assert call([other]) == INVAL
    L._L.lora_kv_destroy(other)
    far.close()


def sel(**over):
    return _lib.BlockSel(**{**dict(lens=4096, pages=8192, n_rows=3, blocks=6), **over})


@pytest.mark.parametrize("over,how,rc", [
    (dict(lens=0), {}, INVAL), (dict(pages=0), {}, INVAL), (dict(pages=8194), {}, INVAL), (dict(n_rows=2), {}, INVAL),
    (dict(blocks=0), {}, INVAL), (dict(blocks=1 << 27), {}, CAPACITY), ({}, dict(heads=6), INVAL), ({}, dict(heads=0), INVAL),
    ({}, dict(q=0), INVAL), ({}, dict(ldq=1000), INVAL), ({}, dict(n=-1), INVAL), (dict(n_rows=1 << 30), dict(n=1 << 27), CAPACITY),
    ({}, {}, UNSUPPORTED)])
def test_selections_that_are_refused(ctx, kv, over, how, rc):
    a = dict(n=3, q=A, ldq=1024, heads=8)
    a.update(how)
    s, b = ctypes.byref(sel(**over)), ctypes.byref(batch())
    assert L._L.lora_kv_attach_bounds(kv, 1 << 22, 1 << 23) == 0
    assert L._L.lora_block_select(ctx.handle, kv, b, a["n"], a["q"], a["ldq"], a["heads"], 1, 1, s, None) == rc
    assert L._L.lora_block_attention(ctx.handle, kv, s, a["n"], a["q"], a["ldq"], a["heads"], 0.1, B, 1024, None) == rc


def test_bounds_and_choice(ctx, kv):
    b, s = ctypes.byref(batch()), ctypes.byref(sel())

    def choose(first=1, last=1, batch=b, heads=8, ldq=1024):
        return L._L.lora_block_select(ctx.handle, kv, batch, 3, A, ldq, heads, first, last, s, None)
    assert L._L.lora_kv_bounds(ctx.handle, kv, b, 3, None) == INVAL and choose() == INVAL        # none attached
    assert L._L.lora_kv_attach_bounds(kv, 1 << 22, None) == INVAL and L._L.lora_kv_attach_bounds(kv, None, 1 << 22) == INVAL
    assert L._L.lora_kv_attach_bounds(kv, (1 << 22) + 16, 1 << 22) == INVAL and L._L.lora_kv_attach_bounds(kv, 1 << 22, 2) == INVAL
    assert L._L.lora_kv_attach_bounds(None, 1 << 22, 1 << 22) == INVAL
    assert L._L.lora_kv_attach_bounds(kv, 1 << 22, 1 << 23) == 0
    assert L._L.lora_kv_bounds(ctx.handle, kv, b, 3, None) == UNSUPPORTED
    assert L._L.lora_kv_bounds(ctx.handle, kv, None, 3, None) == INVAL and L._L.lora_kv_bounds(ctx.handle, kv, b, -1, None) == INVAL
    assert L._L.lora_kv_bounds(None, kv, b, 3, None) == INVAL
    assert choose(first=-1) == INVAL and choose(last=0) == INVAL and choose(first=4, last=3) == INVAL and choose(first=6) == INVAL
    assert choose(first=5) == UNSUPPORTED and choose(first=3, last=3) == UNSUPPORTED
    assert choose(first=(1 << 31) - 1, last=(1 << 31) - 1) == INVAL
    assert choose(batch=ctypes.byref(batch(n_cols=45057, ld_pages=1 << 19))) == CAPACITY
    assert choose(heads=4 * 129, ldq=4 * 129 * 128) == CAPACITY
    assert L._L.lora_kv_attach_bounds(kv, None, None) == 0
    assert choose() == INVAL
    for scale in (float("nan"), float("inf")):
        assert L._L.lora_block_attention(ctx.handle, kv, s, 3, A, 1024, 8, scale, B, 1024, None) == INVAL


def test_the_binding_checks_shapes_and_types(ctx):
    f = torch.ones(64)
    with pytest.raises(TypeError):
        L.HeadRope(f, 128)                                            # not device memory
    for bad in (dict(freqs=f.double(), head_dim=128), dict(freqs=f[None], head_dim=128), dict(freqs=None, head_dim=128, q_weight=f),
                dict(freqs=None, head_dim=128, k_weight=f.int())):
        with pytest.raises(ValueError):
            L.HeadRope(**bad)
    i = torch.zeros(3, dtype=torch.int32)
    for bad in ((i, i, i, 16), (i, torch.zeros((2, 4), dtype=torch.int32), i, 16), (i.long(), torch.zeros((3, 4), dtype=torch.int32), i, 16),
                (i, torch.zeros((4, 3), dtype=torch.int32).T[:3], i, 16)):
        with pytest.raises(ValueError):
            L.PageTable(*bad)
    with pytest.raises(TypeError):
        L.PageTable(i, torch.zeros((3, 4), dtype=torch.int32), i, 16)
    for bad in ((i, torch.zeros((3, 4), dtype=torch.int32)), (i, torch.zeros((2, 4, 4), dtype=torch.int32)),
                (i, torch.zeros((3, 4, 4), dtype=torch.int64)), (i, torch.zeros((3, 4, 8), dtype=torch.int32)[..., ::2])):
        with pytest.raises(ValueError):
            L.BlockSelection(*bad)
    with pytest.raises(TypeError):
        L.BlockSelection(i, torch.zeros((3, 4, 4), dtype=torch.int32))
    pool = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    cache = L.KvCache(ctx, pool, pool)
    codes, unit = torch.zeros((4, 2, 2, 64), dtype=torch.int8), torch.zeros((4, 2))
    cache.attach_bounds(codes, unit)
    for bad in ((codes, None), (None, unit), (codes.float(), unit), (codes[:2], unit), (codes, unit.double()), (codes, unit.T.contiguous())):
        with pytest.raises(ValueError):
            cache.attach_bounds(*bad)
    cache.attach_bounds(None, None)
    cache.close()

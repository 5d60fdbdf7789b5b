"""GB300 (sm_103a) heterogeneous multi-LoRA delta: y_i += s_k (x_i A_k) B_k over a
batch whose rows are grouped by adapter id, with paged adapter storage, released
rows skipped, and an in-place merge / unmerge of W +/- s A B.

Every step runs in the CUDA kernels of ``liblora.so`` behind the C ABI declared in
``include/lora.h``; this module only marshals torch tensors (device memory and
streams) and numpy id arrays into those calls, under the same names.  Importing it
without the built library raises: there is no other implementation.
"""
from __future__ import annotations

import ctypes
import weakref

import numpy as np
import torch

from . import _lib

__all__ = ["LoraError", "Context", "AdapterTable", "lora_plan_build", "lora_shrink",
           "lora_expand", "lora_fused", "lora_fused_noalloc", "lora_base_fused", "PreparedFused", "PreparedFusedDeviceIds", "lora_merge", "lora_unmerge", "lora_page_in", "lora_fused_device_ids", "lora_tune_shape",
           "KvCache", "KvBatch", "lora_kv_write", "lora_kv_read", "lora_attention",
           "HeadRope", "lora_head_rope", "lora_kv_write_rope",
           "PageTable", "PAGE_PINNED", "lora_pages_extend", "lora_pages_fork", "lora_pages_free", "lora_pages_compact", "lora_kv_copy",
           "BlockSelection", "lora_kv_bounds", "lora_block_select", "lora_block_attention",
           "KIND_ROWS_FUSED", "KIND_SHRINK", "KIND_EXPAND", "KIND_TILE_FUSED", "KIND_MERGE",
           "OPT_TILE_PATH", "OPT_MERGE_KERNEL", "OPT_TILE_MIN_RUN", "OPT_EARLY_PAGES", "OPT_DEVICE_PLAN",
           "OPT_EARLY_INPUT", "OPT_ROWS_B_OVER_A",
           "library_path"]

KIND_ROWS_FUSED, KIND_SHRINK, KIND_EXPAND, KIND_TILE_FUSED, KIND_MERGE = range(5)
OPT_TILE_PATH, OPT_MERGE_KERNEL, OPT_TILE_MIN_RUN, OPT_EARLY_PAGES, OPT_DEVICE_PLAN = 1, 2, 3, 4, 5
OPT_EARLY_INPUT = 6
OPT_ROWS_B_OVER_A = 7
ERROR_NAMES = {0: "LORA_OK", -1: "LORA_E_INVAL", -2: "LORA_E_RANK", -3: "LORA_E_ADAPTER",
               -4: "LORA_E_NOT_RESIDENT", -5: "LORA_E_PAGE", -6: "LORA_E_CUDA",
               -7: "LORA_E_TIMEOUT", -8: "LORA_E_NOMEM", -9: "LORA_E_CAPACITY",
               -10: "LORA_E_UNSUPPORTED", -11: "LORA_E_IO", -12: "LORA_E_NOTUNED"}

_L = _lib.load()


def library_path() -> str:
    return _lib.LIB_PATH


class LoraError(RuntimeError):
    def __init__(self, code: int, detail: str = ""):
        self.code = code
        self.name = ERROR_NAMES.get(code, str(code))
        msg = f"{self.name}: {_L.lora_strerror(code).decode()}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


def _check(rc: int, ctx: "Context | None" = None) -> int:
    if rc < 0:
        detail = ""
        if rc == -6 and ctx is not None and ctx.handle:
            detail = (_L.lora_last_cuda_error(ctx.handle) or b"").decode()
        raise LoraError(rc, detail)
    return rc


def _stream(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev_ptr(t: torch.Tensor, what: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    return t.data_ptr()


def _ids(ids):
    """(int32 contiguous array, its address, length)."""
    if not (isinstance(ids, np.ndarray) and ids.dtype == np.int32 and ids.flags.c_contiguous):
        ids = np.ascontiguousarray(np.asarray(ids), dtype=np.int32)
    if ids.ndim != 1:
        raise ValueError("ids must be one-dimensional")
    return ids, ids.__array_interface__["data"][0], ids.shape[0]


def _rows(t: torch.Tensor, what: str):
    """(pointer, row stride in elements, columns) of a 2-D row-major 16-bit CUDA tensor."""
    st = t.stride()
    if len(st) != 2 or st[1] != 1 or t.element_size() != 2 or not t.is_cuda:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what} must be a CUDA tensor")
        raise ValueError(f"{what} must be a 2-D row-major bf16 tensor")
    return t.data_ptr(), st[0], t.shape[1]


class Context:
    """A library context on one device (plan staging buffers, status word, tile table)."""

    def __init__(self, device: int = 0, max_rows: int = 1 << 16, max_rank: int = 64):
        """device = -1: host-only context (plans and tile tables, no launches)."""
        if isinstance(device, int) and device < 0:
            self.device, idx, self.device_index = None, -1, None
        else:
            self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
            self.device_index = idx = self.device.index or 0
        h = ctypes.c_void_p()
        self.handle = None
        self._tables = weakref.WeakSet()
        _check(_L.lora_ctx_create(idx, int(max_rows), int(max_rank), ctypes.byref(h)))
        self.handle = h.value

    def close(self):
        """Destroy the context and every table and cache registered with it."""
        if self.handle:
            for t in list(self._tables):
                t.close()
            _L.lora_ctx_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def tiles_load(self, path: str):
        _check(_L.lora_tiles_load(self.handle, path.encode()), self)

    def tiles_save(self, path: str):
        _check(_L.lora_tiles_save(self.handle, path.encode()), self)

    def tiles_count(self) -> int:
        return int(_L.lora_tiles_count(self.handle))

    def tile_status(self) -> str:
        """"LORA_OK" if the last call found all its launch shapes in the tile table,
        "LORA_E_NOTUNED" if it took a built-in default for one of them."""
        return ERROR_NAMES[int(_L.lora_tile_status(self.handle))]

    def tune(self, shapes_path: str, out_path: str | None = None, stream=None):
        """lora_tune: the offline search over a shape file (see include/lora.h); the
        winners go into this context's table, and to out_path if given."""
        _check(_L.lora_tune(self.handle, shapes_path.encode(),
                            out_path.encode() if out_path else None,
                            _stream(stream, self.device) if self.device is not None else None),
               self)

    def sync_status(self, stream=None) -> int:
        """Synchronize and read back what kernels recorded (see include/lora.h): raises on a
        timeout, a device-resident id or a cache batch that could not be served."""
        return _check(_L.lora_sync_status(self.handle, _stream(stream, self.device)), self)

    def selftest_timeout(self, limit_us: int = 10000, stream=None):
        """Launch a bounded wait that runs out (see include/lora.h): the next
        sync_status raises LORA_E_TIMEOUT and the context stays usable."""
        _check(_L.lora_selftest_timeout(self.handle, int(limit_us), _stream(stream, self.device)), self)

    def set_option(self, option: int, value: int):
        """LORA_OPT_* (see include/lora.h): OPT_TILE_PATH, OPT_MERGE_KERNEL,
        OPT_TILE_MIN_RUN, OPT_EARLY_PAGES, OPT_DEVICE_PLAN, OPT_EARLY_INPUT,
        OPT_ROWS_B_OVER_A."""
        _check(_L.lora_ctx_set_option(self.handle, int(option), int(value)), self)

    def profile_begin(self, every: int = 1):
        """Start bracketing every `every`-th kernel launch with CUDA events."""
        _check(_L.lora_profile_begin(self.handle, int(every)), self)

    def profile_end(self):
        """Stop; returns {family: (device ms, launches)} for the row-gather, tile shrink,
        merge and streaming expand kernels: every launch made while profiling, and
        their device time (the bracketed launches' mean times that count)."""
        ms = (ctypes.c_double * 5)()
        n = (ctypes.c_int64 * 5)()
        _check(_L.lora_profile_end(self.handle, ms, n), self)
        return {name: (ms[i], int(n[i]))
                for i, name in enumerate(("rows", "shrink", "merge", "expand", "proj"))}

    def launch_count(self) -> int:
        """Kernels launched by this context so far."""
        return int(_L.lora_launch_count(self.handle))

    def last_path(self):
        """(path bits, launches) of the last call: 1 row-gather, 2 tensor-core tile,
        4 merge, 8 page-in, 16 base projection, 32 cache write / read, 64 attention of few
        rows, 128 attention of many, 256 norms and rotation of heads, 512 page tables, 1024 page
        copies, 2048 bounds and choice of pages."""
        n = ctypes.c_int()
        p = _L.lora_last_path(self.handle, ctypes.byref(n))
        return p, n.value


class AdapterTable:
    """Registered adapter table over caller-owned device pools of bf16 pages.

    a_pool / b_pool: CUDA tensors [n_pages, page_width] (bf16 or 16-bit ints); may be
    the same tensor.  rank, scale: [n_adapters]; a_pages, b_pages: [n_adapters,
    max_rank] page ids (-1 = not resident).  The pools are kept referenced here so
    they outlive the table."""

    def __init__(self, ctx: Context, a_pool: torch.Tensor, b_pool: torch.Tensor, rank, scale,
                 a_pages, b_pages):
        self.ctx = ctx
        self.a_pool, self.b_pool = a_pool, b_pool
        for t, nm in ((a_pool, "a_pool"), (b_pool, "b_pool")):
            if t.dim() != 2 or t.element_size() != 2 or not t.is_contiguous():
                raise ValueError(f"{nm} must be a contiguous 2-D 16-bit tensor")
        self.rank = np.ascontiguousarray(rank, dtype=np.int32)
        self.scale = np.ascontiguousarray(scale, dtype=np.float32)
        self.a_pages = np.ascontiguousarray(a_pages, dtype=np.int32)
        self.b_pages = np.ascontiguousarray(b_pages, dtype=np.int32)
        n_adapters, max_rank = self.a_pages.shape
        self.n_adapters, self.max_rank = n_adapters, max_rank
        h = ctypes.c_void_p()
        if ctx.device is None:      # host-only context: pools are never dereferenced
            pa, pb = a_pool.data_ptr(), b_pool.data_ptr()
        else:
            pa, pb = _dev_ptr(a_pool, "a_pool"), _dev_ptr(b_pool, "b_pool")
        _check(_L.lora_table_create(
            ctx.handle, pa, a_pool.shape[0], a_pool.shape[1],
            pb, b_pool.shape[0], b_pool.shape[1], n_adapters, max_rank,
            self.rank.ctypes.data, self.scale.ctypes.data, self.a_pages.ctypes.data,
            self.b_pages.ctypes.data, ctypes.byref(h)), ctx)
        self.handle = h.value
        ctx._tables.add(self)

    def invalidate(self, adapter: int = -1):
        """The pages of `adapter` (-1: every adapter) were written outside lora_page_in:
        the table's dense copy of them is stale (see include/lora.h)."""
        _check(_L.lora_table_invalidate(self.handle, int(adapter)))

    def close(self):
        if getattr(self, "handle", None):
            _L.lora_table_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def lora_plan_build(ctx: Context, table: AdapterTable, ids) -> dict:
    """Host-side grouping of one batch (copies of the context's plan arrays)."""
    ids, pid, n = _ids(ids)
    v = _lib.PlanView()
    _check(_L.lora_plan_build(ctx.handle, table.handle, pid, n, ctypes.byref(v)), ctx)

    def arr(p, n):
        return np.ctypeslib.as_array(p, shape=(n,)).copy() if n > 0 else np.zeros(0, np.int32)
    return {"active_rows": arr(v.active_rows, v.n_active), "perm": arr(v.perm, v.n_active),
            "seg_offsets": arr(v.seg_offsets, v.n_segments + 1),
            "seg_adapter": arr(v.seg_adapter, v.n_segments),
            "row_items": int(v.row_items), "tile_items": int(v.tile_items),
            "rows_per_item": int(v.rows_per_item), "tile_min_run": int(v.tile_min_run)}


def lora_shrink(ctx: Context, table: AdapterTable, ids, x: torch.Tensor, v: torch.Tensor,
                stream=None):
    """v[i, :r_k] = x_i A_k (fp32) for rows with ids[i] >= 0."""
    ids, pid, n = _ids(ids)
    px, ldx, d_in = _rows(x, "x")
    if v.dtype != torch.float32 or v.dim() != 2 or v.stride(1) != 1:
        raise ValueError("v must be a 2-D row-major float32 tensor")
    _check(_L.lora_shrink(ctx.handle, table.handle, pid, n, px, ldx, d_in, _dev_ptr(v, "v"),
                          v.stride(0), _stream(stream, ctx.device)), ctx)


def lora_expand(ctx: Context, table: AdapterTable, ids, v: torch.Tensor, y: torch.Tensor,
                stream=None):
    """y_i <- bf16(y_i + s_k v_i B_k) in place for rows with ids[i] >= 0."""
    ids, pid, n = _ids(ids)
    py, ldy, d_out = _rows(y, "y")
    if v.dtype != torch.float32 or v.dim() != 2 or v.stride(1) != 1:
        raise ValueError("v must be a 2-D row-major float32 tensor")
    _check(_L.lora_expand(ctx.handle, table.handle, pid, n, _dev_ptr(v, "v"), v.stride(0), py,
                          ldy, d_out, _stream(stream, ctx.device)), ctx)


def lora_fused(ctx: Context, table: AdapterTable, ids, x: torch.Tensor, y: torch.Tensor,
               stream=None):
    """y_i <- bf16(y_i + s_k (x_i A_k) B_k) in place for rows with ids[i] >= 0."""
    ids, pid, n = _ids(ids)
    px, ldx, d_in = _rows(x, "x")
    py, ldy, d_out = _rows(y, "y")
    rc = _L.lora_fused(ctx.handle, table.handle, pid, n, px, ldx, d_in, py, ldy, d_out,
                       _stream(stream, ctx.device))
    if rc:
        _check(rc, ctx)


def lora_fused_device_ids(ctx: Context, table: AdapterTable, ids: torch.Tensor, x: torch.Tensor,
                          y: torch.Tensor, stream=None):
    """lora_fused with the ids in device memory (a CUDA int32 tensor [n], -1 =
    released): planned on the GPU, nothing read on the host, graph-capturable.  An
    id the table cannot serve leaves its row unchanged and shows up as
    LORA_E_ADAPTER at the next sync_status (see include/lora.h)."""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda or ids.dtype != torch.int32 or \
            ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 1-D int32 CUDA tensor")
    px, ldx, d_in = _rows(x, "x")
    py, ldy, d_out = _rows(y, "y")
    _check(_L.lora_fused_device_ids(ctx.handle, table.handle, ids.data_ptr(), ids.shape[0], px,
                                    ldx, d_in, py, ldy, d_out, _stream(stream, ctx.device)), ctx)


def lora_base_fused(ctx: Context, table: AdapterTable, ids, x: torch.Tensor, W: torch.Tensor,
                    y: torch.Tensor, stream=None):
    """y_i <- bf16(x_i W + s_k (x_i A_k) B_k) (x_i W alone for ids[i] == -1): the base
    projection with the adapter term in one tensor-core GEMM; y is written, not read.
    W is [d_in, d_out] row-major."""
    ids, pid, n = _ids(ids)
    px, ldx, d_in = _rows(x, "x")
    pw, ldw, d_out = _rows(W, "W")
    py, ldy, d_out_y = _rows(y, "y")
    if W.shape[0] != d_in or d_out_y != d_out:
        raise ValueError("shapes: x [n, d_in], W [d_in, d_out], y [n, d_out]")
    _check(_L.lora_base_fused(ctx.handle, table.handle, pid, n, px, ldx, d_in, pw, ldw, py, ldy,
                              d_out, _stream(stream, ctx.device)), ctx)


def lora_fused_noalloc(ctx: Context, table: AdapterTable, ids, x: torch.Tensor, y: torch.Tensor,
                       stream=None):
    """lora_fused for callers that must not allocate while it runs: its scratch is
    fixed device arrays inside the library (12 MB: 4 MB of partial V and 8 MB of
    dense adapter rows, committed when a context is created); raises
    LORA_E_CAPACITY beyond their limits (see include/lora.h)."""
    ids, pid, n = _ids(ids)
    px, ldx, d_in = _rows(x, "x")
    py, ldy, d_out = _rows(y, "y")
    _check(_L.lora_fused_noalloc(ctx.handle, table.handle, pid, n, px, ldx, d_in, py, ldy, d_out,
                                 _stream(stream, ctx.device)), ctx)


class _PreparedCall:
    """A fused call with fixed x, y, table and stream (a decode loop's persistent
    buffers).  The marshalling happens once: for each ids object among the last 256
    it was handed, a filled lora_fused_args block is kept, and a call passes only
    that block's address.  Only the object is recognised, never its contents: the
    library reads the ids on every call."""

    _KEEP = 256
    _ENTRY = ""

    def __init__(self, ctx: Context, table: AdapterTable, x: torch.Tensor, y: torch.Tensor,
                 stream=None):
        px, ldx, d_in = _rows(x, "x")
        py, ldy, d_out = _rows(y, "y")
        self._keep = (ctx, table, x, y)
        self._ctx = ctx
        self._fn = _lib.untyped(self._ENTRY)
        self._fields = dict(ctx=ctx.handle, table=table.handle, x=px, ldx=ldx, d_in=d_in, y=py,
                            ldy=ldy, d_out=d_out, stream=_stream(stream, ctx.device))
        # id(ids object) -> (the object, kept alive so its id stays its own; its
        # argument block; the block's address)
        self._seen = {}

    def _ids_ptr(self, ids):
        raise NotImplementedError

    def _block(self, ids):
        ptr, n, keep = self._ids_ptr(ids)
        blk = _lib.FusedArgs(ids=ptr, n=n, **self._fields)
        ref = ctypes.byref(blk)
        if keep:
            if len(self._seen) >= self._KEEP:
                self._seen.pop(next(iter(self._seen)))
            self._seen[id(ids)] = (ids, blk, ref)
        return blk, ref

    def bind(self, ids):
        """Convert and keep the arguments for this ids object without launching, so
        that the first call with it costs no more than the later ones."""
        self._block(ids)

    def __call__(self, ids):
        hit = self._seen.get(id(ids))
        if hit is not None and hit[0] is ids:
            rc = self._fn(hit[2])
        else:
            blk, ref = self._block(ids)
            rc = self._fn(ref)
        if rc:
            _check(rc, self._ctx)


class PreparedFused(_PreparedCall):
    """lora_fused with fixed x, y, table and stream; call it with the host ids
    (int32 array, -1 = released).  An array used as it is (int32, contiguous) is
    remembered, so a persistent ids buffer rewritten in place between steps, or a
    ring of them, costs little more than the C function itself."""

    _ENTRY = "lora_fused_args_call"

    def _ids_ptr(self, ids):
        arr, pid, n = _ids(ids)
        return pid, n, arr is ids


class PreparedFusedDeviceIds(_PreparedCall):
    """lora_fused_device_ids with fixed x, y, table and stream; call it with the ids
    as a contiguous 1-D int32 CUDA tensor (its data pointer and length are taken when
    the tensor is first seen)."""

    _ENTRY = "lora_fused_device_ids_args_call"

    def _ids_ptr(self, ids):
        if not isinstance(ids, torch.Tensor) or not ids.is_cuda or ids.dtype != torch.int32 or \
                ids.dim() != 1 or not ids.is_contiguous():
            raise ValueError("ids must be a contiguous 1-D int32 CUDA tensor")
        return ids.data_ptr(), ids.shape[0], True


def lora_merge(ctx: Context, table: AdapterTable, adapter: int, W: torch.Tensor, stream=None):
    """W <- bf16(W + s_k A_k B_k) in place (W is [d_in, d_out] row-major)."""
    pw, ldw, d_out = _rows(W, "W")
    _check(_L.lora_merge(ctx.handle, table.handle, int(adapter), pw, ldw, W.shape[0], d_out,
                         _stream(stream, ctx.device)), ctx)


def lora_unmerge(ctx: Context, table: AdapterTable, adapter: int, W: torch.Tensor, stream=None):
    """W <- bf16(W - s_k A_k B_k) in place."""
    pw, ldw, d_out = _rows(W, "W")
    _check(_L.lora_unmerge(ctx.handle, table.handle, int(adapter), pw, ldw, W.shape[0], d_out,
                           _stream(stream, ctx.device)), ctx)


def lora_page_in(ctx: Context, table: AdapterTable, adapter: int, host_a: torch.Tensor,
                 host_b: torch.Tensor, stream=None):
    """Copy adapter `adapter`'s A and B into its pages of the table's pools, on
    `stream` (asynchronous).  host_a: [rank, d_in] and host_b: [rank, d_out] bf16 (or
    their 16-bit images) in page-locked CPU memory, contiguous; row j of host_a is
    column j of A_k, row j of host_b is row j of B_k.  Keep both alive and unchanged
    until the stream has passed the call (see include/lora.h)."""
    r = int(table.rank[int(adapter)]) if 0 <= int(adapter) < table.n_adapters else -1
    for name, h in (("host_a", host_a), ("host_b", host_b)):
        if not isinstance(h, torch.Tensor) or h.device.type != "cpu" or not h.is_pinned():
            raise ValueError(f"{name} must be a page-locked CPU tensor")
        if h.dim() != 2 or not h.is_contiguous() or h.element_size() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D 16-bit tensor")
        if r >= 0 and h.shape[0] != r:
            raise ValueError(f"{name} has {h.shape[0]} rows, adapter {adapter} has rank {r}")
    _check(_L.lora_page_in(ctx.handle, table.handle, int(adapter), host_a.data_ptr(),
                           host_a.shape[1], host_b.data_ptr(), host_b.shape[1],
                           _stream(stream, ctx.device)), ctx)


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_KV_FORMATS = {torch.bfloat16: 0, torch.int8: 1, torch.float8_e4m3fn: 2}


class KvCache:
    """A paged key/value cache over caller-owned device pools (see include/lora.h).

    k_pool / v_pool: CUDA tensors [n_pages, page_size, n_heads, head_dim] of bf16, int8 or
    float8_e4m3fn with the same strides, the last dimension contiguous; any other order
    of memory is a view of this shape (heads first: pool.transpose(1, 2)).  k_scale /
    v_scale: float32 [n_pages, page_size, n_heads] with the same strides, for the 8-bit
    types.  The tensors are kept referenced here."""

    def __init__(self, ctx: Context, k_pool: torch.Tensor, v_pool: torch.Tensor,
                 k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None):
        self.handle = None
        for t, nm in ((k_pool, "k_pool"), (v_pool, "v_pool")):
            if t.dim() != 4 or t.dtype not in _KV_FORMATS or t.stride(3) != 1:
                raise ValueError(f"{nm} must be [n_pages, page_size, n_heads, head_dim] of bf16, int8 or "
                                 "float8_e4m3fn with a contiguous last dimension")
        if k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype or \
                k_pool.stride() != v_pool.stride():
            raise ValueError("k_pool and v_pool must have the same shape, type and strides")
        d = _lib.KvDesc()
        d.format = _KV_FORMATS[k_pool.dtype]
        if d.format:
            for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if t is None or t.dtype != torch.float32 or t.shape != k_pool.shape[:3]:
                    raise ValueError(f"{nm} must be float32 [n_pages, page_size, n_heads] for 8-bit pools")
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale must have the same strides")
            d.scale_page_stride, d.scale_cell_stride, d.scale_head_stride = k_scale.stride()
        elif k_scale is not None or v_scale is not None:
            raise ValueError("bf16 pools have no scales")
        d.n_pages, d.page_size, d.n_heads, d.head_dim = k_pool.shape
        d.page_stride, d.cell_stride, d.head_stride = k_pool.stride()[:3]
        if ctx.device is None:      # host-only context: pools are never dereferenced
            self.device_index = None
            ptr = lambda t, nm: t.data_ptr()  # noqa: E731
        else:
            self.device_index = ctx.device.index or 0

            def ptr(t, nm):
                p = _dev_ptr(t, nm)
                if t.get_device() != self.device_index:
                    raise ValueError(f"{nm} must be on the context's device")
                return p
        d.k_pool, d.v_pool = ptr(k_pool, "k_pool"), ptr(v_pool, "v_pool")
        if d.format:
            d.k_scale, d.v_scale = ptr(k_scale, "k_scale"), ptr(v_scale, "v_scale")
        self.ctx = ctx
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = k_pool, v_pool, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads, self.head_dim = k_pool.shape
        h = ctypes.c_void_p()
        _check(_L.lora_kv_create(ctx.handle, ctypes.byref(d), ctypes.byref(h)), ctx)
        self.handle = h.value
        self.bounds = None
        ctx._tables.add(self)

    def attach_bounds(self, codes: torch.Tensor | None, unit: torch.Tensor | None):
        """The memory for each page's smallest and largest keys (see include/lora.h): codes int8
        [n_pages, n_heads, 2, head_dim] and unit float32 [n_pages, n_heads], contiguous; both None
        to detach.  lora_kv_bounds fills it, lora_block_select reads it, lora_kv_copy moves it."""
        if (codes is None) != (unit is None):
            raise ValueError("codes and unit come together")
        if codes is not None:
            for t, nm, dt, sh in ((codes, "codes", torch.int8, (self.n_pages, self.n_heads, 2, self.head_dim)),
                                  (unit, "unit", torch.float32, (self.n_pages, self.n_heads))):
                if not isinstance(t, torch.Tensor) or t.dtype != dt or tuple(t.shape) != sh or not t.is_contiguous():
                    raise ValueError(f"{nm} must be a contiguous {dt} tensor of shape {list(sh)}")
                if self.device_index is not None and (not t.is_cuda or t.get_device() != self.device_index):
                    raise ValueError(f"{nm} must be on the context's device")
        _check(_L.lora_kv_attach_bounds(self.handle, None if codes is None else codes.data_ptr(),
                                        None if unit is None else unit.data_ptr()), self.ctx)
        self.bounds = None if codes is None else (codes, unit)

    def close(self):
        if getattr(self, "handle", None):
            _L.lora_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KvBatch:
    """The sequences of a cache call (see include/lora.h): starts [n_seqs + 1], lens
    [n_seqs] and pages [n_seqs, n_cols], int32 CUDA tensors whose contents the kernels
    read; update them in place between steps (or between replays of a graph).  max_new
    bounds a sequence's new tokens (None: the call's rows)."""

    def __init__(self, starts: torch.Tensor, lens: torch.Tensor, pages: torch.Tensor,
                 max_new: int | None = None):
        for t, nm, dim in ((starts, "starts", 1), (lens, "lens", 1), (pages, "pages", 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dim or \
                    (t.numel() and t.stride(-1) != 1):
                raise ValueError(f"{nm} must be a {dim}-D int32 tensor, contiguous in its last dimension")
        if starts.shape[0] != lens.shape[0] + 1 or pages.shape[0] != lens.shape[0]:
            raise ValueError("shapes: starts [n_seqs + 1], lens [n_seqs], pages [n_seqs, n_cols]")
        self.starts, self.lens, self.pages = starts, lens, pages
        a = _lib.KvBatchArgs()
        a.starts = _dev_ptr(starts, "starts")
        a.lens = _dev_ptr(lens, "lens")
        a.pages = _dev_ptr(pages, "pages")
        self.device_index = starts.get_device()
        if lens.get_device() != self.device_index or pages.get_device() != self.device_index:
            raise ValueError("starts, lens and pages must be on one device")
        a.n_seqs, a.n_cols = pages.shape
        a.ld_pages = max(pages.stride(0), pages.shape[1]) if pages.shape[0] > 1 else pages.shape[1]
        if pages.shape[0] > 1 and pages.stride(0) < pages.shape[1]:
            raise ValueError("the rows of pages overlap")
        a.max_new = (1 << 31) - 1 if max_new is None else int(max_new)
        self._args = a
        self._ref = ctypes.addressof(a)


def _head_rows(t: torch.Tensor, what: str, cache: KvCache):
    """(pointer, row stride, rows, heads) of bf16 rows [n, heads, head_dim] (the heads one
    after another) or [n, heads * head_dim] on the cache's device."""
    head_dim = cache.head_dim
    try:
        sh, st = t.shape, t.stride()
        if len(sh) == 3:
            n, heads, width = sh
            ok = width == head_dim and st[2] == 1 and (heads == 1 or st[1] == head_dim)
        else:
            n, width = sh
            heads = width // head_dim
            ok = st[1] == 1 and heads * head_dim == width
        ok = ok and t.dtype is torch.bfloat16 and t.get_device() == cache.device_index
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{what} must be a CUDA tensor")
        if t.get_device() != cache.device_index:
            raise ValueError(f"{what} must be on the context's device")
        raise ValueError(f"{what} must be bf16 [n, heads, {head_dim}] or [n, heads * {head_dim}] rows")
    # the stride of a single row says nothing
    return t.data_ptr(), st[0] if n > 1 else heads * head_dim, n, heads


def _raw_stream(stream, ctx: Context):
    """_stream for the calls of a decode loop: the current stream's handle without a
    Stream object around it."""
    if stream is None and _current_raw_stream is not None and ctx.device is not None:
        return _current_raw_stream(ctx.device_index)
    return _stream(stream, ctx.device)


def _kv_rows(ctx, cache, batch, k, v, stream, fn):
    pk, ldk, n, hk = _head_rows(k, "k", cache)
    pv, ldv, nv, hv = _head_rows(v, "v", cache)
    if batch.device_index != cache.device_index:
        raise ValueError("the batch must be on the context's device")
    if nv != n or hk != cache.n_heads or hv != cache.n_heads:
        raise ValueError("k and v must have one row a token and the cache's heads")
    rc = fn(ctx.handle, cache.handle, batch._ref, n, pk, ldk, pv, ldv, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_kv_write(ctx: Context, cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor,
                  stream=None):
    """Store the batch's new keys and values (bf16 [n, n_heads, head_dim]) in their cells,
    in the cache's format."""
    _kv_rows(ctx, cache, batch, k, v, stream, _L.lora_kv_write)


def lora_kv_read(ctx: Context, cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor,
                 stream=None):
    """The cells of the batch's rows back as bf16 rows k and v (written)."""
    _kv_rows(ctx, cache, batch, k, v, stream, _L.lora_kv_read)


def lora_attention(ctx: Context, cache: KvCache, batch: KvBatch, q: torch.Tensor, out: torch.Tensor,
                   scale: float | None = None, window: int = 0, sinks: int = 0, stream=None):
    """out <- attention of the batch's new tokens (q, bf16 [n, heads, head_dim]) over the
    cache, which already holds their keys and values: causal by position, with a sliding
    window and `sinks` first tokens that stay visible when window > 0.  scale: None for
    head_dim ** -0.5."""
    pq, ldq, n, hq = _head_rows(q, "q", cache)
    po, ldo, no, ho = _head_rows(out, "out", cache)
    if batch.device_index != cache.device_index:
        raise ValueError("the batch must be on the context's device")
    if no != n or ho != hq:
        raise ValueError("out must have the shape of q")
    if scale is None:
        scale = cache.head_dim ** -0.5
    if (window | sinks) >> 31:      # beyond an int: no position is that far away; negative: refused
        window, sinks = (max(-1, min(v, (1 << 31) - 1)) for v in (window, sinks))
    rc = _L.lora_attention(ctx.handle, cache.handle, batch._ref, n, pq, ldq, hq, scale, window, sinks,
                           po, ldo, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


class HeadRope:
    """What lora_head_rope does to each head (see include/lora.h): freqs, float32 [pairs] on the
    GPU, turns the first 2 * pairs elements (None: no rotation), as pairs (j, j + pairs) or, when
    interleaved, (2j, 2j + 1); q_weight and k_weight [head_dim], where given, are the weights of
    the norms (kept as float32: another type is converted here, once, on the current stream)."""

    def __init__(self, freqs: torch.Tensor | None, head_dim: int, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False):
        self.head_dim, self.device_index = int(head_dim), None
        r = _lib.Rope()
        r.eps, r.head_dim, r.interleaved = float(eps), self.head_dim, int(bool(interleaved))
        if freqs is not None and freqs.numel() == 0:
            freqs = None
        kept = {}
        for t, nm, field in ((freqs, "freqs", "freqs"), (q_weight, "q_weight", "q_weight"), (k_weight, "k_weight", "k_weight")):
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or t.dim() != 1 or not t.is_floating_point():
                raise ValueError(f"{nm} must be a 1-D tensor of floating point")
            if nm == "freqs":
                if t.dtype != torch.float32:
                    raise ValueError("freqs must be float32")
            elif t.shape[0] != self.head_dim:
                raise ValueError(f"{nm} must have head_dim elements")
            t = t.float().contiguous()
            if t.data_ptr() % 16:
                t = t.clone()
            setattr(r, field, _dev_ptr(t, nm))
            if self.device_index is not None and t.get_device() != self.device_index:
                raise ValueError("freqs, q_weight and k_weight must be on one device")
            self.device_index = t.get_device()
            kept[nm] = t
        r.rot_dim = 0 if freqs is None else 2 * freqs.shape[0]
        self._kept, self._args = kept, r
        self._ref = ctypes.addressof(r)


class _HeadsOn:
    """What _head_rows looks at, for rows that go with no cache."""

    def __init__(self, head_dim, device_index):
        self.head_dim, self.device_index = head_dim, device_index


def _alike(x, y, where):
    """(pointer, stride, rows, heads, pointer, stride) of two tensors of bf16 rows [n, heads, head_dim] of
    the same shape, or None where they are not that: _head_rows says what is wrong."""
    try:
        sh, st, so, dev = x.shape, x.stride(), y.stride(), where.device_index
        n, heads, width = sh
        if x.dtype is torch.bfloat16 and y.dtype is torch.bfloat16 and width == where.head_dim and \
                st[1] == so[1] == width and st[2] == so[2] == 1 and y.shape == sh and x.get_device() == y.get_device() == dev:
            # the stride of a single row says nothing
            return x.data_ptr(), st[0] if n > 1 else heads * width, n, heads, y.data_ptr(), so[0] if n > 1 else heads * width
    except (AttributeError, ValueError):
        pass
    return None


def _rope_side(x, out, what, where):
    """The same of a side and where it goes, which has its shape."""
    both = _alike(x, out, where)
    if both is None:
        px, ldx, n, heads = _head_rows(x, what, where)
        po, ldo, no, ho = _head_rows(out, what + "_out", where)
        if no != n or ho != heads:
            raise ValueError(f"{what}_out must have the shape of {what}")
        both = px, ldx, n, heads, po, ldo
    return both


def _rope_on(ctx, rope, batch, head_dim):
    """What the rows have to be like: head_dim elements a head, on the context's device."""
    dev = batch.device_index
    if dev != ctx.device_index:
        raise ValueError("the batch must be on the context's device")
    if rope.head_dim != head_dim:
        raise ValueError("the rotation is of another head_dim than the cache")
    if rope.device_index == dev:
        return rope
    if rope.device_index is not None:
        raise ValueError("the rotation's tensors must be on the context's device")
    return _HeadsOn(head_dim, dev)


def lora_head_rope(ctx: Context, rope: HeadRope, batch: KvBatch, q: torch.Tensor | None, k: torch.Tensor | None,
                   q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norms and rotation of q and k (bf16 [n, heads, head_dim]; either may be None) by the
    positions of the batch's new tokens, into q_out and k_out (None: in place)."""
    if q is None and k is None:
        raise ValueError("q or k has to be there")
    where = _rope_on(ctx, rope, batch, rope.head_dim)
    pq, ldq, nq, hq, pqo, ldqo = (0,) * 6 if q is None else _rope_side(q, q if q_out is None else q_out, "q", where)
    pk, ldk, nk, hk, pko, ldko = (0,) * 6 if k is None else _rope_side(k, k if k_out is None else k_out, "k", where)
    if q is not None and k is not None and nq != nk:
        raise ValueError("q and k must have one row a token")
    rc = _L.lora_head_rope(ctx.handle, rope._ref, batch._ref, nk if q is None else nq, pq, ldq, hq, pqo, ldqo,
                           pk, ldk, hk, pko, ldko, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_kv_write_rope(ctx: Context, cache: KvCache, rope: HeadRope, batch: KvBatch, q: torch.Tensor | None,
                       k: torch.Tensor, v: torch.Tensor, q_out: torch.Tensor | None = None, stream=None):
    """lora_head_rope and lora_kv_write in one pass: q, normed and rotated, into q_out (None:
    in place), k, normed and rotated, and v, as it is, into their cells."""
    where = _rope_on(ctx, rope, batch, cache.head_dim)
    if where.device_index != cache.device_index:
        raise ValueError("the batch must be on the context's device")
    both = _alike(k, v, cache)
    if both is not None:
        pk, ldk, n, hk, pv, ldv = both
        nv, hv = n, hk
    else:
        pk, ldk, n, hk = _head_rows(k, "k", cache)
        pv, ldv, nv, hv = _head_rows(v, "v", cache)
    pq, ldq, nq, hq, pqo, ldqo = (0, 0, n, 0, 0, 0) if q is None else _rope_side(q, q if q_out is None else q_out, "q", where)
    if nv != n or nq != n or hk != cache.n_heads or hv != cache.n_heads:
        raise ValueError("q, k and v must have one row a token, k and v the cache's heads")
    rc = _L.lora_kv_write_rope(ctx.handle, cache.handle, rope._ref, batch._ref, n, pq, ldq, hq, pqo, ldqo,
                               pk, ldk, pv, ldv, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def _ints(t: torch.Tensor, what: str, device: int, n: int | None = None) -> int:
    """Pointer of a contiguous 1-D int32 tensor (of n elements) on a device."""
    try:
        sh = t.shape
        if t.dtype is torch.int32 and t.get_device() == device and len(sh) == 1 and (n is None or sh[0] == n) and \
                (sh[0] <= 1 or t.stride()[0] == 1):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{what} must be on the context's device")
    raise ValueError(f"{what} must be a contiguous int32 tensor [{'n' if n is None else n}]")


PAGE_PINNED = 1 << 30


class PageTable:
    """Which sequence holds which pages (see include/lora.h): lens [n_seqs], pages [n_seqs,
    n_cols] and refs [n_pages], int32 CUDA tensors that the lora_pages_* calls change.  lens and
    pages may be a KvBatch's.  refs[page] |= PAGE_PINNED keeps a page that something else uses,
    an adapter's in a unified pool for instance, where it is."""

    def __init__(self, lens: torch.Tensor, pages: torch.Tensor, refs: torch.Tensor, page_size: int):
        for t, nm, dim in ((lens, "lens", 1), (pages, "pages", 2), (refs, "refs", 1)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dim or \
                    (t.numel() and t.stride(-1) != 1):
                raise ValueError(f"{nm} must be a {dim}-D int32 tensor, contiguous in its last dimension")
        if pages.shape[0] != lens.shape[0]:
            raise ValueError("shapes: lens [n_seqs], pages [n_seqs, n_cols], refs [n_pages]")
        if pages.shape[0] > 1 and pages.stride(0) < pages.shape[1]:
            raise ValueError("the rows of pages overlap")
        self.lens, self.pages, self.refs, self.page_size = lens, pages, refs, int(page_size)
        a = _lib.PageTableArgs()
        a.lens, a.pages, a.refs = _dev_ptr(lens, "lens"), _dev_ptr(pages, "pages"), _dev_ptr(refs, "refs")
        self.device_index = lens.get_device()
        if pages.get_device() != self.device_index or refs.get_device() != self.device_index:
            raise ValueError("lens, pages and refs must be on one device")
        a.n_seqs, a.n_cols = pages.shape
        a.ld_pages = max(pages.stride(0), pages.shape[1]) if pages.shape[0] > 1 else pages.shape[1]
        a.n_pages, a.page_size = refs.shape[0], self.page_size
        self._args = a
        self._ref = ctypes.addressof(a)


def _table_on(ctx: Context, table: PageTable) -> int:
    if table.device_index != ctx.device_index:
        raise ValueError("the page table must be on the context's device")
    return table.device_index


def lora_pages_extend(ctx: Context, table: PageTable, grow: torch.Tensor, got: torch.Tensor, src: torch.Tensor,
                      dst: torch.Tensor, cells: torch.Tensor, stream=None):
    """Sequence s grows by grow[s] tokens, as far as the free pages go: got[s] is what it got.
    src, dst and cells are the pages to copy (lora_kv_copy) before the new tokens are written.
    All int32 [n_seqs].  A batch that has rows for sequences that got none takes the lengths
    torch.where(got == grow, table.lens, 0): table.lens would have them replace tokens that are there."""
    dev, n = _table_on(ctx, table), table.lens.shape[0]
    rc = _L.lora_pages_extend(ctx.handle, table._ref, _ints(grow, "grow", dev, n), _ints(got, "got", dev, n),
                              _ints(src, "src", dev, n), _ints(dst, "dst", dev, n), _ints(cells, "cells", dev, n),
                              _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_pages_fork(ctx: Context, table: PageTable, parents: torch.Tensor, children: torch.Tensor, stream=None):
    """Sequence children[i], empty so far, becomes a copy of parents[i] that shares its pages."""
    dev = _table_on(ctx, table)
    n = children.shape[0]
    rc = _L.lora_pages_fork(ctx.handle, table._ref, _ints(parents, "parents", dev, n), _ints(children, "children", dev), n,
                            _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_pages_free(ctx: Context, table: PageTable, seqs: torch.Tensor, keep: torch.Tensor | None = None, stream=None):
    """Sequence seqs[i] is cut to its first keep[i] tokens (None: none) and gives the other pages back."""
    dev = _table_on(ctx, table)
    n = seqs.shape[0]
    rc = _L.lora_pages_free(ctx.handle, table._ref, _ints(seqs, "seqs", dev),
                            None if keep is None else _ints(keep, "keep", dev, n), n, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_pages_compact(ctx: Context, table: PageTable, src: torch.Tensor, dst: torch.Tensor,
                       top: torch.Tensor | None = None, stream=None):
    """Moves held pages to the front of the pool, pinned ones apart, as many as src and dst (int32
    [n]) list: the moves for lora_kv_copy, -1 behind the last.  top (int32 [1]) becomes the end of the highest
    held page."""
    dev = _table_on(ctx, table)
    n = src.shape[0]
    rc = _L.lora_pages_compact(ctx.handle, table._ref, _ints(src, "src", dev), _ints(dst, "dst", dev, n), n,
                               None if top is None else _ints(top, "top", dev, 1), _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_kv_copy(ctx: Context, caches, src: torch.Tensor, dst: torch.Tensor, cells: torch.Tensor | None = None,
                 stream=None):
    """Page src[i] to page dst[i] in every one of `caches` (a KvCache or a sequence of them, alike in
    page size, heads, head_dim and format): the first cells[i] cells, or all.  src[i] < 0: nothing."""
    if isinstance(caches, KvCache):
        caches = (caches,)
    if not caches or ctx.device is None:
        raise ValueError("no caches, or a context without a device")
    dev, n = ctx.device_index, src.shape[0]
    handles = (ctypes.c_void_p * len(caches))(*[c.handle for c in caches])
    rc = _L.lora_kv_copy(ctx.handle, handles, len(caches), _ints(src, "src", dev), _ints(dst, "dst", dev, n),
                         None if cells is None else _ints(cells, "cells", dev, n), n, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


class BlockSelection:
    """The pages chosen for each row and key head (see include/lora.h): lens int32 [rows] and pages
    int32 [rows, key heads, blocks], contiguous CUDA tensors that lora_block_select writes and
    lora_block_attention reads."""

    def __init__(self, lens: torch.Tensor, pages: torch.Tensor):
        for t, nm, dim in ((lens, "lens", 1), (pages, "pages", 3)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
                raise ValueError(f"{nm} must be a contiguous {dim}-D int32 tensor")
        if pages.shape[0] != lens.shape[0]:
            raise ValueError("shapes: lens [rows], pages [rows, key heads, blocks]")
        self.lens, self.pages = lens, pages
        a = _lib.BlockSel()
        a.lens, a.pages = _dev_ptr(lens, "lens"), _dev_ptr(pages, "pages")
        self.device_index = lens.get_device()
        if pages.get_device() != self.device_index:
            raise ValueError("lens and pages must be on one device")
        a.n_rows, self.heads, a.blocks = pages.shape
        self._args = a
        self._ref = ctypes.addressof(a)

    @classmethod
    def empty(cls, rows: int, cache: KvCache, blocks: int) -> "BlockSelection":
        """A selection with new tensors for up to `rows` rows over a cache."""
        dev = cache.k_pool.device
        return cls(torch.empty(rows, dtype=torch.int32, device=dev),
                   torch.empty((rows, cache.n_heads, blocks), dtype=torch.int32, device=dev))


def lora_kv_bounds(ctx: Context, cache: KvCache, batch: KvBatch, rows: int, stream=None):
    """Brings up to date the attached bounds of the pages in which the batch's new tokens (`rows`
    of them, already written) lie."""
    if batch.device_index != cache.device_index:
        raise ValueError("the batch must be on the context's device")
    rc = _L.lora_kv_bounds(ctx.handle, cache.handle, batch._ref, rows, _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def _selected(cache: KvCache, selection: BlockSelection, rows: int):
    if selection.device_index != cache.device_index:
        raise ValueError("the selection must be on the context's device")
    if selection.heads != cache.n_heads or selection.lens.shape[0] < rows:
        raise ValueError("the selection must have the cache's heads and a place for every row")


def lora_block_select(ctx: Context, cache: KvCache, batch: KvBatch, q: torch.Tensor, selection: BlockSelection,
                      first: int = 1, last: int = 1, stream=None):
    """Chooses pages for the batch's new tokens (q, bf16 [n, heads, head_dim]): the first and the
    last ones, and those whose bounds score highest."""
    pq, ldq, n, hq = _head_rows(q, "q", cache)
    if batch.device_index != cache.device_index:
        raise ValueError("the batch must be on the context's device")
    _selected(cache, selection, n)
    rc = _L.lora_block_select(ctx.handle, cache.handle, batch._ref, n, pq, ldq, hq, first, last, selection._ref,
                              _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_block_attention(ctx: Context, cache: KvCache, selection: BlockSelection, q: torch.Tensor, out: torch.Tensor,
                         scale: float | None = None, stream=None):
    """out <- attention of q (bf16 [n, heads, head_dim]) over the pages chosen for each row.
    scale: None for head_dim ** -0.5."""
    both = _alike(q, out, cache)
    if both is not None:
        pq, ldq, n, hq, po, ldo = both
    else:
        pq, ldq, n, hq = _head_rows(q, "q", cache)
        po, ldo, no, ho = _head_rows(out, "out", cache)
        if no != n or ho != hq:
            raise ValueError("out must have the shape of q")
    _selected(cache, selection, n)
    if scale is None:
        scale = cache.head_dim ** -0.5
    rc = _L.lora_block_attention(ctx.handle, cache.handle, selection._ref, n, pq, ldq, hq, scale, po, ldo,
                                 _raw_stream(stream, ctx))
    if rc:
        _check(rc, ctx)


def lora_tune_shape(ctx: Context, table: AdapterTable, kind: int, ids, x: torch.Tensor,
                    y: torch.Tensor, iters: int = 20, stream=None) -> float:
    """Offline search for one shape (see include/lora.h); returns the best time in us
    and keeps the winning configuration in the context's table.  For KIND_MERGE, x is
    W, y is ignored and ids[0] is the adapter."""
    ids, pid, n = _ids(ids)
    px, ldx, d_in = _rows(x, "x")
    if kind == KIND_MERGE:
        py, ldy, d_out = px, ldx, d_in
        d_in = x.shape[0]
    else:
        py, ldy, d_out = _rows(y, "y")
    best = ctypes.c_float()
    _check(_L.lora_tune_shape(ctx.handle, table.handle, int(kind), pid, n, px, ldx, d_in, py,
                              ldy, d_out, int(iters),
                              ctypes.byref(best), _stream(stream, ctx.device)), ctx)
    return float(best.value)
